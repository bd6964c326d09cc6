// api_common.cuh -- what the C entry points share on the host: argument
// checks, the per-device set-up, stream-ordered scratch and the launch count
// (defined in selscan_api.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "selscan.h"

namespace selscan {

constexpr int kMaxDevices = 64;

// Bit of the device error word: a slot or a sequence start that the kernel
// refused (the bounded waits' bits are in scan_diag.cuh).
constexpr unsigned int kErrIndex = 0x100u;

struct DeviceInfo {
    bool ready = false;
    int sm_count = 0;
    unsigned int *err = nullptr;
};

// The current device's number and data (device error word, SM count).
selscan_status device_setup(int *dev_out, DeviceInfo **info_out);

// Status of the launch just made; counts it when it succeeded.
cudaError_t counted_launch();

// Stream-ordered scratch memory; give it back with cudaFreeAsync.
cudaError_t scratch_alloc(void **p, size_t bytes, cudaStream_t stream);

unsigned long long default_timeout_ns();

inline size_t elem_size(int32_t dt) { return dt == SELSCAN_BF16 ? 2 : 4; }

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int64_t numel(const selscan_tensor *t)
{
    int64_t n = 1;
    for (int i = 0; i < t->ndim && i < 4; ++i)
        n *= t->shape[i];
    return n;
}

// Present: non-NULL descriptor whose data is non-NULL, or that holds no
// element at all (frameworks hand out NULL data for empty tensors).
inline bool present(const selscan_tensor *t)
{
    return t && (t->data || (t->ndim >= 1 && t->ndim <= 4 && numel(t) == 0));
}

// A "sequence" tensor: rank 3 (outer0, outer1, L) with time stride 1 and
// 16-byte aligned rows, as the bulk tensor copies need.
inline selscan_status check_seq(const selscan_tensor *t, int64_t d0, int64_t d1, int64_t L,
                         int32_t dtype)
{
    if (!present(t))
        return SELSCAN_ERR_NULL;
    if (t->ndim != 3 || t->shape[0] != d0 || t->shape[1] != d1 || t->shape[2] != L)
        return SELSCAN_ERR_SHAPE;
    if (t->dtype != dtype)
        return SELSCAN_ERR_DTYPE;
    if (d0 == 0 || d1 == 0 || L == 0)
        return SELSCAN_OK;  // nothing will be read or written
    if (L > 1 && t->stride[2] != 1)
        return SELSCAN_ERR_STRIDE;
    if (t->stride[0] < 0 || t->stride[1] < 0)
        return SELSCAN_ERR_STRIDE;
    const int64_t es = int64_t(elem_size(dtype));
    if (!aligned16(t->data) || ((t->stride[0] * es) & 15) || ((t->stride[1] * es) & 15))
        return SELSCAN_ERR_ALIGN;
    return SELSCAN_OK;
}

// A small fp32 parameter tensor with the given shape, contiguous.
inline selscan_status check_param(const selscan_tensor *t, int ndim, const int64_t *shape,
                           bool nullable)
{
    if (!t || !t->data) {
        if (nullable)
            return SELSCAN_OK;
        if (!present(t))
            return SELSCAN_ERR_NULL;
    }
    if (t->ndim != ndim)
        return SELSCAN_ERR_SHAPE;
    int64_t expect = 1, count = 1;
    for (int i = ndim - 1; i >= 0; --i) {
        if (t->shape[i] != shape[i])
            return SELSCAN_ERR_SHAPE;
        count *= shape[i];
    }
    for (int i = ndim - 1; i >= 0 && count > 0; --i) {
        if (shape[i] > 1 && t->stride[i] != expect)
            return SELSCAN_ERR_STRIDE;
        expect *= shape[i];
    }
    if (t->dtype != SELSCAN_F32)
        return SELSCAN_ERR_DTYPE;
    if ((reinterpret_cast<uintptr_t>(t->data) & 3u) != 0)
        return SELSCAN_ERR_ALIGN;
    return SELSCAN_OK;
}

inline const void *opt_data(const selscan_tensor *t) { return (t && t->data) ? t->data : nullptr; }


// A per-token tensor (d0, d1): any non-negative element strides, element-
// aligned data.
inline selscan_status check_tok(const selscan_tensor *t, int64_t d0, int64_t d1, int32_t dtype)
{
    if (!present(t))
        return SELSCAN_ERR_NULL;
    if (t->ndim != 2 || t->shape[0] != d0 || t->shape[1] != d1)
        return SELSCAN_ERR_SHAPE;
    if (t->dtype != dtype)
        return SELSCAN_ERR_DTYPE;
    if (d0 == 0 || d1 == 0)
        return SELSCAN_OK;
    if (t->stride[0] < 0 || t->stride[1] < 0)
        return SELSCAN_ERR_STRIDE;
    if (reinterpret_cast<uintptr_t>(t->data) % elem_size(dtype))
        return SELSCAN_ERR_ALIGN;
    return SELSCAN_OK;
}

// B or C of one token: (batch, N) or (batch, G, N); returns G through *G.
inline selscan_status check_tok_bc(const selscan_tensor *t, int64_t batch, int64_t N, int32_t dtype,
                            int64_t *G, int64_t s[3])
{
    if (!present(t))
        return SELSCAN_ERR_NULL;
    if (t->dtype != dtype)
        return SELSCAN_ERR_DTYPE;
    if (t->ndim == 2) {
        if (t->shape[0] != batch || t->shape[1] != N)
            return SELSCAN_ERR_SHAPE;
        *G = 1;
        s[0] = t->stride[0];
        s[1] = 0;
        s[2] = t->stride[1];
    } else if (t->ndim == 3) {
        if (t->shape[0] != batch || t->shape[2] != N || t->shape[1] <= 0)
            return SELSCAN_ERR_SHAPE;
        *G = t->shape[1];
        s[0] = t->stride[0];
        s[1] = t->stride[1];
        s[2] = t->stride[2];
    } else {
        return SELSCAN_ERR_SHAPE;
    }
    if (s[0] < 0 || s[1] < 0 || s[2] < 0)
        return SELSCAN_ERR_STRIDE;
    if (numel(t) > 0 && reinterpret_cast<uintptr_t>(t->data) % elem_size(dtype))
        return SELSCAN_ERR_ALIGN;
    return SELSCAN_OK;
}

// A vector of n 32-bit indexes on the device, contiguous.
inline selscan_status check_index(const selscan_tensor *t, int64_t n, bool nullable)
{
    if (!t || !t->data) {
        if (nullable && !t)
            return SELSCAN_OK;
        if (!present(t))
            return SELSCAN_ERR_NULL;
    }
    if (t->ndim != 1 || t->shape[0] != n)
        return SELSCAN_ERR_SHAPE;
    if (t->dtype != SELSCAN_I32)
        return SELSCAN_ERR_DTYPE;
    if (n > 1 && t->stride[0] != 1)
        return SELSCAN_ERR_STRIDE;
    if (reinterpret_cast<uintptr_t>(t->data) & 3u)
        return SELSCAN_ERR_ALIGN;
    return SELSCAN_OK;
}

}  // namespace selscan
