// conv.cuh -- the short causal convolution in front of the scan: per channel
// c and token t, with W = 2, 3 or 4 taps,
//
//   v_t = bias_c + sum_{k<W} w[c][k] e_{t-(W-1)+k}      y_t = v_t sigmoid(v_t)
//
// (SiLU optional), where e is the input x behind its W-1 predecessors: an
// initial state, or zeros.  The state of a sequence is its last W-1 inputs.
// The layer around the selective scan filters x with it before the scan
// ("P20 -- Mamba": the block's local convolution).  Gradients, with g_t =
// dy_t (sg + v_t sg (1 - sg)) and sg = sigmoid(v_t) (g = dy without SiLU):
//
//   de_i = sum_k w[k] g_{i+(W-1)-k}   dw[k] = sum_t g_t e_{t-(W-1)+k}   db = sum_t g_t
//
// Every kernel works on blocks of CH channels x TB tokens per thread, held
// as pairs of adjacent channels, so that a 16-byte piece of a token-major
// row (channels contiguous) and of a channels-first row (time contiguous)
// both are whole vectors of the block: a token-major input is turned into a
// channels-first output in registers.  Sums are fp32.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>
#include <type_traits>

#include "api_common.cuh"
#include "f32x2.cuh"
#include "ptx.cuh"
#include "scan_diag.cuh"

namespace selscan {

// ------------------------------------------------- pairs of channels
// A pair of adjacent channels' values at one token, as stored in registers:
// bf16x2 word, or two fp32 in 64 bits.
template <typename T>
struct PairOf;
template <>
struct PairOf<__nv_bfloat16> {
    using type = uint32_t;
    static __device__ __forceinline__ uint64_t f2(uint32_t w) { return bf2_to_f2(w); }
    static __device__ __forceinline__ uint32_t make(__nv_bfloat16 a, __nv_bfloat16 b)
    {
        return uint32_t(__bfloat16_as_ushort(a)) | (uint32_t(__bfloat16_as_ushort(b)) << 16);
    }
    static __device__ __forceinline__ __nv_bfloat16 lo(uint32_t w)
    {
        return __ushort_as_bfloat16((unsigned short)(w & 0xffffu));
    }
    static __device__ __forceinline__ __nv_bfloat16 hi(uint32_t w)
    {
        return __ushort_as_bfloat16((unsigned short)(w >> 16));
    }
    static __device__ __forceinline__ uint32_t round(uint64_t v)
    {
        return pack2_bf16(lo2(v), hi2(v));
    }
};
template <>
struct PairOf<float> {
    using type = uint64_t;
    static __device__ __forceinline__ uint64_t f2(uint64_t w) { return w; }
    static __device__ __forceinline__ uint64_t make(float a, float b) { return pk2(a, b); }
    static __device__ __forceinline__ float lo(uint64_t w) { return lo2(w); }
    static __device__ __forceinline__ float hi(uint64_t w) { return hi2(w); }
    static __device__ __forceinline__ uint64_t round(uint64_t v) { return v; }
};

template <typename T>
using pair_t = typename PairOf<T>::type;

__device__ __forceinline__ float conv_zero(const float *) { return 0.f; }
__device__ __forceinline__ __nv_bfloat16 conv_zero(const __nv_bfloat16 *)
{
    return __ushort_as_bfloat16(0);
}

// CH/2 pairs of one token from CH contiguous channels, and back (CH * sizeof(T)
// is 8 or 16 bytes, aligned).
template <typename T, int CH>
__device__ __forceinline__ void load_row(const T *p, pair_t<T> (&w)[CH / 2])
{
    if constexpr (CH * sizeof(T) == 16) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        if constexpr (sizeof(T) == 2) {
            w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        } else {
            w[0] = uint64_t(v.x) | (uint64_t(v.y) << 32);
            w[1] = uint64_t(v.z) | (uint64_t(v.w) << 32);
        }
    } else {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        if constexpr (sizeof(T) == 2) {
            w[0] = v.x; w[1] = v.y;
        } else {
            w[0] = uint64_t(v.x) | (uint64_t(v.y) << 32);
        }
    }
}

template <typename T, int CH>
__device__ __forceinline__ void store_row(T *p, const pair_t<T> (&w)[CH / 2])
{
    if constexpr (CH * sizeof(T) == 16) {
        uint4 v;
        if constexpr (sizeof(T) == 2)
            v = make_uint4(w[0], w[1], w[2], w[3]);
        else
            v = make_uint4(uint32_t(w[0]), uint32_t(w[0] >> 32), uint32_t(w[1]),
                           uint32_t(w[1] >> 32));
        *reinterpret_cast<uint4 *>(p) = v;
    } else {
        uint2 v;
        if constexpr (sizeof(T) == 2)
            v = make_uint2(w[0], w[1]);
        else
            v = make_uint2(uint32_t(w[0]), uint32_t(w[0] >> 32));
        *reinterpret_cast<uint2 *>(p) = v;
    }
}

// A (batch, dim, L) operand: element strides and whether whole vectors of it
// may be read and written (contiguous in the layout's direction, 16-byte
// aligned base and rows).
struct ConvView {
    void *data;
    int64_t sb, sd, st;
    int vec;
};

// Tokens [t0 - HLO, t0 + TB) of CH channels from c0 of batch row b, as pairs
// xp[channel pair][token].  Tokens before 0 come from `past` (row (b, c) of
// W-1 elements, HLO <= W-1) or are zero, tokens from L on and channels from
// dim on are zero.  TOK: channels are the contiguous direction.
template <typename T, bool TOK, int CH, int TB, int HLO>
__device__ __forceinline__ void load_block(pair_t<T> (&xp)[CH / 2][HLO + TB], const ConvView &v,
                                           const T *past, int past_n, int b, int c0, int t0,
                                           int dim, int L)
{
    constexpr int VEC = 16 / int(sizeof(T));
    const T *base = static_cast<const T *>(v.data) + b * v.sb;
    const T zero = conv_zero(static_cast<const T *>(nullptr));
    const bool whole_c = c0 + CH <= dim;
    const auto at = [&](int c, int t) -> T {
        if (c >= dim || t >= L)
            return zero;
        if (t < 0)
            return past ? past[(int64_t(b) * dim + c) * past_n + past_n + t] : zero;
        return base[c * v.sd + t * v.st];
    };
    if (TOK) {
        if (v.vec && whole_c && (t0 >= HLO || !past)) {
#pragma unroll
            for (int i = 0; i < HLO + TB; ++i) {
                const int t = t0 - HLO + i;
                pair_t<T> w[CH / 2];
#pragma unroll
                for (int q = 0; q < CH / 2; ++q)
                    w[q] = 0;
                if (t >= 0 && t < L)
                    load_row<T, CH>(base + c0 + t * v.st, w);
#pragma unroll
                for (int q = 0; q < CH / 2; ++q)
                    xp[q][i] = w[q];
            }
            return;
        }
    } else if (v.vec && whole_c && t0 + TB <= L && (t0 >= VEC || !past || HLO == 0)) {
        static_assert(TB % VEC == 0, "whole 16-byte pieces of a time row");
#pragma unroll
        for (int q = 0; q < CH / 2; ++q) {
            const T *r0 = base + (c0 + 2 * q) * v.sd + t0;
            const T *r1 = r0 + v.sd;
            const auto put = [&](const T *a, const T *bb, int i0, int from) {
                // VEC tokens of two channels; the first `from` of them are dropped
                if constexpr (sizeof(T) == 2) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(a);
                    const uint4 y = *reinterpret_cast<const uint4 *>(bb);
                    const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        if (i >= from)
                            xp[q][i0 + i - from] =
                                __byte_perm(xs[i / 2], ys[i / 2], i % 2 ? 0x7632 : 0x5410);
                } else {
                    const float4 x = *reinterpret_cast<const float4 *>(a);
                    const float4 y = *reinterpret_cast<const float4 *>(bb);
                    const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        if (i >= from)
                            xp[q][i0 + i - from] = pk2(xs[i], ys[i]);
                }
            };
            if (HLO > 0) {
                if (t0 >= VEC) {
                    put(r0 - VEC, r1 - VEC, 0, VEC - HLO);
                } else {
#pragma unroll
                    for (int i = 0; i < HLO; ++i)
                        xp[q][i] = 0;
                }
            }
#pragma unroll
            for (int j = 0; j < TB / VEC; ++j)
                put(r0 + j * VEC, r1 + j * VEC, HLO + j * VEC, 0);
        }
        return;
    }
#pragma unroll
    for (int q = 0; q < CH / 2; ++q)
#pragma unroll
        for (int i = 0; i < HLO + TB; ++i)
            xp[q][i] = PairOf<T>::make(at(c0 + 2 * q, t0 - HLO + i),
                                       at(c0 + 2 * q + 1, t0 - HLO + i));
}

// The block back: pairs yp[channel pair][token], rounded to T.
template <typename T, bool TOK, int CH, int TB>
__device__ __forceinline__ void store_block(const pair_t<T> (&yp)[CH / 2][TB], const ConvView &v,
                                            int b, int c0, int t0, int dim, int L)
{
    constexpr int VEC = 16 / int(sizeof(T));
    T *base = static_cast<T *>(v.data) + b * v.sb;
    if (TOK) {
        if (v.vec && c0 + CH <= dim) {
#pragma unroll
            for (int i = 0; i < TB; ++i)
                if (t0 + i < L) {
                    pair_t<T> w[CH / 2];
#pragma unroll
                    for (int q = 0; q < CH / 2; ++q)
                        w[q] = yp[q][i];
                    store_row<T, CH>(base + c0 + (t0 + i) * v.st, w);
                }
            return;
        }
    } else if (v.vec && c0 + CH <= dim && t0 + TB <= L) {
#pragma unroll
        for (int q = 0; q < CH / 2; ++q) {
            T *r0 = base + (c0 + 2 * q) * v.sd + t0;
            T *r1 = r0 + v.sd;
#pragma unroll
            for (int j = 0; j < TB / VEC; ++j) {
                if constexpr (sizeof(T) == 2) {
                    uint32_t x[4], y[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t a = yp[q][j * VEC + 2 * i], c = yp[q][j * VEC + 2 * i + 1];
                        x[i] = __byte_perm(a, c, 0x5410);
                        y[i] = __byte_perm(a, c, 0x7632);
                    }
                    *reinterpret_cast<uint4 *>(r0 + j * VEC) = make_uint4(x[0], x[1], x[2], x[3]);
                    *reinterpret_cast<uint4 *>(r1 + j * VEC) = make_uint4(y[0], y[1], y[2], y[3]);
                } else {
                    const int o = j * VEC;
                    *reinterpret_cast<float4 *>(r0 + o) =
                        make_float4(lo2(yp[q][o]), lo2(yp[q][o + 1]), lo2(yp[q][o + 2]),
                                    lo2(yp[q][o + 3]));
                    *reinterpret_cast<float4 *>(r1 + o) =
                        make_float4(hi2(yp[q][o]), hi2(yp[q][o + 1]), hi2(yp[q][o + 2]),
                                    hi2(yp[q][o + 3]));
                }
            }
        }
        return;
    }
#pragma unroll
    for (int q = 0; q < CH / 2; ++q)
#pragma unroll
        for (int i = 0; i < TB; ++i) {
            const int t = t0 + i, c = c0 + 2 * q;
            if (t < L && c < dim)
                base[c * v.sd + t * v.st] = PairOf<T>::lo(yp[q][i]);
            if (t < L && c + 1 < dim)
                base[(c + 1) * v.sd + t * v.st] = PairOf<T>::hi(yp[q][i]);
        }
}

// Taps and bias of CH channels as pairs (zero past dim).
template <int W, int CH>
__device__ __forceinline__ void load_taps(uint64_t (&w)[CH / 2][W], uint64_t (&bias)[CH / 2],
                                          const float *weight, const float *b, int c0, int dim)
{
#pragma unroll
    for (int q = 0; q < CH / 2; ++q) {
        const int c = c0 + 2 * q;
        const bool a0 = c < dim, a1 = c + 1 < dim;
#pragma unroll
        for (int k = 0; k < W; ++k)
            w[q][k] = pk2(a0 ? weight[int64_t(c) * W + k] : 0.f,
                          a1 ? weight[int64_t(c + 1) * W + k] : 0.f);
        bias[q] = pk2(a0 && b ? b[c] : 0.f, a1 && b ? b[c + 1] : 0.f);
    }
}

// v sigmoid(v): the special-function unit for bf16 results (its error, about
// 2^-21, is far below their rounding), the accurate functions for fp32.
template <typename T>
__device__ __forceinline__ uint64_t silu2(uint64_t v)
{
    if constexpr (std::is_same<T, float>::value)
        return pk2(silu_exact(lo2(v)), silu_exact(hi2(v)));
    else
        return pk2(silu_fast(lo2(v)), silu_fast(hi2(v)));
}

template <int W>
__device__ __forceinline__ uint64_t tap_sum(const uint64_t (&w)[W], const uint64_t (&x)[W],
                                            uint64_t bias)
{
    uint64_t v = bias;
#pragma unroll
    for (int k = 0; k < W; ++k)
        v = fma2(w[k], x[k], v);
    return v;
}

// --------------------------------------------------------------- forward
struct ConvParams {
    int batch, dim, L;
    int cg_log2;        // a warp holds 2^cg_log2 channel blocks x 32 / 2^cg_log2 token blocks
    int ctiles, ttiles; // warp tiles over channels and tokens
    ConvView x, y;
    const float *weight;  // (dim, W)
    const float *bias;    // (dim) or null
    const void *h0;       // (batch, dim, W-1) or null
    void *last;           // (batch, dim, W-1) or null
    int silu;
};

// Element i of the state that the sequence ends with: input L-(W-1)+i, taken
// from the initial state where that is before the sequence.
template <typename T, int W>
__device__ __forceinline__ T conv_tail(const T *x, int64_t st, int L, const T *past, int i)
{
    const int t = L - (W - 1) + i;
    if (t >= 0)
        return x[t * st];
    return past ? past[W - 1 + t] : conv_zero(static_cast<const T *>(nullptr));
}

// A thread owns CH channels x TB tokens (16 bytes of either layout); a block
// of four warps holds four neighbouring token tiles, so that the W-1 rows
// that a tile reads from the tile before it come from L1.
template <typename T, int W, bool XTOK, bool YTOK>
__global__ void __launch_bounds__(128) conv_fwd_kernel(const __grid_constant__ ConvParams p)
{
    constexpr int CH = 16 / int(sizeof(T)), TB = CH;
    const int lane = threadIdx.x & 31;
    const int cg = lane & ((1 << p.cg_log2) - 1), tg = lane >> p.cg_log2;
    const int tq = (p.ttiles + 3) >> 2;  // groups of four token tiles
    // neighbouring blocks along the contiguous direction of x
    const int ct = XTOK ? int(blockIdx.x % unsigned(p.ctiles)) : int(blockIdx.x / unsigned(tq));
    const int tt = (XTOK ? int(blockIdx.x / unsigned(p.ctiles)) : int(blockIdx.x % unsigned(tq))) * 4 +
                   int(threadIdx.x >> 5);
    const int b = int(blockIdx.y);
    const int c0 = ((ct << p.cg_log2) + cg) * CH;
    const int64_t tl = (int64_t(tt) * (32 >> p.cg_log2) + tg) * TB;
    if (c0 >= p.dim || tl >= p.L)
        return;
    const int t0 = int(tl);
    const T *past = static_cast<const T *>(p.h0);
    pair_t<T> xp[CH / 2][W - 1 + TB], yp[CH / 2][TB];
    load_block<T, XTOK, CH, TB, W - 1>(xp, p.x, past, W - 1, b, c0, t0, p.dim, p.L);
    uint64_t w[CH / 2][W], bias[CH / 2];
    load_taps<W, CH>(w, bias, p.weight, p.bias, c0, p.dim);
#pragma unroll
    for (int q = 0; q < CH / 2; ++q) {
        uint64_t e[W];
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            e[k + 1] = PairOf<T>::f2(xp[q][k]);
#pragma unroll
        for (int i = 0; i < TB; ++i) {
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
                e[k] = e[k + 1];
            e[W - 1] = PairOf<T>::f2(xp[q][W - 1 + i]);
            uint64_t v = tap_sum<W>(w[q], e, bias[q]);
            if (p.silu)
                v = silu2<T>(v);
            yp[q][i] = PairOf<T>::round(v);
        }
    }
    store_block<T, YTOK, CH, TB>(yp, p.y, b, c0, t0, p.dim, p.L);
    // The owner of a channel's first tokens is the only reader of its initial
    // state, and writes its final state after that: both may be one buffer.
    if (p.last && t0 == 0) {
        const T *xb = static_cast<const T *>(p.x.data) + b * p.x.sb;
        for (int j = 0; j < CH && c0 + j < p.dim; ++j) {
            const int64_t row = (int64_t(b) * p.dim + c0 + j) * (W - 1);
            T tail[W - 1];
#pragma unroll
            for (int i = 0; i < W - 1; ++i)
                tail[i] = conv_tail<T, W>(xb + (c0 + j) * p.x.sd, p.x.st, p.L,
                                          past ? past + row : nullptr, i);
#pragma unroll
            for (int i = 0; i < W - 1; ++i)
                static_cast<T *>(p.last)[row + i] = tail[i];
        }
    }
}

// ------------------------------------------------------- single tokens
struct ConvStepParams {
    int batch, dim, vec;
    const void *x;
    int64_t sx0, sx1;
    void *y;
    int64_t sy0, sy1;
    const float *weight, *bias;
    void *state;       // (slot_count, dim, W-1) contiguous
    const int *slots;  // or null: row b owns slot b
    int slot_count;
    int silu;
    unsigned int *err;
};

// One token of every row: e = [state | x], the state shifted by one.  A
// thread owns CH channels of a row, whose (W-1) CH state elements are W-1
// whole 16-byte vectors (VEC), or one channel (any strides, any dim).
// Slots as in the scan's decode step: negative is padding, a slot past the
// end or owned by an earlier row is refused.
template <typename T, int W, bool VEC>
__global__ void __launch_bounds__(128) conv_step_kernel(const __grid_constant__ ConvStepParams p)
{
    constexpr int CH = VEC ? 16 / int(sizeof(T)) : 1;
    const int b = int(blockIdx.y);
    int64_t row = b;
    if (p.slots) {
        const int slot = p.slots[b];
        if (slot < 0)
            return;
        bool bad = slot >= p.slot_count;
        for (int j = int(threadIdx.x); j < b; j += 128)
            bad |= p.slots[j] == slot;
        if (__syncthreads_or(bad)) {
            if (threadIdx.x == 0)
                atomicOr(p.err, kErrIndex);
            return;
        }
        row = slot;
    }
    const int c0 = (int(blockIdx.x) * 128 + int(threadIdx.x)) * CH;
    if (c0 >= p.dim)
        return;
    T e[CH][W];
    T *st = static_cast<T *>(p.state) + (row * p.dim + c0) * (W - 1);
    const T *x = static_cast<const T *>(p.x) + b * p.sx0 + c0 * p.sx1;
    if constexpr (VEC) {
        alignas(16) T raw[(W - 1) * CH];
        alignas(16) T xr[CH];
#pragma unroll
        for (int i = 0; i < W - 1; ++i)
            *reinterpret_cast<uint4 *>(raw + i * CH) = reinterpret_cast<const uint4 *>(st)[i];
        *reinterpret_cast<uint4 *>(xr) = *reinterpret_cast<const uint4 *>(x);
#pragma unroll
        for (int j = 0; j < CH; ++j) {
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
                e[j][k] = raw[j * (W - 1) + k];
            e[j][W - 1] = xr[j];
        }
    } else {
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            e[0][k] = st[k];
        e[0][W - 1] = x[0];
    }
    alignas(16) T yr[CH], sr[(W - 1) * CH];
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        float v = p.bias ? p.bias[c0 + j] : 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k)
            v = fmaf(p.weight[int64_t(c0 + j) * W + k], float(e[j][k]), v);
        if (p.silu)
            v = std::is_same<T, float>::value ? silu_exact(v) : silu_fast(v);
        yr[j] = T(v);
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            sr[j * (W - 1) + k] = e[j][k + 1];
    }
    T *y = static_cast<T *>(p.y) + b * p.sy0 + c0 * p.sy1;
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < W - 1; ++i)
            reinterpret_cast<uint4 *>(st)[i] = *reinterpret_cast<uint4 *>(sr + i * CH);
        *reinterpret_cast<uint4 *>(y) = *reinterpret_cast<uint4 *>(yr);
    } else {
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            st[k] = sr[k];
        y[0] = yr[0];
    }
}

// ------------------------------------------------------ packed prompts
// Sequences of unequal length, one after the other in the rows of a
// token-major buffer: sequence i owns rows [start[i], start[i+1]) and slot
// slots[i] of the cache.  All of that is on the device, so a launch is sized
// by the rows alone and every warp looks its sequences up.
struct PackedIndex {
    int tokens, seqs, slot_count;
    const int *start;  // (seqs + 1)
    const int *slots;  // (seqs)
    const int *seen;   // (seqs) or null: tokens already in the state, 0 = start from zero
    unsigned int *err;
};

struct PackedSeq {
    int begin, end, slot;
    bool fresh;
};

// The last sequence that does not begin behind `key`, where sequence i begins
// at start[i] / div + i * mul (a non-decreasing map), by the whole warp: 32
// probes a step.
__device__ __forceinline__ int packed_find(const PackedIndex &ix, int64_t key, int div, int mul,
                                           int lane)
{
    int lo = 0, hi = ix.seqs;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int i = lo + lane * step;
        const bool le = i < hi && int64_t(ix.start[i]) / div + int64_t(i) * mul <= key;
        const unsigned m = __ballot_sync(0xffffffffu, le);
        const int k = m ? 31 - __clz(m) : 0;
        lo += k * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// Sequence s as the warp may work on it: false for padding (a negative slot)
// and for one that is refused, which sets the error word: rows outside the
// buffer, a slot past the cache's end, or a slot that an earlier sequence
// owns (two owners would race on its state).
__device__ __forceinline__ bool packed_seq(const PackedIndex &ix, int s, int lane, PackedSeq &q)
{
    q.begin = ix.start[s];
    q.end = ix.start[s + 1];
    q.slot = ix.slots[s];
    q.fresh = ix.seen && ix.seen[s] <= 0;
    if (q.slot < 0)
        return false;
    bool bad = q.begin < 0 || q.end < q.begin || q.end > ix.tokens || q.slot >= ix.slot_count;
    for (int j = lane; j < s; j += 32)
        bad |= ix.slots[j] == q.slot;
    if (__any_sync(0xffffffffu, bad)) {
        if (lane == 0)
            atomicOr(ix.err, kErrIndex);
        return false;
    }
    return true;
}

struct ConvPackedParams {
    PackedIndex ix;
    int dim, vec, runs, ctiles;
    const void *x;
    int64_t sx;  // row stride; channels are contiguous
    void *y;
    int64_t sy;
    const float *weight, *bias;
    void *state;  // (slot_count, dim, W-1) contiguous
    int silu;
};

constexpr int kConvRun = 8;  // rows of a warp

// A warp owns kConvRun rows x 32 CH channels.  The usual warp lies inside one
// sequence, W-1 rows or more behind its first: it loads its rows and the W-1
// before them and is done.  The others go token by token.  A sequence's first
// W-1 tokens, which need the old state, are all taken by the warp that holds
// its first row, which also writes the new state: no other warp touches the
// slot.  One more warp (run == runs) looks after sequences without rows.
template <typename T, int W, bool VEC>
__global__ void __launch_bounds__(128) conv_packed_kernel(const __grid_constant__ ConvPackedParams p)
{
    constexpr int CH = VEC ? 16 / int(sizeof(T)) : 2;
    const int lane = threadIdx.x & 31;
    const int64_t wid = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int ct = int(wid % p.ctiles), run = int(wid / p.ctiles);
    if (run > p.runs)
        return;
    const PackedIndex &ix = p.ix;
    const int c0 = (ct * 32 + lane) * CH;
    const bool live = c0 < p.dim;
    const T *xb = static_cast<const T *>(p.x);
    T *yb = static_cast<T *>(p.y);
    T *state = static_cast<T *>(p.state);
    const T zero = conv_zero(static_cast<const T *>(nullptr));

    if (run == p.runs) {
        for (int s0 = 0; s0 < ix.seqs; s0 += 32) {
            const int s = s0 + lane;
            bool empty = false;
            if (s < ix.seqs) {
                const int bg = ix.start[s], en = ix.start[s + 1];
                const bool owns = ix.slots[s] >= 0;
                if (owns && (bg < 0 || en < bg || en > ix.tokens))
                    atomicOr(ix.err, kErrIndex);
                empty = owns && bg == en && ix.seen && ix.seen[s] <= 0;
            }
            unsigned m = __ballot_sync(0xffffffffu, empty);
            while (m) {
                const int i = s0 + __ffs(m) - 1;
                m &= m - 1;
                PackedSeq q;
                if (!packed_seq(ix, i, lane, q) || !live)
                    continue;
                for (int j = 0; j < CH && c0 + j < p.dim; ++j)
                    for (int k = 0; k < W - 1; ++k)
                        state[(int64_t(q.slot) * p.dim + c0 + j) * (W - 1) + k] = zero;
            }
        }
        return;
    }

    const int t0 = run * kConvRun, t1 = min(t0 + kConvRun, ix.tokens);
    int s = packed_find(ix, t0, 1, 0, lane);
    PackedSeq q;
    bool ok = packed_seq(ix, s, lane, q);
    uint64_t w[CH / 2][W], bias[CH / 2];
    load_taps<W, CH>(w, bias, p.weight, p.bias, live ? c0 : p.dim, p.dim);

    if (VEC && ok && q.begin + (W - 1) <= t0 && q.end >= t1 && t1 - t0 == kConvRun) {
        if (!live)
            return;
        pair_t<T> xp[W - 1 + kConvRun][CH / 2];
#pragma unroll
        for (int i = 0; i < W - 1 + kConvRun; ++i)
            load_row<T, CH>(xb + int64_t(t0 - (W - 1) + i) * p.sx + c0, xp[i]);
#pragma unroll
        for (int i = 0; i < kConvRun; ++i) {
            pair_t<T> out[CH / 2];
#pragma unroll
            for (int r = 0; r < CH / 2; ++r) {
                uint64_t e[W];
#pragma unroll
                for (int k = 0; k < W; ++k)
                    e[k] = PairOf<T>::f2(xp[i + k][r]);
                uint64_t v = tap_sum<W>(w[r], e, bias[r]);
                if (p.silu)
                    v = silu2<T>(v);
                out[r] = PairOf<T>::round(v);
            }
            store_row<T, CH>(yb + int64_t(t0 + i) * p.sy + c0, out);
        }
        return;
    }

    for (;;) {
        if (ok && q.begin < q.end) {
            const bool mine = q.begin >= t0 && q.begin < t1;
            const int lo = mine ? q.begin : max(t0, min(q.end, q.begin + W - 1));
            const int hi = mine ? max(min(t1, q.end), min(q.end, q.begin + W - 1))
                                : min(t1, q.end);
            if (live) {
                const int64_t srow = (int64_t(q.slot) * p.dim + c0) * (W - 1);
                // element t of the sequence's input behind its past, channel c0 + j
                const auto at = [&](int t, int j) -> T {
                    if (c0 + j >= p.dim)
                        return zero;
                    if (t >= q.begin)
                        return xb[int64_t(t) * p.sx + c0 + j];
                    return q.fresh ? zero : state[srow + j * (W - 1) + W - 1 + (t - q.begin)];
                };
                for (int t = lo; t < hi; ++t) {
#pragma unroll
                    for (int r = 0; r < CH / 2; ++r) {
                        uint64_t e[W];
#pragma unroll
                        for (int k = 0; k < W; ++k)
                            e[k] = PairOf<T>::f2(PairOf<T>::make(at(t - (W - 1) + k, 2 * r),
                                                                 at(t - (W - 1) + k, 2 * r + 1)));
                        uint64_t v = tap_sum<W>(w[r], e, bias[r]);
                        if (p.silu)
                            v = silu2<T>(v);
                        const pair_t<T> o = PairOf<T>::round(v);
                        T *y = yb + int64_t(t) * p.sy + c0 + 2 * r;
                        if (c0 + 2 * r < p.dim)
                            y[0] = PairOf<T>::lo(o);
                        if (c0 + 2 * r + 1 < p.dim)
                            y[1] = PairOf<T>::hi(o);
                    }
                }
                if (mine) {
                    for (int j = 0; j < CH && c0 + j < p.dim; ++j) {
                        T tail[W - 1];
#pragma unroll
                        for (int k = 0; k < W - 1; ++k)
                            tail[k] = at(q.end - (W - 1) + k, j);
#pragma unroll
                        for (int k = 0; k < W - 1; ++k)
                            state[srow + j * (W - 1) + k] = tail[k];
                    }
                }
            }
        }
        if (++s >= ix.seqs || ix.start[s] >= t1)
            break;
        ok = packed_seq(ix, s, lane, q);
    }
}

// -------------------------------------------------------------- backward
struct ConvBwdParams {
    int batch, dim, L;
    int cg_log2;
    int ctiles, runs;   // warp tiles over channels, runs of steps over tokens
    int steps;          // warp steps (token tiles) per run
    ConvView x, dy, dx;
    const float *weight, *bias;
    const void *h0, *dlast;  // (batch, dim, W-1) or null
    void *dh0;               // (batch, dim, W-1) or null
    float *part;             // [batch * runs][dim][W + 1]: dw | db of a run
    int silu;
};

// A warp walks a run of token tiles from the last to the first.  Per tile a
// thread recomputes v of its CH channels x TB tokens, forms g, adds g e to
// the taps' gradients, and forms dx, for which it needs the first W-1 g of
// the tokens behind its own: those of the lane that holds the next token
// block (a shuffle), or, for the warp's last block, of the first block of the
// tile done before.  Above a run they are recomputed: the run's first step is
// the tile behind it, of which only those W-1 tokens are formed.
template <typename T, int W, bool XTOK, bool YTOK>
__global__ void __launch_bounds__(128) conv_bwd_kernel(const __grid_constant__ ConvBwdParams p)
{
    constexpr int CH = 4, TB = 16 / int(sizeof(T)), Q = CH / 2, H = W - 1;
    const int lane = threadIdx.x & 31;
    const int ngr = 32 >> p.cg_log2;  // token blocks of a tile
    const int cg = lane & ((1 << p.cg_log2) - 1), tg = lane >> p.cg_log2;
    const int64_t wid = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int ct = int(wid % p.ctiles), run = int(wid / p.ctiles);
    if (run >= p.runs)
        return;
    const int b = int(blockIdx.y);
    const int c0 = ((ct << p.cg_log2) + cg) * CH;
    const int tile = ngr * TB;
    const T *past = static_cast<const T *>(p.h0);
    uint64_t w[Q][W], bias[Q], dw[Q][W], db[Q];
    load_taps<W, CH>(w, bias, p.weight, p.bias, c0, p.dim);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        db[q] = 0;
#pragma unroll
        for (int k = 0; k < W; ++k)
            dw[q][k] = 0;
    }
    uint64_t head[Q][H];  // this block's first W-1 g of the tile done before
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int k = 0; k < H; ++k)
            head[q][k] = 0;

    const int64_t first = int64_t(run) * p.steps * tile;
    for (int step = p.steps; step >= 0; --step) {
        const int64_t tl = first + int64_t(step) * tile;  // the tile's first token
        if (tl >= p.L)
            continue;  // nothing there: g is zero (uniform over the warp)
        const int t0 = int(min(tl + int64_t(tg) * TB, int64_t(p.L)));
        const bool above = step == p.steps;  // the tile behind the run
        pair_t<T> xp[Q][H + TB], yp[Q][TB];
        load_block<T, XTOK, CH, TB, H>(xp, p.x, past, H, b, c0, t0, p.dim, p.L);
        load_block<T, YTOK, CH, TB, 0>(yp, p.dy, nullptr, 0, b, c0, t0, p.dim, p.L);
        uint64_t g[Q][TB + H];
#pragma unroll
        for (int q = 0; q < Q; ++q) {
#pragma unroll
            for (int i = 0; i < TB; ++i) {
                uint64_t e[W];
#pragma unroll
                for (int k = 0; k < W; ++k)
                    e[k] = PairOf<T>::f2(xp[q][i + k]);
                const uint64_t dy = PairOf<T>::f2(yp[q][i]);
                uint64_t gv = dy;
                if (p.silu) {
                    const uint64_t v = tap_sum<W>(w[q], e, bias[q]);
                    const auto slope = [](float v, float d) {
                        const float s = std::is_same<T, float>::value
                                            ? 1.f / (1.f + expf(-v))
                                            : rcp_approx(1.f + ex2_approx(-v * kLog2e));
                        return d * fmaf(v * s, 1.f - s, s);
                    };
                    gv = pk2(slope(lo2(v), lo2(dy)), slope(hi2(v), hi2(dy)));
                }
                g[q][i] = gv;
                if (!above) {
#pragma unroll
                    for (int k = 0; k < W; ++k)
                        dw[q][k] = fma2(gv, e[k], dw[q][k]);
                    db[q] = add2(db[q], gv);
                }
            }
            // the W-1 g behind this block
            const int src = ((tg + 1) & (ngr - 1)) * (32 / ngr) + cg;
#pragma unroll
            for (int k = 0; k < H; ++k) {
                const uint64_t give = tg == 0 ? head[q][k] : g[q][k];
                g[q][TB + k] = __shfl_sync(0xffffffffu, (unsigned long long)give, src);
                head[q][k] = g[q][k];
            }
        }
        if (above)
            continue;
        pair_t<T> dp[Q][TB];
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            uint64_t d[TB];
#pragma unroll
            for (int i = 0; i < TB; ++i) {
                uint64_t a = 0;
#pragma unroll
                for (int k = 0; k < W; ++k)
                    a = fma2(w[q][k], g[q][i + H - k], a);
                d[i] = a;
            }
            if (p.dlast && t0 + TB > p.L - H) {
                // the state that the sequence ends with is its last inputs
#pragma unroll
                for (int i = 0; i < TB; ++i) {
                    const int j = t0 + i - (p.L - H), c = c0 + 2 * q;
                    if (j >= 0 && j < H) {
                        const T *dl = static_cast<const T *>(p.dlast) +
                                      (int64_t(b) * p.dim + c) * H + j;
                        d[i] = add2(d[i], pk2(c < p.dim ? float(dl[0]) : 0.f,
                                              c + 1 < p.dim ? float(dl[H]) : 0.f));
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < TB; ++i)
                dp[q][i] = PairOf<T>::round(d[i]);
        }
        if (t0 < p.L)
            store_block<T, XTOK, CH, TB>(dp, p.dx, b, c0, t0, p.dim, p.L);
        if (p.dh0 && t0 == 0) {
            // element j of the initial state is input j - (W-1)
#pragma unroll
            for (int q = 0; q < Q; ++q) {
#pragma unroll
                for (int j = 0; j < H; ++j) {
                    uint64_t a = 0;
#pragma unroll
                    for (int k = 0; k <= j; ++k)
                        a = fma2(w[q][k], g[q][j - k], a);
                    const int c = c0 + 2 * q, o = j - (p.L);  // index in dlast: j - H - (L - H)
                    float f[2] = {lo2(a), hi2(a)};
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (c + h >= p.dim)
                            continue;
                        const int64_t row = (int64_t(b) * p.dim + c + h) * H;
                        if (p.dlast && o >= 0)
                            f[h] += float(static_cast<const T *>(p.dlast)[row + o]);
                        static_cast<T *>(p.dh0)[row + j] = T(f[h]);
                    }
                }
            }
        }
    }
    // the run's sums over the warp's token blocks
    for (int off = 16; off >= (1 << p.cg_log2); off >>= 1)
#pragma unroll
        for (int q = 0; q < Q; ++q) {
#pragma unroll
            for (int k = 0; k < W; ++k)
                dw[q][k] = add2(dw[q][k],
                                __shfl_xor_sync(0xffffffffu, (unsigned long long)dw[q][k], off));
            db[q] = add2(db[q], __shfl_xor_sync(0xffffffffu, (unsigned long long)db[q], off));
        }
    if (tg == 0) {
#pragma unroll
        for (int q = 0; q < Q; ++q)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int c = c0 + 2 * q + h;
                if (c >= p.dim)
                    continue;
                float *o = p.part + ((int64_t(b) * p.runs + run) * p.dim + c) * (W + 1);
#pragma unroll
                for (int k = 0; k < W; ++k)
                    o[k] = h ? hi2(dw[q][k]) : lo2(dw[q][k]);
                o[W] = h ? hi2(db[q]) : lo2(db[q]);
            }
    }
}

// dweight and dbias: the runs' sums added in a fixed order, by one warp per
// 32 (channel, tap) columns and 8 rows of runs at a time.
template <int W>
__global__ void __launch_bounds__(256) conv_bwd_sum_kernel(const float *part, int rows, int dim,
                                                           float *dweight, float *dbias)
{
    __shared__ float s[8][33];
    const int col = int(blockIdx.x) * 32 + (threadIdx.x & 31), r0 = threadIdx.x >> 5;
    const int64_t cols = int64_t(dim) * (W + 1);
    float a = 0.f;
    if (col < cols)
        for (int r = r0; r < rows; r += 8)
            a += part[r * cols + col];
    s[r0][threadIdx.x & 31] = a;
    __syncthreads();
    if (r0 == 0 && col < cols) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v += s[i][threadIdx.x & 31];
        const int c = col / (W + 1), k = col % (W + 1);
        if (k < W)
            dweight[int64_t(c) * W + k] = v;
        else if (dbias)
            dbias[c] = v;
    }
}

}  // namespace selscan
