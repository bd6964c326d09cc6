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
//
// What bounds them is HBM in the end (4 bytes per element forward, 6 backward,
// 16 per channel and row for single tokens, in bf16), and on the way to it the
// instructions per element (about 14 forward, 38 backward) and the loads in
// flight.  Measured, bf16, four taps, SiLU, whole calls on inputs that change from
// call to call: forward 4 x 5120 x 4096, token-major in, channels-first out, 77 us
// (4.4 TB/s); packed 8192 x 2560 23.6 us (3.6 TB/s); backward 8 x 2560 x 2048 84
// us (3.0 TB/s, 5 us of it the sum of the runs); single tokens 1024 x 5120 18.5 us
// (4.5 TB/s).  The figures beside choices below compare kernels on inputs that
// stay, and are up to a tenth lower.
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
    } else if constexpr (CH * sizeof(T) == 4) {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
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
    } else if constexpr (CH * sizeof(T) == 4) {
        *reinterpret_cast<uint32_t *>(p) = w[0];
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

// A block of tokens [t0 - HLO, t0 + TB) x CH channels as its vectors in
// memory: rows of CH channels (TOK), or, per channel, 16-byte pieces of time
// (with HLO, the piece before the block too).
template <typename T, bool TOK, int CH, int TB, int HLO>
struct BlockIO {
    static constexpr int VEC = 16 / int(sizeof(T));
    static constexpr int PER = TB / VEC + (HLO > 0);  // pieces of a channel
    static constexpr int N = TOK ? HLO + TB : CH * PER;
    static constexpr int BYTES = TOK ? CH * int(sizeof(T)) : 16;
    using Piece = std::conditional_t<BYTES == 16, uint4, std::conditional_t<BYTES == 8, uint2, uint32_t>>;
    static_assert(BYTES == 16 || BYTES == 8 || BYTES == 4, "pieces that one copy can move");
    static_assert(TOK || TB % VEC == 0, "whole 16-byte pieces of a time row");

    // Whether all of it is inside the tensor, in whole aligned vectors.
    static __device__ __forceinline__ bool inside(const ConvView &v, int c0, int t0, int dim, int L)
    {
        return v.vec && c0 + CH <= dim && t0 >= (HLO ? (TOK ? HLO : VEC) : 0) && t0 + TB <= L;
    }
    // f(piece's number, its address)
    template <typename F>
    static __device__ __forceinline__ void each(const ConvView &v, int b, int c0, int t0, F f)
    {
        const T *base = static_cast<const T *>(v.data) + b * v.sb;
        if (TOK) {
            const T *r = base + c0 + (t0 - HLO) * v.st;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                f(i, r);
                r += v.st;
            }
        } else {
            const T *r = base + c0 * v.sd + t0 - (HLO ? VEC : 0);
#pragma unroll
            for (int c = 0; c < CH; ++c) {
#pragma unroll
                for (int j = 0; j < PER; ++j)
                    f(c * PER + j, r + j * VEC);
                r += v.sd;
            }
        }
    }
    // One pair of channels of a time layout from its two channels' pieces, the
    // first at w[0], each `step` after the one before.
    static __device__ __forceinline__ void pair(const Piece *w, int step, pair_t<T> (&o)[HLO + TB])
    {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const uint4 x = w[j * step], y = w[(PER + j) * step];
            const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
            // the piece's first token, counted from the block's halo
            const int i0 = HLO ? HLO + (j - 1) * VEC : j * VEC;
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (i0 + i >= 0) {
                    if constexpr (sizeof(T) == 2)
                        o[i0 + i < 0 ? 0 : i0 + i] =
                            __byte_perm(xs[i / 2], ys[i / 2], i % 2 ? 0x7632 : 0x5410);
                    else
                        o[i0 + i < 0 ? 0 : i0 + i] = uint64_t(xs[i]) | (uint64_t(ys[i]) << 32);
                }
        }
    }
    // A lane's pieces in shared memory, 32 places apart: pair q of its channels
    static __device__ __forceinline__ void take(const Piece *w, int q, pair_t<T> (&o)[HLO + TB])
    {
        if constexpr (TOK) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                o[i] = reinterpret_cast<const pair_t<T> *>(w + i * 32)[q];
        } else {
            pair(w + 2 * q * PER * 32, 32, o);
        }
    }
    // and pairs into such pieces (what lies before the halo is left out)
    static __device__ __forceinline__ void give(Piece *w, const pair_t<T> (&xp)[CH / 2][HLO + TB])
    {
        if constexpr (TOK) {
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int q = 0; q < CH / 2; ++q)
                    reinterpret_cast<pair_t<T> *>(w + i * 32)[q] = xp[q][i];
        } else {
#pragma unroll
            for (int q = 0; q < CH / 2; ++q)
#pragma unroll
                for (int i = 0; i < HLO + TB; ++i) {
                    const int at = (HLO ? VEC - HLO : 0) + i;  // in the channel's pieces
                    T *lo = reinterpret_cast<T *>(w + (2 * q * PER + at / VEC) * 32) + at % VEC;
                    T *hi = reinterpret_cast<T *>(w + ((2 * q + 1) * PER + at / VEC) * 32) + at % VEC;
                    *lo = PairOf<T>::lo(xp[q][i]);
                    *hi = PairOf<T>::hi(xp[q][i]);
                }
        }
    }
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
    using IO = BlockIO<T, TOK, CH, TB, HLO>;
    if (IO::inside(v, c0, t0, dim, L)) {
        if constexpr (TOK) {
            IO::each(v, b, c0, t0, [&](int i, const T *r) {
                pair_t<T> w[CH / 2];
                load_row<T, CH>(r, w);
#pragma unroll
                for (int q = 0; q < CH / 2; ++q)
                    xp[q][i] = w[q];
            });
        } else {
            typename IO::Piece w[IO::N];
            IO::each(v, b, c0, t0, [&](int i, const T *r) {
                w[i] = *reinterpret_cast<const typename IO::Piece *>(r);
            });
#pragma unroll
            for (int q = 0; q < CH / 2; ++q)
                IO::pair(w + 2 * q * IO::PER, 1, xp[q]);
        }
        return;
    }
    const T *base = static_cast<const T *>(v.data) + b * v.sb;
    const T zero = conv_zero(static_cast<const T *>(nullptr));
    const auto at = [&](int c, int t) -> T {
        if (c >= dim || t >= L)
            return zero;
        if (t < 0)
            return past ? past[(int64_t(b) * dim + c) * past_n + past_n + t] : zero;
        return base[c * v.sd + t * v.st];
    };
    if (v.vec && c0 + CH <= dim && (TOK || t0 + TB <= L)) {
        // an end of the sequence: whole vectors inside, the rest as it comes
#pragma unroll
        for (int q = 0; q < CH / 2; ++q)
#pragma unroll
            for (int i = 0; i < HLO + (TOK ? TB : 0); ++i)
                xp[q][i] = t0 - HLO + i < 0 && past
                               ? PairOf<T>::make(at(c0 + 2 * q, t0 - HLO + i),
                                                 at(c0 + 2 * q + 1, t0 - HLO + i))
                               : pair_t<T>(0);
        if constexpr (TOK) {
#pragma unroll
            for (int i = 0; i < HLO + TB; ++i)
                if (t0 - HLO + i >= 0 && t0 - HLO + i < L) {
                    pair_t<T> w[CH / 2];
                    load_row<T, CH>(base + c0 + (t0 - HLO + i) * v.st, w);
#pragma unroll
                    for (int q = 0; q < CH / 2; ++q)
                        xp[q][i] = w[q];
                }
        } else {
            // (the block at token 0: nothing before it is in the tensor)
            using Inner = BlockIO<T, TOK, CH, TB, 0>;
            typename Inner::Piece w[Inner::N];
            Inner::each(v, b, c0, t0, [&](int i, const T *r) {
                w[i] = *reinterpret_cast<const typename Inner::Piece *>(r);
            });
#pragma unroll
            for (int q = 0; q < CH / 2; ++q) {
                pair_t<T> o[TB];
                Inner::pair(w + 2 * q * Inner::PER, 1, o);
#pragma unroll
                for (int i = 0; i < TB; ++i)
                    xp[q][HLO + i] = o[i];
            }
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

// The block back: the first TB tokens of the pairs yp[channel pair][token].
template <typename T, bool TOK, int CH, int TB, int N>
__device__ __forceinline__ void store_block(const pair_t<T> (&yp)[CH / 2][N], const ConvView &v,
                                            int b, int c0, int t0, int dim, int L)
{
    constexpr int VEC = 16 / int(sizeof(T));
    T *base = static_cast<T *>(v.data) + b * v.sb;
    if (TOK) {
        if (v.vec && c0 + CH <= dim && t0 + TB <= L) {
            T *r = base + c0 + t0 * v.st;
#pragma unroll
            for (int i = 0; i < TB; ++i) {
                pair_t<T> w[CH / 2];
#pragma unroll
                for (int q = 0; q < CH / 2; ++q)
                    w[q] = yp[q][i];
                store_row<T, CH>(r, w);
                r += v.st;
            }
            return;
        }
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

// The taps and biases of the `n` channels from c0, which a block's four warps
// share, in shared memory: rows [k][channel], biases in row W (read straight
// from the weight rows, 32 lanes would touch 32 lines for every element).  The
// caller synchronises the block.
template <int W, int CT>
struct ConvTaps {
    static constexpr int kPitch = CT + 8;  // a warp's writes fall into different banks
    float v[W + 1][kPitch];
    __device__ __forceinline__ void stage(const float *weight, const float *bias, int c0, int n,
                                          int dim)
    {
        const int have = min(n, dim - c0) * W;
        const float *src = weight + int64_t(c0) * W;
        const bool vec = (reinterpret_cast<uintptr_t>(src) & 15) == 0;
        // 16-byte pieces, all of a thread's in flight at once
        constexpr int PIECES = (CT * W / 4 + 127) / 128;
        float f[PIECES][4];
#pragma unroll
        for (int m = 0; m < PIECES; ++m) {
            const int i = 4 * (m * 128 + int(threadIdx.x));
            if (vec && i + 4 <= have) {
                const float4 x = *reinterpret_cast<const float4 *>(src + i);
                f[m][0] = x.x;
                f[m][1] = x.y;
                f[m][2] = x.z;
                f[m][3] = x.w;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    f[m][j] = i + j < have ? src[i + j] : 0.f;
            }
        }
        for (int i = threadIdx.x; i < n; i += 128)
            v[W][i] = bias && c0 + i < dim ? bias[c0 + i] : 0.f;
#pragma unroll
        for (int m = 0; m < PIECES; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = 4 * (m * 128 + int(threadIdx.x)) + j;
                if (i < n * W)
                    v[i % W][i / W] = f[m][j];
            }
    }
    // taps and bias of the pair of channels from the block's channel o (even)
    __device__ __forceinline__ void read(uint64_t (&w)[W], uint64_t &b, int o) const
    {
#pragma unroll
        for (int k = 0; k < W; ++k) {
            const float2 f = *reinterpret_cast<const float2 *>(&v[k][o]);
            w[k] = pk2(f.x, f.y);
        }
        const float2 f = *reinterpret_cast<const float2 *>(&v[W][o]);
        b = pk2(f.x, f.y);
    }
};

// v sigmoid(v): the special-function unit for bf16 results (its error, about
// 2^-21, is far below their rounding), the accurate functions for fp32.
template <typename T>
__device__ __forceinline__ uint64_t silu2(uint64_t v)
{
    if constexpr (std::is_same<T, float>::value)
        return pk2(silu_exact(lo2(v)), silu_exact(hi2(v)));
    const uint64_t m = mul2(v, pk2(-kLog2e, -kLog2e));
    const uint64_t d = add2(pk2(ex2_approx(lo2(m)), ex2_approx(hi2(m))), pk2(1.f, 1.f));
    return mul2(v, pk2(rcp_approx(lo2(d)), rcp_approx(hi2(d))));
}

// dy times the slope of v sigmoid(v): sg + v sg (1 - sg).
template <typename T>
__device__ __forceinline__ uint64_t silu_grad2(uint64_t v, uint64_t dy)
{
    uint64_t s;
    if constexpr (std::is_same<T, float>::value) {
        s = pk2(1.f / (1.f + expf(-lo2(v))), 1.f / (1.f + expf(-hi2(v))));
    } else {
        const uint64_t m = mul2(v, pk2(-kLog2e, -kLog2e));
        const uint64_t d = add2(pk2(ex2_approx(lo2(m)), ex2_approx(hi2(m))), pk2(1.f, 1.f));
        s = pk2(rcp_approx(lo2(d)), rcp_approx(hi2(d)));
    }
    const uint64_t rest = fma2(s, pk2(-1.f, -1.f), pk2(1.f, 1.f));
    return mul2(dy, fma2(mul2(v, s), rest, s));
}

// f(true_type) or f(false_type): a uniform flag tested once instead of at
// every value.
template <typename F>
__device__ __forceinline__ void with_flag(bool flag, F f)
{
    if (flag)
        f(std::true_type());
    else
        f(std::false_type());
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
// that a tile reads from the tile before it come from L1.  Five blocks per SM:
// 72 us for 4 x 5120 x 4096 bf16 (four 77, six, with 80 registers, 86).
template <typename T, int W, bool XTOK, bool YTOK>
__global__ void __launch_bounds__(128, 5) conv_fwd_kernel(const __grid_constant__ ConvParams p)
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
    const int cb = (ct << p.cg_log2) * CH, c0 = cb + cg * CH;
    const int64_t tl = (int64_t(tt) * (32 >> p.cg_log2) + tg) * TB;
    const bool live = c0 < p.dim && tl < p.L;
    const int t0 = live ? int(tl) : 0;
    const T *past = static_cast<const T *>(p.h0);
    __shared__ __align__(16) ConvTaps<W, 32 * CH> taps;
    pair_t<T> xp[CH / 2][W - 1 + TB];
    if (live)
        load_block<T, XTOK, CH, TB, W - 1>(xp, p.x, past, W - 1, b, c0, t0, p.dim, p.L);
    taps.stage(p.weight, p.bias, cb, CH << p.cg_log2, p.dim);
    __syncthreads();
    if (!live)
        return;
    with_flag(p.silu, [&](auto silu) {
#pragma unroll
        for (int q = 0; q < CH / 2; ++q) {
            uint64_t w[W], bias, e[W];
            taps.read(w, bias, cg * CH + 2 * q);
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
                e[k + 1] = PairOf<T>::f2(xp[q][k]);
#pragma unroll
            for (int i = 0; i < TB; ++i) {
#pragma unroll
                for (int k = 0; k < W - 1; ++k)
                    e[k] = e[k + 1];
                e[W - 1] = PairOf<T>::f2(xp[q][W - 1 + i]);
                uint64_t v = tap_sum<W>(w, e, bias);
                if (decltype(silu)::value)
                    v = silu2<T>(v);
                xp[q][i] = PairOf<T>::round(v);  // in place of an input that is done with
            }
        }
    });
    store_block<T, YTOK, CH, TB>(xp, p.y, b, c0, t0, p.dim, p.L);
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
    int wvec;  // the taps may be read as 16-byte pieces
    int rows;  // of a block
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
// thread owns CH channels, whose (W-1) CH state elements are W-1 whole 16-byte
// vectors (VEC), or one channel (any strides, any dim); its taps serve all of
// a block's rows.  A warp's state of a row is one contiguous piece: it comes
// and goes through shared memory in whole lines (the threads' own vectors lie
// W-1 vectors apart, and stores of 16 bytes out of every 48 cost the L2 twice
// the sectors: 23.6 us, now 18.0, for 1024 rows of 5120), kStepDepth rows on
// their way at a time.  Slots as in the scan's decode step: negative is
// padding, a slot past the end or owned by an earlier row is refused.
constexpr int kConvStepRows = 16;  // most rows of a block
constexpr int kStepDepth = 4;

template <typename T, int W, bool VEC>
__global__ void __launch_bounds__(128) conv_step_kernel(const __grid_constant__ ConvStepParams p)
{
    constexpr int CH = VEC ? 16 / int(sizeof(T)) : 1, NV = W - 1;
    __shared__ int row_s[kConvStepRows];  // the row's place in the cache, or -1
    // [warp][row][the state's vectors, then x's]
    __shared__ uint4 ring[4][VEC ? kStepDepth : 1][VEC ? 32 * (NV + 1) : 1];
    const int tid = threadIdx.x, lane = tid & 31;
    const int c0 = (int(blockIdx.x) * 128 + tid) * CH;
    const bool live = c0 < p.dim;
    const int b0 = int(blockIdx.y) * p.rows, nb = min(p.rows, p.batch - b0);
    if (tid < nb) {
        int slot = p.slots ? p.slots[b0 + tid] : b0 + tid;
        if (slot >= p.slot_count) {
            atomicOr(p.err, kErrIndex);
            slot = -1;
        }
        row_s[tid] = slot;
    }
    // taps [channel][k], as they lie in memory
    float w[CH * W], bias[CH];
    if (live) {
        const float *wr = p.weight + int64_t(c0) * W;
        if (VEC && p.wvec) {
#pragma unroll
            for (int i = 0; i < CH * W / 4; ++i) {
                const float4 f = reinterpret_cast<const float4 *>(wr)[i];
                w[4 * i] = f.x;
                w[4 * i + 1] = f.y;
                w[4 * i + 2] = f.z;
                w[4 * i + 3] = f.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < CH * W; ++i)
                w[i] = wr[i];
        }
#pragma unroll
        for (int j = 0; j < CH; ++j)
            bias[j] = p.bias ? p.bias[c0 + j] : 0.f;
    }
    __syncthreads();

    const T *x = static_cast<const T *>(p.x) + c0 * p.sx1;
    T *y = static_cast<T *>(p.y) + c0 * p.sy1;
    // the warp's piece of a state row, and how many vectors of it there are
    const int cw = (int(blockIdx.x) * 128 + (tid & ~31)) * CH;
    const int vecs = VEC ? max(0, min(32, (p.dim - cw) / CH)) * NV : 0;
    T *state = static_cast<T *>(p.state) + int64_t(VEC ? cw : c0) * NV;
    uint4(*mine)[VEC ? 32 * (NV + 1) : 1] = ring[tid >> 5];
    const auto fetch = [&](int i) {
        const int row = i < nb ? row_s[i] : -1;
        if (VEC && row >= 0) {
            const uint4 *src = reinterpret_cast<const uint4 *>(state + int64_t(row) * p.dim * NV);
            uint4 *dst = mine[i % kStepDepth];
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (k * 32 + lane < vecs)
                    cp_async16(dst + k * 32 + lane, src + k * 32 + lane, 16);
            if (live)
                cp_async16(dst + NV * 32 + lane, x + (b0 + i) * p.sx0, 16);
        }
        cp_async_commit();
    };
    if (VEC)
#pragma unroll
        for (int i = 0; i < kStepDepth - 1; ++i)
            fetch(i);

    if (p.slots) {
        // earlier rows with one of this block's slots, eight loads at a time
        unsigned bad = 0;
        for (int j0 = tid; j0 < b0 + nb - 1; j0 += 8 * 128) {
            int other[8];
#pragma unroll
            for (int m = 0; m < 8; ++m)
                other[m] = j0 + m * 128 < b0 + nb - 1 ? p.slots[j0 + m * 128] : -1;
            for (int i = 0; i < nb; ++i) {
                const int own = row_s[i];
#pragma unroll
                for (int m = 0; m < 8; ++m)
                    if (other[m] >= 0 && other[m] == own && j0 + m * 128 < b0 + i)
                        bad |= 1u << i;
            }
        }
        __syncthreads();
        for (int i = 0; bad && i < nb; ++i)
            if (bad >> i & 1) {
                row_s[i] = -1;
                atomicOr(p.err, kErrIndex);
            }
        __syncthreads();
    }
    // one channel: state and input in, output and state out
    const auto channel = [&](const T(&e)[W], int j, T(&next)[NV]) -> T {
        float v = bias[j];
#pragma unroll
        for (int k = 0; k < W; ++k)
            v = fmaf(w[j * W + k], float(e[k]), v);
        if (p.silu)
            v = std::is_same<T, float>::value ? silu_exact(v) : silu_fast(v);
#pragma unroll
        for (int k = 0; k < NV; ++k)
            next[k] = e[k + 1];
        return T(v);
    };
    if constexpr (!VEC) {
        for (int i = 0; i < nb && live; ++i) {
            if (row_s[i] < 0)
                continue;
            T *st = state + int64_t(row_s[i]) * p.dim * NV;
            T e[W], next[NV];
#pragma unroll
            for (int k = 0; k < NV; ++k)
                e[k] = st[k];
            e[NV] = x[(b0 + i) * p.sx0];
            y[(b0 + i) * p.sy0] = channel(e, 0, next);
#pragma unroll
            for (int k = 0; k < NV; ++k)
                st[k] = next[k];
        }
    } else {
        for (int i = 0; i < nb; ++i) {
            fetch(i + kStepDepth - 1);
            cp_async_wait<kStepDepth - 1>();
            __syncwarp();
            const int row = row_s[i];
            if (row < 0)
                continue;  // the same for the whole block
            uint4 *buf = mine[i % kStepDepth];
            alignas(16) T raw[NV * CH], xr[CH], yr[CH];
#pragma unroll
            for (int k = 0; k < NV; ++k)
                *reinterpret_cast<uint4 *>(raw + k * CH) = buf[lane * NV + k];
            *reinterpret_cast<uint4 *>(xr) = buf[NV * 32 + lane];
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                T e[W], next[NV];
#pragma unroll
                for (int k = 0; k < NV; ++k)
                    e[k] = raw[j * NV + k];
                e[NV] = xr[j];
                yr[j] = channel(e, j, next);
#pragma unroll
                for (int k = 0; k < NV; ++k)
                    raw[j * NV + k] = next[k];
            }
            if (live)
                *reinterpret_cast<uint4 *>(y + (b0 + i) * p.sy0) = *reinterpret_cast<uint4 *>(yr);
#pragma unroll
            for (int k = 0; k < NV; ++k)
                buf[lane * NV + k] = *reinterpret_cast<uint4 *>(raw + k * CH);
            __syncwarp();
            uint4 *dst = reinterpret_cast<uint4 *>(state + int64_t(row) * p.dim * NV);
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (k * 32 + lane < vecs)
                    dst[k * 32 + lane] = buf[k * 32 + lane];
            __syncwarp();  // before the next row comes into this place
        }
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

    // Whether sequence s (rows [bg, en)) is to be reported: its rows are not in
    // the buffer, or, be it padding or not, the next sequence begins before it:
    // the search for a row's sequence may then miss others.
    __device__ __forceinline__ bool disorder(int s, int bg, int en, bool owns) const
    {
        return (owns && (bg < 0 || en < bg || en > tokens)) || (s + 1 < seqs && en < bg);
    }
};

struct PackedSeq {
    int begin, end, slot;
    bool fresh;
};

// A warp's view of the sequences.  Up to 32 of them are held one per lane, all
// their numbers loaded at once, so that finding and checking one costs no
// further trip to memory; more are searched 32 probes a step.
struct PackedView {
    const PackedIndex &ix;
    int lane;
    int begin_, end_, slot_, seen_;  // of sequence `lane` (few sequences)

    __device__ __forceinline__ PackedView(const PackedIndex &i, int l) : ix(i), lane(l)
    {
        if (lane < ix.seqs && ix.seqs <= 32) {
            begin_ = ix.start[lane];
            end_ = ix.start[lane + 1];
            slot_ = ix.slots[lane];
            seen_ = ix.seen ? ix.seen[lane] : 1;
        } else {
            begin_ = end_ = seen_ = 0;
            slot_ = -1;
        }
    }

    // The last sequence that does not begin behind `key`, where sequence i
    // begins at start[i] / div + i * mul (a non-decreasing map); 0 if all do.
    __device__ __forceinline__ int find(int64_t key, int div, int mul) const
    {
        if (ix.seqs <= 32) {
            const bool le = lane < ix.seqs && int64_t(begin_) / div + int64_t(lane) * mul <= key;
            const unsigned m = __ballot_sync(0xffffffffu, le);
            return m ? 31 - __clz(m) : 0;
        }
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

    // Where sequence s begins.
    __device__ __forceinline__ int begin(int s) const
    {
        return ix.seqs <= 32 ? __shfl_sync(0xffffffffu, begin_, s & 31) : ix.start[s];
    }

    // Sequence s as the warp may work on it: false for padding (a negative
    // slot) and for one that is refused, which sets the error word: rows
    // outside the buffer, a slot past the cache's end, or a slot that an
    // earlier sequence owns (two owners would race on its state).
    __device__ __forceinline__ bool get(int s, PackedSeq &q) const
    {
        bool bad = false;
        if (ix.seqs <= 32) {
            q.begin = __shfl_sync(0xffffffffu, begin_, s);
            q.end = __shfl_sync(0xffffffffu, end_, s);
            q.slot = __shfl_sync(0xffffffffu, slot_, s);
            q.fresh = __shfl_sync(0xffffffffu, seen_, s) <= 0;
            bad = lane < s && slot_ == q.slot;
        } else {
            q.begin = ix.start[s];
            q.end = ix.start[s + 1];
            q.slot = ix.slots[s];
            q.fresh = ix.seen && ix.seen[s] <= 0;
#pragma unroll 4
            for (int j = lane; j < s; j += 32)
                bad |= ix.slots[j] == q.slot;
        }
        if (q.slot < 0)
            return false;
        bad |= q.begin < 0 || q.end < q.begin || q.end > ix.tokens || q.slot >= ix.slot_count;
        if (__any_sync(0xffffffffu, bad)) {
            if (lane == 0)
                atomicOr(ix.err, kErrIndex);
            return false;
        }
        return true;
    }
};

struct ConvPackedParams {
    PackedIndex ix;
    int dim, vec, runs, ctiles;
    int subs;  // kConvRun rows at a time, this many times a run
    int svec;  // the state may be read and written as 16-byte pieces
    const void *x;
    int64_t sx;  // row stride; channels are contiguous
    void *y;
    int64_t sy;
    const float *weight, *bias;
    void *state;  // (slot_count, dim, W-1) contiguous
    int silu;
};

constexpr int kConvRun = 8;   // rows that a warp holds at once
constexpr int kConvSubs = 8;  // most of those in a row (64 rows: one mask)

// A warp owns p.subs times kConvRun rows x 32 CH channels; a block's four
// warps take neighbouring runs of the same channels.  The first kConvRun rows
// and the W-1 before them are loaded before the warp knows whose they are;
// then it walks the sequences in its rows, and each next kConvRun rows are on
// their way while the last are computed.  A sequence's first W-1 tokens, which
// need the old state, are all taken by the warp that holds its first row
// (packed_head), which also writes the new state: no other warp touches the
// slot.  The other tokens are computed from the loaded rows, under a mask.
// One more warp (run == runs) looks after sequences without rows.
//
// packed_head: sequence q's first W-1 tokens and its new state, of CH channels
// from c0.  state: the slot's row, whose (W-1) CH elements of these channels
// are W-1 whole vectors where svec says so.
template <typename T, int W, bool VEC, int CH>
__device__ __forceinline__ void packed_head(const PackedSeq &q, int c0, int dim, const T *xb,
                                            int64_t sx, T *yb, int64_t sy, T *state, bool svec,
                                            const ConvTaps<W, 32 * CH> &taps, int o, int silu)
{
    constexpr int H = W - 1;
    const T zero = conv_zero(static_cast<const T *>(nullptr));
    alignas(16) T old[CH * H], first[H][CH], tail[H][CH], out[CH * H];
    const int chans = min(CH, dim - c0);
    const auto row = [&](int t, T(&v)[CH]) {
        if (VEC) {
            *reinterpret_cast<uint4 *>(v) = *reinterpret_cast<const uint4 *>(xb + int64_t(t) * sx + c0);
        } else {
#pragma unroll
            for (int j = 0; j < CH; ++j)
                v[j] = j < chans ? xb[int64_t(t) * sx + c0 + j] : zero;
        }
    };
#pragma unroll
    for (int k = 0; k < H; ++k) {
        if (svec && !q.fresh) {
            *reinterpret_cast<uint4 *>(old + k * (16 / int(sizeof(T)))) =
                reinterpret_cast<const uint4 *>(state)[k];
        } else {
#pragma unroll
            for (int j = 0; j < CH; ++j)
                old[j * H + k] = q.fresh || j >= chans ? zero : state[j * H + k];
        }
        if (q.begin + k < q.end)
            row(q.begin + k, first[k]);
        if (q.end - H + k >= q.begin)
            row(q.end - H + k, tail[k]);
    }
#pragma unroll
    for (int i = 0; i < H; ++i) {
        if (q.begin + i >= q.end)
            break;
        T yv[CH];
#pragma unroll
        for (int r = 0; r < CH / 2; ++r) {
            uint64_t w[W], bias, e[W];
            taps.read(w, bias, o + 2 * r);
#pragma unroll
            for (int k = 0; k < W; ++k) {
                const int pos = i - H + k;  // place in the sequence
                e[k] = pos >= 0 ? pk2(float(first[pos >= 0 ? pos : 0][2 * r]),
                                      float(first[pos >= 0 ? pos : 0][2 * r + 1]))
                                : pk2(float(old[2 * r * H + (pos < 0 ? H + pos : 0)]),
                                      float(old[(2 * r + 1) * H + (pos < 0 ? H + pos : 0)]));
            }
            uint64_t v = tap_sum<W>(w, e, bias);
            if (silu)
                v = silu2<T>(v);
            const pair_t<T> o = PairOf<T>::round(v);
            yv[2 * r] = PairOf<T>::lo(o);
            yv[2 * r + 1] = PairOf<T>::hi(o);
        }
        T *y = yb + int64_t(q.begin + i) * sy + c0;
        if (VEC) {
            *reinterpret_cast<uint4 *>(y) = *reinterpret_cast<uint4 *>(yv);
        } else {
#pragma unroll
            for (int j = 0; j < CH; ++j)
                if (j < chans)
                    y[j] = yv[j];
        }
    }
    const int len = q.end - q.begin;
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int k = 0; k < H; ++k) {
            // input len - H + k, one of the old state's where that is negative
            T v = tail[k][j];
#pragma unroll
            for (int l = 1; l < H; ++l)
                if (len == l && k + l < H)
                    v = old[j * H + (k + l < H ? k + l : 0)];
            out[j * H + k] = v;
        }
#pragma unroll
    for (int k = 0; k < H; ++k) {
        if (svec) {
            reinterpret_cast<uint4 *>(state)[k] =
                *reinterpret_cast<uint4 *>(out + k * (16 / int(sizeof(T))));
        } else {
#pragma unroll
            for (int j = 0; j < CH; ++j)
                if (j < chans)
                    state[j * H + k] = out[j * H + k];
        }
    }
}

template <typename T, int W, bool VEC>
__global__ void __launch_bounds__(128, 3) conv_packed_kernel(const __grid_constant__ ConvPackedParams p)
{
    constexpr int CH = VEC ? 16 / int(sizeof(T)) : 4, H = W - 1;
    __shared__ __align__(16) ConvTaps<W, 32 * CH> taps;
    const int lane = threadIdx.x & 31;
    const int ct = int(blockIdx.x % unsigned(p.ctiles));
    const int64_t run64 = int64_t(blockIdx.x / unsigned(p.ctiles)) * 4 + (threadIdx.x >> 5);
    const int run = int(min(run64, int64_t(p.runs) + 1));
    const PackedIndex &ix = p.ix;
    const int c0 = (ct * 32 + lane) * CH;
    const bool live = c0 < p.dim;
    const T *xb = static_cast<const T *>(p.x);
    T *yb = static_cast<T *>(p.y);
    T *state = static_cast<T *>(p.state);
    const T zero = conv_zero(static_cast<const T *>(nullptr));

    const int rows = p.subs * kConvRun;
    const int t0 = int(min(int64_t(run) * rows, int64_t(ix.tokens)));
    const int t1 = int(min(int64_t(t0) + rows, int64_t(ix.tokens)));
    const auto fetch = [&](int t, pair_t<T>(&v)[CH / 2]) {
        if (!live || t < 0 || t >= t1) {
#pragma unroll
            for (int r = 0; r < CH / 2; ++r)
                v[r] = 0;
        } else if (VEC) {
            load_row<T, CH>(xb + int64_t(t) * p.sx + c0, v);
        } else {
            const T *x = xb + int64_t(t) * p.sx + c0;
#pragma unroll
            for (int r = 0; r < CH / 2; ++r)
                v[r] = PairOf<T>::make(c0 + 2 * r < p.dim ? x[2 * r] : zero,
                                       c0 + 2 * r + 1 < p.dim ? x[2 * r + 1] : zero);
        }
    };
    pair_t<T> xp[H + kConvRun][CH / 2];
    if (VEC && live && run < p.runs && t0 >= H && t0 + kConvRun <= t1) {
        const T *x = xb + int64_t(t0 - H) * p.sx + c0;
#pragma unroll
        for (int i = 0; i < H + kConvRun; ++i) {
            load_row<T, CH>(x, xp[i]);
            x += p.sx;
        }
    } else if (run < p.runs) {
#pragma unroll
        for (int i = 0; i < H + kConvRun; ++i)
            fetch(t0 - H + i, xp[i]);
    }
    const PackedView view(ix, lane);
    taps.stage(p.weight, p.bias, ct * 32 * CH, 32 * CH, p.dim);
    __syncthreads();
    if (run > p.runs)
        return;

    if (run == p.runs) {
        for (int s0 = 0; s0 < ix.seqs; s0 += 32) {
            const int s = s0 + lane;
            bool empty = false;
            if (s < ix.seqs) {
                const int bg = ix.start[s], en = ix.start[s + 1];
                const bool owns = ix.slots[s] >= 0;
                if (ix.disorder(s, bg, en, owns))
                    atomicOr(ix.err, kErrIndex);
                empty = owns && bg == en && ix.seen && ix.seen[s] <= 0;
            }
            unsigned m = __ballot_sync(0xffffffffu, empty);
            while (m) {
                const int i = s0 + __ffs(m) - 1;
                m &= m - 1;
                PackedSeq q;
                if (!view.get(i, q) || !live)
                    continue;
                for (int j = 0; j < CH && c0 + j < p.dim; ++j)
                    for (int k = 0; k < H; ++k)
                        state[(int64_t(q.slot) * p.dim + c0 + j) * H + k] = zero;
            }
        }
        return;
    }

    // the sequences in this run: which rows are behind a head, and whether any
    // sequence begins here
    uint64_t mask = 0;
    bool heads = false;
    const int s0 = view.find(t0, 1, 0);
    for (int s = s0; s < ix.seqs && view.begin(s) < t1; ++s) {
        PackedSeq q;
        if (!view.get(s, q) || q.begin >= q.end)
            continue;
        const int lo = max(t0, min(q.end, q.begin + H)) - t0, hi = min(t1, q.end) - t0;
        if (lo < hi)  // bits lo .. hi - 1
            mask |= (~uint64_t(0) >> (64 - (hi - lo))) << lo;
        heads |= q.begin >= t0;
    }
    for (int sub = t0; sub < t1 && live; sub += kConvRun) {
        pair_t<T> nx[kConvRun][CH / 2];
        if (VEC && sub + 2 * kConvRun <= t1) {
            const T *x = xb + int64_t(sub + kConvRun) * p.sx + c0;
#pragma unroll
            for (int i = 0; i < kConvRun; ++i) {
                load_row<T, CH>(x, nx[i]);
                x += p.sx;
            }
        } else if (sub + kConvRun < t1) {
#pragma unroll
            for (int i = 0; i < kConvRun; ++i)
                fetch(sub + kConvRun + i, nx[i]);
        }
        // pair by pair of channels; the outputs take the places of the inputs
        with_flag(p.silu, [&](auto silu) {
#pragma unroll
            for (int r = 0; r < CH / 2; ++r) {
                uint64_t w[W], bias, e[W];
                taps.read(w, bias, lane * CH + 2 * r);
#pragma unroll
                for (int k = 0; k < H; ++k)
                    e[k + 1] = PairOf<T>::f2(xp[k][r]);
#pragma unroll
                for (int i = 0; i < kConvRun; ++i) {
#pragma unroll
                    for (int k = 0; k < H; ++k)
                        e[k] = e[k + 1];
                    e[H] = PairOf<T>::f2(xp[H + i][r]);
                    uint64_t v = tap_sum<W>(w, e, bias);
                    if (decltype(silu)::value)
                        v = silu2<T>(v);
                    xp[i][r] = PairOf<T>::round(v);
                }
            }
        });
        const unsigned some = unsigned(mask) & 255u;
        mask >>= kConvRun;
        T *y = yb + int64_t(sub) * p.sy + c0;
        if (VEC && some == 255u) {
#pragma unroll
            for (int i = 0; i < kConvRun; ++i) {
                store_row<T, CH>(y, xp[i]);
                y += p.sy;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kConvRun; ++i) {
                if (some >> i & 1) {
                    if (VEC) {
                        store_row<T, CH>(y, xp[i]);
                    } else {
#pragma unroll
                        for (int r = 0; r < CH / 2; ++r) {
                            if (c0 + 2 * r < p.dim)
                                y[2 * r] = PairOf<T>::lo(xp[i][r]);
                            if (c0 + 2 * r + 1 < p.dim)
                                y[2 * r + 1] = PairOf<T>::hi(xp[i][r]);
                        }
                    }
                }
                y += p.sy;
            }
        }
        // the last W-1 rows go in front of the next
#pragma unroll
        for (int r = 0; r < CH / 2; ++r) {
#pragma unroll
            for (int i = 0; i < H; ++i)
                xp[i][r] = xp[kConvRun + i][r];
#pragma unroll
            for (int i = 0; i < kConvRun; ++i)
                xp[H + i][r] = nx[i][r];
        }
    }
    if (!heads)
        return;
    for (int s = s0; s < ix.seqs && view.begin(s) < t1; ++s) {
        PackedSeq q;
        if (view.get(s, q) && q.begin < q.end && q.begin >= t0 && live)
            packed_head<T, W, VEC, CH>(q, c0, p.dim, xb, p.sx, yb, p.sy,
                                       state + (int64_t(q.slot) * p.dim + c0) * H, p.svec, taps,
                                       lane * CH, p.silu);
    }
}

// -------------------------------------------------------------- backward
struct ConvBwdParams {
    int batch, dim, L;
    int cg_log2;
    int ctiles, runs;   // warp tiles over channels, runs of steps over tokens
    int across;         // a block's warps: over channels (else over runs)
    int steps;          // warp steps (token tiles) per run
    ConvView x, dy, dx;
    const float *weight, *bias;
    const void *h0, *dlast;  // (batch, dim, W-1) or null
    void *dh0;               // (batch, dim, W-1) or null
    float *part;             // [batch * runs][dim][W + 1]: dw | db of a run
    int silu;
};

// A lane's pieces of a tile that is not all inside whole vectors: an end of the
// sequence, odd channels, unaligned rows (zeros behind the end).
template <typename T, bool TOK, int CH, int TB, int HLO>
__device__ __forceinline__ void stage_edge(typename BlockIO<T, TOK, CH, TB, HLO>::Piece *w,
                                        const ConvView &v, const T *past, int b, int c0, int t0,
                                        int dim, int L)
{
    pair_t<T> xp[CH / 2][HLO + TB];
    load_block<T, TOK, CH, TB, HLO>(xp, v, past, HLO, b, c0, t0, dim, L);
    BlockIO<T, TOK, CH, TB, HLO>::give(w, xp);
}

// Channels of a thread: with two, 96 registers keep 20 warps on an SM (four
// channels: 168 and 12 warps, 87 us instead of 79 for 8 x 2560 x 2048 bf16).
constexpr int kConvBwdCh = 2;

// A warp walks a run of token tiles from the last to the first.  Per tile a
// thread recomputes v of its CH channels x TB tokens, forms g, adds g e to
// the taps' gradients, and forms dx, for which it needs the first W-1 g of
// the tokens behind its own: those of the lane that holds the next token
// block (a shuffle), or, for the warp's last block, of the first block of the
// tile done before.  Those behind the run are recomputed first.  The next
// tile's vectors are on their way into shared memory, each lane's into places
// of its own, while a tile is computed.
template <typename T, int W, bool XTOK, bool YTOK>
__global__ void __launch_bounds__(128, 5) conv_bwd_kernel(const __grid_constant__ ConvBwdParams p)
{
    constexpr int CH = kConvBwdCh, TB = 16 / int(sizeof(T)), Q = CH / 2, H = W - 1;
    using XIO = BlockIO<T, XTOK, CH, TB, H>;
    using YIO = BlockIO<T, YTOK, CH, TB, 0>;
    constexpr int NS = 2;  // tiles staged: this one and the next
    static_assert((XIO::N * XIO::BYTES + YIO::N * YIO::BYTES) * 32 * 4 * NS +
                          int(sizeof(ConvTaps<W, 64 * CH>)) <= 48 * 1024,
                  "both tiles of four warps beside the taps in static shared memory");
    __shared__ __align__(16) ConvTaps<W, 64 * CH> taps;
    __shared__ typename XIO::Piece xring[4][NS][XIO::N][32];
    __shared__ typename YIO::Piece yring[4][NS][YIO::N][32];
    const int lane = threadIdx.x & 31;
    const int ngr = 32 >> p.cg_log2;  // token blocks of a tile
    const int cg = lane & ((1 << p.cg_log2) - 1), tg = lane >> p.cg_log2;
    // a block's warps take neighbouring channels of one run or, where one warp
    // takes as many channels as the taps' place holds, neighbouring runs
    const int wp = int(threadIdx.x >> 5);
    const int ctb = p.across ? (p.ctiles + 3) / 4 : p.ctiles;
    const int ct = int(blockIdx.x % unsigned(ctb)) * (p.across ? 4 : 1) + (p.across ? wp : 0);
    const int run = int(blockIdx.x / unsigned(ctb)) * (p.across ? 1 : 4) + (p.across ? 0 : wp);
    const int b = int(blockIdx.y);
    const int cb = (int(blockIdx.x % unsigned(ctb)) * (p.across ? 4 : 1) << p.cg_log2) * CH;
    const int co = ((p.across ? wp << p.cg_log2 : 0) + cg) * CH, c0 = cb + co;
    const int tile = ngr * TB;
    const T *past = static_cast<const T *>(p.h0);
    taps.stage(p.weight, p.bias, cb, (CH << p.cg_log2) * (p.across ? 4 : 1), p.dim);
    __syncthreads();
    if (run >= p.runs || ct >= p.ctiles)
        return;
    uint64_t dw[Q][W], db[Q];
    uint64_t head[Q][H];  // this block's first W-1 g of the tile done before
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        db[q] = 0;
#pragma unroll
        for (int k = 0; k < W; ++k)
            dw[q][k] = 0;
#pragma unroll
        for (int k = 0; k < H; ++k)
            head[q][k] = 0;
    }

    const int64_t first = int64_t(run) * p.steps * tile;
    // this lane's first token of a tile
    const auto start = [&](int step) {
        return int(min(first + int64_t(step) * tile + int64_t(tg) * TB, int64_t(p.L)));
    };
    const auto fetch = [&](int step) {
        if (step < 0)
            return;
        const int t0 = start(step);
        typename XIO::Piece *xr = &xring[wp][step % NS][0][lane];
        typename YIO::Piece *yr = &yring[wp][step % NS][0][lane];
        if (XIO::inside(p.x, c0, t0, p.dim, p.L) && YIO::inside(p.dy, c0, t0, p.dim, p.L)) {
            XIO::each(p.x, b, c0, t0,
                      [&](int i, const T *r) { cp_async_ca<XIO::BYTES>(xr + i * 32, r); });
            YIO::each(p.dy, b, c0, t0,
                      [&](int i, const T *r) { cp_async_ca<YIO::BYTES>(yr + i * 32, r); });
        } else {
            stage_edge<T, XTOK, CH, TB, H>(xr, p.x, past, b, c0, t0, p.dim, p.L);
            stage_edge<T, YTOK, CH, TB, 0>(yr, p.dy, nullptr, b, c0, t0, p.dim, p.L);
        }
    };
    const bool above = first + int64_t(p.steps) * tile < p.L;
    if (above && tg == 0)
        fetch(p.steps);  // the block behind the run
    cp_async_commit();
    fetch(p.steps - 1);
    cp_async_commit();
    if (above) {
        // the first W-1 g behind the run
        cp_async_wait<1>();
        if (tg == 0) {
            const typename XIO::Piece *xr = &xring[wp][p.steps % NS][0][lane];
            const typename YIO::Piece *yr = &yring[wp][p.steps % NS][0][lane];
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                uint64_t w[W], bias;
                taps.read(w, bias, co + 2 * q);
                pair_t<T> xq[H + TB], yq[TB];
                XIO::take(xr, q, xq);
                YIO::take(yr, q, yq);
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    uint64_t e[W];
#pragma unroll
                    for (int k = 0; k < W; ++k)
                        e[k] = PairOf<T>::f2(xq[i + k]);
                    head[q][i] = PairOf<T>::f2(yq[i]);
                    if (p.silu)
                        head[q][i] = silu_grad2<T>(tap_sum<W>(w, e, bias), head[q][i]);
                }
            }
        }
    }
    for (int step = p.steps - 1; step >= 0; --step) {
        fetch(step - 1);
        cp_async_commit();
        const int64_t tl = first + int64_t(step) * tile;  // the tile's first token
        cp_async_wait<1>();
        if (tl >= p.L)
            continue;  // nothing there: g is zero (uniform over the warp)
        const int t0 = start(step);
        const typename XIO::Piece *xr = &xring[wp][step % NS][0][lane];
        const typename YIO::Piece *yr = &yring[wp][step % NS][0][lane];
        pair_t<T> dp[Q][TB];
        const int src = ((tg + 1) & (ngr - 1)) * (32 / ngr) + cg;
        const bool tail = p.dlast && t0 + TB > p.L - H;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            uint64_t w[W], bias, g[TB + H];
            taps.read(w, bias, co + 2 * q);
            pair_t<T> xq[H + TB], yq[TB];
            XIO::take(xr, q, xq);
            YIO::take(yr, q, yq);
            with_flag(p.silu, [&](auto silu) {
                uint64_t e[W];
#pragma unroll
                for (int k = 0; k < H; ++k)
                    e[k + 1] = PairOf<T>::f2(xq[k]);
#pragma unroll
                for (int i = 0; i < TB; ++i) {
#pragma unroll
                    for (int k = 0; k < H; ++k)
                        e[k] = e[k + 1];
                    e[H] = PairOf<T>::f2(xq[H + i]);
                    g[i] = PairOf<T>::f2(yq[i]);
                    if (decltype(silu)::value)
                        g[i] = silu_grad2<T>(tap_sum<W>(w, e, bias), g[i]);
                    // Behind the end g is zero, but e still holds the last
                    // inputs: zero times an infinite one is no part of the sum.
                    // (With SiLU such an input makes the g of its own tokens
                    // NaN, and with it every tap's sum.)
                    if (decltype(silu)::value || t0 + i < p.L)
#pragma unroll
                        for (int k = 0; k < W; ++k)
                            dw[q][k] = fma2(g[i], e[k], dw[q][k]);
                    db[q] = add2(db[q], g[i]);
                }
            });
            // the W-1 g behind this block
#pragma unroll
            for (int k = 0; k < H; ++k) {
                const uint64_t give = tg == 0 ? head[q][k] : g[k];
                g[TB + k] = __shfl_sync(0xffffffffu, (unsigned long long)give, src);
                head[q][k] = g[k];
            }
            if (p.dh0 && t0 == 0) {
                // element j of the initial state is input j - (W-1)
#pragma unroll
                for (int j = 0; j < H; ++j) {
                    uint64_t a = 0;
#pragma unroll
                    for (int k = 0; k <= j; ++k)
                        a = fma2(w[k], g[j - k], a);
                    const int c = c0 + 2 * q, o = j - p.L;  // place in dlast, if it is there
                    const float f[2] = {lo2(a), hi2(a)};
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (c + h >= p.dim)
                            continue;
                        const int64_t row = (int64_t(b) * p.dim + c + h) * H;
                        const float more = p.dlast && o >= 0
                                               ? float(static_cast<const T *>(p.dlast)[row + o])
                                               : 0.f;
                        static_cast<T *>(p.dh0)[row + j] = T(f[h] + more);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < TB; ++i) {
                uint64_t a = mul2(w[0], g[i + H]);
#pragma unroll
                for (int k = 1; k < W; ++k)
                    a = fma2(w[k], g[i + H - k], a);
                g[i] = a;
            }
            if (tail) {
                // the state that the sequence ends with is its last inputs
                const int c = c0 + 2 * q;
#pragma unroll
                for (int i = 0; i < TB; ++i)
                    if (t0 + i >= p.L - H && t0 + i < p.L) {
                        const T *dl = static_cast<const T *>(p.dlast) +
                                      (int64_t(b) * p.dim + c) * H + (t0 + i - (p.L - H));
                        g[i] = add2(g[i], pk2(c < p.dim ? float(dl[0]) : 0.f,
                                              c + 1 < p.dim ? float(dl[H]) : 0.f));
                    }
            }
#pragma unroll
            for (int i = 0; i < TB; ++i)
                dp[q][i] = PairOf<T>::round(g[i]);
        }
        if (t0 < p.L)
            store_block<T, XTOK, CH, TB>(dp, p.dx, b, c0, t0, p.dim, p.L);
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
    if (col < cols) {
#pragma unroll 8
        for (int r = r0; r < rows; r += 8)
            a += part[r * cols + col];
    }
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
