// scan_packed.cuh -- the diagonal-A selective scan over packed prompts of
// unequal length, through a cache of states.  Token-major: row t of u, Delta,
// z and y holds the channels of one token, row t of B and C its 16 states'
// factors; sequence i owns rows [start[i], start[i+1]) and slot slots[i] of
// the cache.  Per sequence, channel d and token t
//
//   delta_t = softplus(Delta + bias)      h_t = exp(delta_t A) h_{t-1} + delta_t B_t u_t
//   y_t     = (C_t . h_t + D u_t) * silu(z_t)
//
// from the slot's state (or zero, where seen says that nothing was scanned
// yet), which is left as the state after the sequence's last token.
//
// Work split.  A unit is a segment of at most seg_len tokens of one sequence
// times 128 channels, one thread per channel with its 16 states in registers.
// The lengths are on the device, so the grid holds an upper bound of units,
// tokens / seg_len + seqs, and a block finds its sequence by searching the
// map i -> start[i] / seg_len + i, whose steps leave room for every
// sequence's segments.  A sequence of one segment is scanned in one pass.
// The segments of a longer one do not wait for one another: a first pass
// scans each from zero for its end state E and its sum of step sizes, a small
// kernel folds these along the sequence (h <- exp(A sum delta) h + E), and
// the output pass starts each segment from its folded state.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>
#include <type_traits>

#include "api_common.cuh"
#include "conv.cuh"
#include "f32x2.cuh"
#include "ptx.cuh"
#include "scan_diag.cuh"

namespace selscan {

struct ScanPackedParams {
    PackedIndex ix;
    int dim, seg_len, tiles;
    int vec, bc_vec;    // whole 16-byte (8-byte for B, C) pieces may be read
    const void *u, *delta, *z, *B, *C;
    int64_t su, sd, sz, sB, sC;  // row strides
    void *y;
    int64_t sy;
    const float *A, *delta_bias, *Dskip;
    float *state;  // (slot_count, dim, 16)
    int softplus;
    float *agg;    // [2 (tokens / seg_len) + 2][dim][16]
    float *agg_sd; // [2 (tokens / seg_len) + 2][dim]
};

constexpr int kSpCT = 128;  // channels of a unit

// First entry of a sequence's segments in agg: a sequence of two segments or
// more crosses at least half as many multiples of seg_len.
__device__ __forceinline__ int64_t packed_agg(int begin, int seg_len)
{
    return 2 * int64_t(begin / seg_len);
}

template <typename T>
__device__ __forceinline__ float packed_step(float raw, int softplus)
{
    if (!softplus)
        return raw;
    return std::is_same<T, float>::value ? softplus_exact(raw) : softplus_fast(raw);
}

template <typename T>
struct SpShape {
    static constexpr int kTC = std::is_same<T, float>::value ? 8 : 16;  // tokens staged at once
};

// One chunk of n tokens for one channel.  OUT: also the outputs.
// POW: A[n] = (n+1) A[0], so that the 16 decays are powers of one.
template <typename T, bool OUT, bool POW>
__device__ __forceinline__ void packed_chunk(uint64_t (&h)[8], float &sum, int n, const T *us,
                                             const T *ds, const T *zs, const float *bc,
                                             const uint64_t (&a2)[8], float a0, float bias,
                                             float dskip, int softplus, bool gate, T *y,
                                             int64_t sy, bool live)
{
    constexpr bool kFast = !std::is_same<T, float>::value;
#pragma unroll 4
    for (int t = 0; t < n; ++t) {
        const float u = float(us[t * kSpCT]);
        const float dt = packed_step<T>(float(ds[t * kSpCT]) + bias, softplus);
        const float dx = dt * u;
        const uint64_t dx2 = pk2(dx, dx), dt2 = pk2(dt, dt);
        uint64_t e[8];
        if (POW && kFast) {
            const float r = ex2_approx(dt * a0), r2 = r * r;
            const uint64_t rr = pk2(r2, r2);
            e[0] = pk2(r, r2);
#pragma unroll
            for (int k = 1; k < 8; ++k)
                e[k] = mul2(e[k - 1], rr);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint64_t x = mul2(dt2, a2[k]);
                e[k] = kFast ? pk2(ex2_approx(lo2(x)), ex2_approx(hi2(x)))
                             : pk2(exp_decay(lo2(x)), exp_decay(hi2(x)));
            }
        }
        const ulonglong2 *row = reinterpret_cast<const ulonglong2 *>(bc + t * 32);
        uint64_t acc0 = 0, acc1 = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const ulonglong2 B = row[k];
            h[2 * k] = fma2(e[2 * k], h[2 * k], mul2(dx2, B.x));
            h[2 * k + 1] = fma2(e[2 * k + 1], h[2 * k + 1], mul2(dx2, B.y));
            if (OUT) {
                const ulonglong2 C = row[4 + k];
                acc0 = fma2(C.x, h[2 * k], acc0);
                acc1 = fma2(C.y, h[2 * k + 1], acc1);
            }
        }
        if (OUT) {
            const uint64_t acc = add2(acc0, acc1);
            float v = fmaf(dskip, u, lo2(acc) + hi2(acc));
            if (gate) {
                const float zv = float(zs[t * kSpCT]);
                v *= kFast ? silu_fast(zv) : silu_exact(zv);
            }
            if (live)
                y[t * sy] = T(v);
        } else {
            sum += dt;
        }
    }
}

// OUT false: the first pass of sequences with several segments.
template <typename T, bool OUT>
__global__ void __launch_bounds__(kSpCT) scan_packed_kernel(const __grid_constant__ ScanPackedParams p)
{
    constexpr int TC = SpShape<T>::kTC, VEC = 16 / int(sizeof(T));
    constexpr bool kFast = !std::is_same<T, float>::value;
    __shared__ __align__(16) T tile[2][OUT ? 3 : 2][TC][kSpCT];
    __shared__ __align__(16) float bcf[2][TC][32];
    const PackedIndex &ix = p.ix;
    const int tid = threadIdx.x, lane = tid & 31;
    const int ct = int(blockIdx.x % unsigned(p.tiles));
    const int64_t unit = blockIdx.x / unsigned(p.tiles);

    // with starts in disorder the search may miss a sequence: the units' first
    // blocks look at all of them
    if (OUT && ct == 0 && unit < ix.seqs && tid == 0) {
        const int bg = ix.start[unit], en = ix.start[unit + 1];
        if (ix.slots[unit] >= 0 && (bg < 0 || en < bg || en > ix.tokens))
            atomicOr(ix.err, kErrIndex);
    }
    const int s = packed_find(ix, unit, p.seg_len, 1, lane);
    PackedSeq q;
    if (!packed_seq(ix, s, lane, q))
        return;
    const int64_t seg = unit - (int64_t(q.begin) / p.seg_len + s);
    const int len = q.end - q.begin;
    const int64_t lo = seg * p.seg_len;
    const int cbase = ct * kSpCT, c = cbase + tid;
    const bool live = c < p.dim;
    float *st = p.state + (int64_t(q.slot) * p.dim + (live ? c : 0)) * kDiagN;
    if (seg < 0 || lo >= len) {
        if (OUT && len == 0 && seg == 0 && q.fresh && live)
            for (int k = 0; k < kDiagN; ++k)
                st[k] = 0.f;
        return;
    }
    const bool many = len > p.seg_len;
    const int n_all = int(min(int64_t(p.seg_len), len - lo));
    const bool last = lo + n_all >= len;
    if (!OUT && (!many || last))
        return;
    const int64_t ag = packed_agg(q.begin, p.seg_len) + seg;
    float *agg = p.agg + (ag * p.dim + (live ? c : 0)) * kDiagN;

    uint64_t h[8], a2[8];
    float a0 = 0.f, bias = 0.f, dskip = 0.f;
    bool pow = true;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        h[k] = a2[k] = 0;
    if (live) {
        const float scale = kFast ? kLog2e : 1.f;
        const float2 *ar = reinterpret_cast<const float2 *>(p.A + int64_t(c) * kDiagN);
        const float first = p.A[int64_t(c) * kDiagN];
        a0 = first * scale;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float2 a = ar[k];
            pow = pow && a.x == float(2 * k + 1) * first && a.y == float(2 * k + 2) * first;
            a2[k] = pk2(a.x * scale, a.y * scale);
        }
        if (p.delta_bias)
            bias = p.delta_bias[c];
        if (p.Dskip)
            dskip = p.Dskip[c];
        if (OUT && (many || !q.fresh)) {
            const float2 *src = reinterpret_cast<const float2 *>(many ? agg : st);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float2 v = src[k];
                h[k] = pk2(v.x, v.y);
            }
        }
    }
    pow = __all_sync(0xffffffffu, pow);

    const int t_first = q.begin + int(lo);
    const int chunks = (n_all + TC - 1) / TC;
    const T *src[3] = {static_cast<const T *>(p.u), static_cast<const T *>(p.delta),
                       static_cast<const T *>(p.z)};
    const int64_t stride[3] = {p.su, p.sd, p.sz};
    const bool gate = OUT && p.z;
    const int streams = gate ? 3 : 2;

    // rows of a chunk into shared memory: 16-byte pieces, cut at the last
    // channel and zero-filled behind it
    const auto fetch = [&](int k) {
        const int n = min(TC, n_all - k * TC);
        const int64_t t0 = t_first + int64_t(k) * TC;
        for (int v = 0; v < streams; ++v) {
            const T *b = src[v] + cbase;
            T(*dst)[kSpCT] = tile[k & 1][v];
            if (p.vec) {
                constexpr int PR = kSpCT / VEC;  // pieces per row
                for (int i = tid; i < n * PR; i += kSpCT) {
                    const int r = i / PR, o = (i % PR) * VEC;
                    const int have = min(VEC, max(0, p.dim - cbase - o));
                    cp_async16(&dst[r][o], have ? b + (t0 + r) * stride[v] + o : src[v],
                               uint32_t(have) * uint32_t(sizeof(T)));
                }
            } else {
                for (int r = 0; r < n; ++r)
                    dst[r][tid] = live ? b[(t0 + r) * stride[v] + tid] : T(0.f);
            }
        }
        cp_async_commit();
    };
    // B and C of a chunk: 4 values per thread and 16 tokens
    constexpr int BV = TC * 32 / kSpCT;  // values per thread
    float bcv[BV];
    const auto bc_load = [&](int k) {
        const int r = tid * BV / 32, o = tid * BV % 32;
        const int t = k * TC + r;
        const T *m = static_cast<const T *>(o < 16 ? p.B : p.C) +
                     (int64_t(t_first) + t) * (o < 16 ? p.sB : p.sC) + (o & 15);
        if (t >= n_all || (!OUT && o >= 16)) {
#pragma unroll
            for (int i = 0; i < BV; ++i)
                bcv[i] = 0.f;
        } else if (p.bc_vec) {
            pair_t<T> w[BV / 2];
            load_row<T, BV>(m, w);
#pragma unroll
            for (int i = 0; i < BV / 2; ++i) {
                const uint64_t f = PairOf<T>::f2(w[i]);
                bcv[2 * i] = lo2(f);
                bcv[2 * i + 1] = hi2(f);
            }
        } else {
#pragma unroll
            for (int i = 0; i < BV; ++i)
                bcv[i] = float(m[i]);
        }
    };
    const auto bc_put = [&](int k) {
        float *d = &bcf[k & 1][0][0] + tid * BV;
#pragma unroll
        for (int i = 0; i < BV; ++i)
            d[i] = bcv[i];
    };

    float sum = 0.f;
    fetch(0);
    bc_load(0);
    bc_put(0);
    for (int k = 0; k < chunks; ++k) {
        if (k + 1 < chunks) {
            fetch(k + 1);
            bc_load(k + 1);
            cp_async_wait<1>();
        } else {
            cp_async_wait<0>();
        }
        __syncthreads();
        const int n = min(TC, n_all - k * TC);
        T *y = static_cast<T *>(p.y) + (t_first + int64_t(k) * TC) * p.sy + c;
        const T *us = &tile[k & 1][0][0][tid], *ds = &tile[k & 1][1][0][tid];
        const T *zs = &tile[k & 1][OUT ? 2 : 0][0][tid];
        const float *bc = &bcf[k & 1][0][0];
        if (pow)
            packed_chunk<T, OUT, true>(h, sum, n, us, ds, zs, bc, a2, a0, bias, dskip, p.softplus,
                                       gate, y, p.sy, live);
        else
            packed_chunk<T, OUT, false>(h, sum, n, us, ds, zs, bc, a2, a0, bias, dskip,
                                        p.softplus, gate, y, p.sy, live);
        if (k + 1 < chunks)
            bc_put(k + 1);
        __syncthreads();
    }
    if (!live)
        return;
    if (OUT && !last)
        return;
    float2 *dst = reinterpret_cast<float2 *>(OUT ? st : agg);
#pragma unroll
    for (int k = 0; k < 8; ++k)
        dst[k] = make_float2(lo2(h[k]), hi2(h[k]));
    if (!OUT)
        p.agg_sd[ag * p.dim + c] = sum;
}

// The start state of every segment of the sequences that have several, in
// place of the segments' end states: one thread per channel and state.
static __global__ void __launch_bounds__(256) scan_packed_fold_kernel(const __grid_constant__ ScanPackedParams p)
{
    const PackedIndex &ix = p.ix;
    const int s = int(blockIdx.y);
    const int i = int(blockIdx.x) * 256 + int(threadIdx.x);
    const int begin = ix.start[s], end = ix.start[s + 1];
    if (int64_t(end) - begin <= p.seg_len)
        return;
    PackedSeq q;
    if (!packed_seq(ix, s, threadIdx.x & 31, q) || i >= p.dim * kDiagN)
        return;
    const int c = i / kDiagN;
    const float a = p.A[i];
    const int nseg = (end - begin + p.seg_len - 1) / p.seg_len;
    const int64_t base = packed_agg(begin, p.seg_len);
    float *ag = p.agg + base * p.dim * kDiagN + i;
    const float *sd = p.agg_sd + base * p.dim + c;
    float h = q.fresh ? 0.f : p.state[int64_t(q.slot) * p.dim * kDiagN + i];
    const int64_t hop = int64_t(p.dim) * kDiagN;
#pragma unroll 4
    for (int k = 0; k < nseg - 1; ++k) {
        const float E = ag[k * hop], S = sd[int64_t(k) * p.dim];
        ag[k * hop] = h;
        h = fmaf(expf(a * S), h, E);
    }
    ag[(nseg - 1) * hop] = h;
}

}  // namespace selscan
