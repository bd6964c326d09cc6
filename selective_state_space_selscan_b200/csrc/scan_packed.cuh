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
// times 64 channels, two channels per thread with their states in registers.
// The lengths are on the device, so the grid holds an upper bound of units,
// tokens / seg_len + seqs, and a block finds its sequence by searching the
// map i -> start[i] / seg_len + i, whose steps leave room for every
// sequence's segments.  A sequence of one segment is scanned in one pass.
// The segments of a longer one do not wait for one another: a first pass
// scans each from zero for its end state E and its sum of step sizes, a small
// kernel folds these along the sequence (h <- exp(A sum delta) h + E), and
// the output pass starts each segment from its folded state.  Where there is
// work enough the first pass also writes the outputs of the first segments
// (they and the last then cost one scan, and only those between them two).
//
// What bounds it.  Not HBM (8 bytes per element and pass): a token of a channel
// takes 16 decays, 16 inputs, 16 updates and 16 output products.  With a
// general A the 16 exponentials alone hold the special-function unit for 128 of
// an SM partition's cycles per 32 channels and token (21 with the step size and
// the gate: 168); with A[n] = (n+1) A[0] the packed products hold the FMA pipe
// for about 105 (a packed FMA of three different register pairs issues every
// third cycle, a packed multiply every second, both measured; scalar FMAs in
// their place were 2 % (outputs) to 20 % (updates) slower).  Measured, bf16
// with gate: 131072 x 2048 in one prompt, A[n] = (n+1) A[0], 1.86 ms (pass 1
// 0.74, fold 0.05, output pass 1.1 = 157 cycles); 16384 x 2048 in 32 prompts of
// log-normal lengths, general A, 0.36 ms (0.37 where first segments are scanned
// twice too).  A unit costs its block some 7 us however short it is: 1024 single
// tokens of 2560 channels 0.5 ms (the decode step through slots 0.07).
// Tried and dropped: two of eight pairs of exponentials as polynomials on the
// FMA pipe (10 to 13 instructions per pair instead of 2: issue-bound, 441
// against 408 us), two lanes per channel (414 against 393 us), one channel per
// thread (shared-memory bandwidth, 128 cycles for B and C alone), three staged
// chunks with the outputs leaving through them (fewer blocks per SM).
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

constexpr int kPackedBC = 4;  // values of B or C per load, where bc_vec says so

struct ScanPackedParams {
    PackedIndex ix;
    int dim, seg_len, tiles;
    int vec;            // whole 16-byte pieces of rows may be read
    int y_vec;          // pairs of channels may be written as one word
    int lead;           // first segments' outputs in the first pass
    int bc_vec;         // pieces of kPackedBC values of B and C are aligned loads
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

// First entry of a sequence's segments in agg: a sequence of two segments or
// more crosses at least half as many multiples of seg_len.
__device__ __forceinline__ int64_t packed_agg(int begin, int seg_len)
{
    return 2 * int64_t(begin / seg_len);
}

// 2^x of a pair in fp32: x = n + f with n the nearest integer, 2^f = 1 + f
// p(f) (a least-maximum fit on |f| <= 1/2, relative error 3e-9 before rounding,
// whose first coefficient is ln 2, so that factors next to 1, whose products
// run over thousands of tokens, are not biased), 2^n added to the exponent.
// x is held to [-127, 128], whose ends come out as 0 and infinity (between 2^-127
// and 2^-126 the exponent's sum is off by less than 2^-126); `rest` is what x
// lacks.  The exponent's sum would turn NaN into a number, so a caller whose x may
// be NaN gets x * 0 in `nan`, to be added to what it makes of the result.
__device__ __forceinline__ uint64_t exp2_pair(uint64_t x, const uint64_t *rest, uint64_t *nan)
{
    constexpr float kRound = 12582912.f;  // 1.5 * 2^23: integers in the low bits
    const auto k = [](float v) { return pk2(v, v); };
    const auto hold = [](float v) { return min_nan(max_nan(v, -127.f), 128.f); };
    const uint64_t c = pk2(hold(lo2(x)), hold(hi2(x)));
    const uint64_t t = add2(c, k(kRound));
    uint64_t f = add2(c, fma2(t, k(-1.f), k(kRound)));
    if (rest)
        f = add2(f, *rest);
    if (nan)
        *nan = mul2(c, k(0.f));
    uint64_t q = k(0.00015324314881581813f);
    q = fma2(q, f, k(0.0013390958774834871f));
    q = fma2(q, f, k(0.009618517942726612f));
    q = fma2(q, f, k(0.05550359562039375f));
    q = fma2(q, f, k(0.24022647738456726f));
    q = fma2(q, f, k(kLn2));
    q = fma2(q, f, k(1.f));
    const auto scale = [](float v, float n) {
        return __uint_as_float(__float_as_uint(v) + (__float_as_uint(n) << 23));
    };
    return pk2(scale(lo2(q), lo2(t)), scale(hi2(q), hi2(t)));
}

// exp(x) of a pair: the special-function unit for bf16 results; in fp32 x
// log2 e with what its rounding loses.
template <typename T>
__device__ __forceinline__ uint64_t exp_pair(uint64_t x)
{
    const uint64_t l = pk2(kLog2e, kLog2e);
    if constexpr (!std::is_same<T, float>::value) {
        const uint64_t m = mul2(x, l);
        return pk2(ex2_approx(lo2(m)), ex2_approx(hi2(m)));
    } else {
        // x l - m exactly, and x times the part of log2 e that fp32 does not
        // hold (x finite: infinities have no such rest)
        constexpr float kLog2eLo = 1.92596299e-8f;
        x = pk2(fminf(fmaxf(lo2(x), -87.f), 88.f), fminf(fmaxf(hi2(x), -87.f), 88.f));
        const uint64_t m = mul2(x, l);
        const uint64_t lost = fma2(x, l, mul2(m, pk2(-1.f, -1.f)));
        const uint64_t rest = fma2(x, pk2(kLog2eLo, kLog2eLo), lost);
        return exp2_pair(m, &rest, nullptr);
    }
}

// 1 / d of a pair, d >= 1: in fp32 with a Newton step.  Above 2^126 the result
// is 0 (the unit flushes what is below the normal numbers); a gate is then 0
// where z sigmoid(z) is below 1.1e-36.
template <typename T>
__device__ __forceinline__ uint64_t recip_pair(uint64_t d)
{
    const uint64_t r = pk2(rcp_approx(lo2(d)), rcp_approx(hi2(d)));
    if constexpr (!std::is_same<T, float>::value)
        return r;
    const uint64_t e = fma2(mul2(d, pk2(-1.f, -1.f)), r, pk2(1.f, 1.f));
    return fma2(r, e, r);
}

// softplus(x) = max(x, 0) + log1p(e), e = exp(-|x|) <= 1, with log1p(e) = 2
// atanh(e / (2 + e)): an odd series in s = e / (2 + e) <= 1/3, so that small
// step sizes keep their relative accuracy (about 5e-7 with the fast e and
// reciprocal; lg2 of 1 + e would lose 1.5e-5 where e is 2^-6).  The
// coefficients are a least-maximum fit of 2 atanh(s) / s in s^2 (relative
// error 4e-9).
template <typename T>
__device__ __forceinline__ uint64_t softplus_pair(uint64_t x)
{
    const auto k = [](float v) { return pk2(v, v); };
    const uint64_t e = exp_pair<T>(pk2(-fabsf(lo2(x)), -fabsf(hi2(x))));
    const uint64_t s = mul2(e, recip_pair<T>(add2(e, k(2.f)))), w = mul2(s, s);
    uint64_t q = k(0.2817833423614502f);
    q = fma2(q, w, k(0.27960601449012756f));
    q = fma2(q, w, k(0.40024909377098083f));
    q = fma2(q, w, k(0.6666631698608398f));
    q = fma2(q, w, k(2.0f));
    // NaN passes through the sum; exp_pair in fp32 would hold it to a number
    const uint64_t r = fma2(s, q, pk2(fmaxf(lo2(x), 0.f), fmaxf(hi2(x), 0.f)));
    if constexpr (!std::is_same<T, float>::value)
        return r;
    return pk2(lo2(x) == lo2(x) ? lo2(r) : lo2(x), hi2(x) == hi2(x) ? hi2(r) : hi2(x));
}

// z sigmoid(z) of a pair.
template <typename T>
__device__ __forceinline__ uint64_t gate_pair(uint64_t z)
{
    const uint64_t e = exp_pair<T>(mul2(z, pk2(-1.f, -1.f)));
    return mul2(z, recip_pair<T>(add2(e, pk2(1.f, 1.f))));
}

// Shape of a unit.  A thread holds two adjacent channels (one row of B and C
// from shared memory serves both: at one channel per thread those broadcast
// loads, 128 bytes per channel and token, would bound the kernel), and LPC
// lanes share them, 16 / LPC states each:
//  1: least work per token (the powers of the POW form are one running
//     product);
//  4: a token takes about a quarter of the time, so that most sequences need
//     not be cut into segments to fill the GPU; half as many instructions again
//     per token and channel.  Of four tokens each lane prepares one (step
//     sizes, gate), and they exchange;
//  8: for the smallest calls, whose time is the longest sequence's, half of
//     that again: eight tokens at a time, 32 channels (257 tokens of 64 channels
//     in five prompts, fp32: 18 us, four lanes 27).
template <typename T, int LPC>
struct SpShape {
    static constexpr int kCT = LPC == 8 ? 32 : 64;  // channels
    static constexpr int kThreads = kCT / 2 * LPC;
    static constexpr int kTC = (LPC == 1 ? 32 : 64) / int(sizeof(T));  // tokens staged at once
    // row pitch: with LPC lanes per channel a warp reads LPC rows at once;
    // 128 / LPC bytes more put them into different banks
    static constexpr int kPitch = kCT + (LPC == 1 ? 0 : 128 / LPC / int(sizeof(T)));
    // resident per SM: 168 and 128 registers (six blocks of four lanes, 80
    // registers, spill and were 4 to 20 % slower)
    static constexpr int kBlocks = LPC == 1 ? 12 : 4;
    static constexpr int kGroup = LPC == 8 ? 8 : 4;    // tokens worked on together
    static constexpr int kOwn = kGroup / LPC;          // of these a lane prepares
};

// What a thread holds of its two channels.
template <int LPC>
struct SpChannels {
    static constexpr int Q = 8 / LPC;  // pairs of states
    uint64_t h[2][Q], a2[2][Q];        // the states; A times log2 e
    uint64_t a0, bias, dskip, sum;     // of both channels
    int j;                             // lane of the channels
    int chans;                         // how many of the two exist
    bool pair;                         // both, and y takes them as one word
};

// The decays exp(delta A[n]) of one token of channel ch.  POW: A[n] = (n+1)
// A[0] (bf16), so that they are powers of one exponential.  In fp32 a decay that
// is NaN comes as a number in e and NaN in nan (else 0), which joins the token's
// input: beside the exponential's chain instead of at its end (257 x 64 in five
// prompts 25.1 us, 27.1).
template <typename T, int LPC, bool POW>
__device__ __forceinline__ void packed_decay(uint64_t (&e)[8 / LPC], uint64_t (&nan)[8 / LPC],
                                             const SpChannels<LPC> &s, int ch, float dt)
{
    constexpr bool kFast = !std::is_same<T, float>::value;
    constexpr int Q = 8 / LPC;
    if (POW) {
        const float r = ex2_approx(dt * (ch ? hi2(s.a0) : lo2(s.a0))), r2 = r * r;
        const uint64_t rr = pk2(r2, r2);
        if (LPC == 1) {
            e[0] = pk2(r, r2);
        } else {
            // r^(16 j / LPC + 1) from A itself
            const float f = ex2_approx(dt * lo2(s.a2[ch][0]));
            e[0] = pk2(f, f * r);
        }
#pragma unroll
        for (int k = 1; k < Q; ++k)
            e[k] = mul2(e[k - 1], rr);
        return;
    }
    const uint64_t dt2 = pk2(dt, dt);
#pragma unroll
    for (int k = 0; k < Q; ++k) {
        const uint64_t x = mul2(dt2, s.a2[ch][k]);
        e[k] = kFast ? pk2(ex2_approx(lo2(x)), ex2_approx(hi2(x))) : exp2_pair(x, nullptr, &nan[k]);
    }
}

// Two channels' staged values of one token.
__device__ __forceinline__ uint64_t packed_two(const __nv_bfloat16 *p)
{
    return bf2_to_f2(*reinterpret_cast<const uint32_t *>(p));
}
__device__ __forceinline__ uint64_t packed_two(const float *p)
{
    const float2 v = *reinterpret_cast<const float2 *>(p);
    return pk2(v.x, v.y);
}

// Step size and step size times input of the tokens that this lane prepares.
template <int OWN>
struct SpPrep {
    uint64_t dt[OWN], dx[OWN];
};

template <typename T, int LPC, bool SOFT, bool FULL>
__device__ __forceinline__ SpPrep<SpShape<T, LPC>::kOwn> packed_prepare(const SpChannels<LPC> &s, int t0, int n,
                                                          const T *us, const T *ds)
{
    constexpr int P = SpShape<T, LPC>::kPitch, OWN = SpShape<T, LPC>::kOwn;
    SpPrep<OWN> r;
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
        const int t = t0 + i * LPC + s.j;
        uint64_t d = add2(packed_two(ds + t * P), s.bias);
        if (SOFT)
            d = softplus_pair<T>(d);
        // tokens from n on are not worked on; their step sizes are not summed
        r.dx[i] = mul2(d, packed_two(us + t * P));
        r.dt[i] = FULL || t < n ? d : 0;
    }
    return r;
}

// One token's outputs of channels c and c + 1, of which `chans` exist.
__device__ __forceinline__ void packed_store(__nv_bfloat16 *y, uint64_t v, int chans, bool pair)
{
    if (pair)
        *reinterpret_cast<uint32_t *>(y) = pack2_bf16(lo2(v), hi2(v));
    else {
        if (chans > 0)
            y[0] = __float2bfloat16_rn(lo2(v));
        if (chans > 1)
            y[1] = __float2bfloat16_rn(hi2(v));
    }
}
__device__ __forceinline__ void packed_store(float *y, uint64_t v, int chans, bool pair)
{
    if (pair)
        *reinterpret_cast<float2 *>(y) = make_float2(lo2(v), hi2(v));
    else {
        if (chans > 0)
            y[0] = lo2(v);
        if (chans > 1)
            y[1] = hi2(v);
    }
}

// n tokens (staged at us, ds, zs; B and C rows at bc) of two channels, four at
// a time; the next four's step sizes are prepared meanwhile.  FULL: n is the
// whole chunk.
template <typename T, int LPC, bool OUT, bool POW, bool SOFT, bool GATE, bool FULL>
__device__ __forceinline__ void packed_chunk(SpChannels<LPC> &s, int n, const T *us, const T *ds,
                                             const T *zs, const float *bc, T *y, int64_t sy)
{
    constexpr int P = SpShape<T, LPC>::kPitch, TC = SpShape<T, LPC>::kTC, Q = 8 / LPC;
    constexpr int G = SpShape<T, LPC>::kGroup, OWN = SpShape<T, LPC>::kOwn;
    constexpr bool kFast = !std::is_same<T, float>::value;
    SpPrep<OWN> cur = packed_prepare<T, LPC, SOFT, FULL>(s, 0, n, us, ds);
#pragma unroll 1
    for (int t0 = 0; t0 < (FULL ? TC : n); t0 += G) {
        const SpPrep<OWN> next =
            packed_prepare<T, LPC, SOFT, FULL>(s, min(t0 + G, TC - G), n, us, ds);
        uint64_t part[G];
#pragma unroll
        for (int i = 0; i < G; ++i) {
            if (!FULL && t0 + i >= n) {
                // behind the last token (the same for the whole block): nothing
                // to decay, and exp(0 A) is NaN where A is infinite
                part[i] = 0;
                continue;
            }
            uint64_t d = cur.dt[i / LPC], x = cur.dx[i / LPC];
            if (LPC > 1) {
                const int from = (threadIdx.x & (32 - LPC)) + i % LPC;
                d = pk2(__shfl_sync(0xffffffffu, lo2(d), from), __shfl_sync(0xffffffffu, hi2(d), from));
                x = pk2(__shfl_sync(0xffffffffu, lo2(x), from), __shfl_sync(0xffffffffu, hi2(x), from));
            } else if (!OUT) {
                s.sum = add2(s.sum, d);
            }
            uint64_t e[2][Q], nan[2][Q], acc[2][2];
            packed_decay<T, LPC, POW>(e[0], nan[0], s, 0, lo2(d));
            packed_decay<T, LPC, POW>(e[1], nan[1], s, 1, hi2(d));
            const uint64_t x2[2] = {pk2(lo2(x), lo2(x)), pk2(hi2(x), hi2(x))};
            const float *row = bc + (t0 + i) * 32;  // B, and C 16 behind it
#pragma unroll
            for (int k = 0; k < Q; ++k) {
                // two pairs at a time where there are two
                uint64_t B, C;
                if constexpr (Q > 1) {
                    const ulonglong2 b2 = reinterpret_cast<const ulonglong2 *>(row)[k / 2];
                    const ulonglong2 c2 =
                        OUT ? reinterpret_cast<const ulonglong2 *>(row)[4 + k / 2] : b2;
                    B = k % 2 ? b2.y : b2.x;
                    C = k % 2 ? c2.y : c2.x;
                } else {
                    B = *reinterpret_cast<const uint64_t *>(row);
                    C = OUT ? *reinterpret_cast<const uint64_t *>(row + 16) : B;
                }
#pragma unroll
                for (int ch = 0; ch < 2; ++ch) {
                    uint64_t &h = s.h[ch][k];
                    const uint64_t in = kFast ? mul2(x2[ch], B) : fma2(x2[ch], B, nan[ch][k]);
                    h = fma2(e[ch][k], h, in);
                    if (OUT)
                        acc[ch][k % 2] = k > 1 ? fma2(C, h, acc[ch][k % 2]) : mul2(C, h);
                }
            }
            if (OUT) {
                const uint64_t a = Q > 1 ? add2(acc[0][0], acc[0][1]) : acc[0][0];
                const uint64_t b = Q > 1 ? add2(acc[1][0], acc[1][1]) : acc[1][0];
                part[i] = add2(pk2(lo2(a), lo2(b)), pk2(hi2(a), hi2(b)));
            }
        }
        if (LPC > 1 && !OUT)
#pragma unroll
            for (int i = 0; i < OWN; ++i)
                s.sum = add2(s.sum, cur.dt[i]);
        cur = next;
        if (!OUT)
            continue;
        if (LPC > 1) {
            // the sums of its own tokens come to each lane
            const auto swap = [](uint64_t v, int lanes) {
                return uint64_t(__shfl_xor_sync(0xffffffffu, (unsigned long long)v, lanes));
            };
#pragma unroll
            for (int o = LPC / 2; o > 0; o /= 2)
#pragma unroll
                for (int i = 0; i < o; ++i)
                    part[i] = add2(s.j & o ? part[i + o] : part[i],
                                   swap(s.j & o ? part[i] : part[i + o], o));
        }
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            const int t = t0 + i * LPC + s.j;
            uint64_t v = fma2(s.dskip, packed_two(us + t * P), part[i]);
            if (GATE) {
                v = mul2(v, gate_pair<T>(packed_two(zs + t * P)));
            }
            if (FULL || t < n)
                packed_store(y + t * sy, v, s.chans, s.pair);
        }
    }
}

// FIRST: the first pass, for the states at the segments' ends.  With p.lead it
// also writes the outputs of each sequence's first segment, whose start is
// known; the second pass then has the others only.
template <typename T, int LPC, bool FIRST, bool SOFT, bool GATE>
__global__ void __launch_bounds__(SpShape<T, LPC>::kThreads, SpShape<T, LPC>::kBlocks)
    scan_packed_kernel(const __grid_constant__ ScanPackedParams p)
{
    using Shape = SpShape<T, LPC>;
    constexpr int TC = Shape::kTC, VEC = 16 / int(sizeof(T));
    constexpr int CT = Shape::kCT, NT = Shape::kThreads, Q = 8 / LPC;
    constexpr int NS = GATE ? 3 : 2;  // staged rows: u, Delta, z
    constexpr bool LEADS = LPC == 4;  // p.lead may be set
    constexpr bool kFast = !std::is_same<T, float>::value;
    __shared__ __align__(16) T tile[2][NS][TC][Shape::kPitch];
    __shared__ __align__(16) float bcf[2][TC][32];
    const PackedIndex &ix = p.ix;
    const bool lead = LEADS && p.lead, main = FIRST == lead;  // main: runs in any case
    const int tid = threadIdx.x, lane = tid & 31;
    const int ct = int(blockIdx.x % unsigned(p.tiles));
    const int64_t unit = blockIdx.x / unsigned(p.tiles);

    // with starts in disorder the search may miss a sequence: the units' first
    // blocks look at all of them
    if (main && ct == 0 && unit < ix.seqs && tid == 0) {
        const int bg = ix.start[unit], en = ix.start[unit + 1];
        if (ix.disorder(int(unit), bg, en, ix.slots[unit] >= 0))
            atomicOr(ix.err, kErrIndex);
    }
    const PackedView view(ix, lane);
    const int sq = view.find(unit, p.seg_len, 1);
    PackedSeq q;
    if (!view.get(sq, q))
        return;
    const int64_t seg = unit - (int64_t(q.begin) / p.seg_len + sq);
    const int len = q.end - q.begin;
    const int64_t lo = seg * p.seg_len;
    const int cbase = ct * CT, c = cbase + tid / LPC * 2, j = tid % LPC;  // channels c, c + 1
    const int chans = min(2, max(0, p.dim - c));
    const int n0 = j * (kDiagN / LPC);  // this lane's first state
    float *st = p.state + (int64_t(q.slot) * p.dim + (chans ? c : 0)) * kDiagN + n0;
    if (seg < 0 || lo >= len) {
        if (main && len == 0 && seg == 0 && q.fresh)
            for (int ch = 0; ch < chans; ++ch)
                for (int k = 0; k < kDiagN / LPC; ++k)
                    st[ch * kDiagN + k] = 0.f;
        return;
    }
    const bool many = len > p.seg_len;
    const int n_all = int(min(int64_t(p.seg_len), len - lo));
    const bool last = lo + n_all >= len;
    const bool out = FIRST ? lead && seg == 0 : true;  // y is written
    if (FIRST ? !out && last : lead && seg == 0)
        return;
    const int64_t ag = packed_agg(q.begin, p.seg_len);
    const int nseg = (len - 1) / p.seg_len + 1;
    // agg[k] of a sequence: the end of segment k, the start of k + 1; the last
    // entry the start of the first, where the second pass has that too
    const auto agg = [&](int64_t k) {
        return p.agg + ((ag + k) * p.dim + (chans ? c : 0)) * kDiagN + n0;
    };

    const int t_first = q.begin + int(lo);
    const int chunks = (n_all + TC - 1) / TC;
    const T *src[3] = {static_cast<const T *>(p.u), static_cast<const T *>(p.delta),
                       static_cast<const T *>(p.z)};
    const int64_t stride[3] = {p.su, p.sd, p.sz};
    constexpr int PR = CT / VEC;  // 16-byte pieces of a row

    // rows of a chunk into shared memory: 16-byte pieces, cut at the last
    // channel and zero-filled behind it
    const int pr = tid / PR, po = (tid % PR) * VEC;
    const int have = min(VEC, max(0, p.dim - cbase - po));
    const T *at[NS];
#pragma unroll
    for (int v = 0; v < NS; ++v)
        at[v] = src[v] + (have ? (int64_t(t_first) + pr) * stride[v] + cbase + po : 0);
    const auto fetch = [&](int k, int buf) {
        const int n = min(TC, n_all - k * TC);
        constexpr int STEP = NT / PR;  // rows between a thread's pieces
#pragma unroll
        for (int v = 0; v < NS; ++v) {
            if (FIRST && v == 2 && !out)
                break;
            if (p.vec) {
                const T *g = at[v];
#pragma unroll
                for (int i = 0; i < (TC + STEP - 1) / STEP; ++i) {
                    if (pr + i * STEP < n)
                        cp_async16(&tile[buf][v][pr + i * STEP][po], g,
                                   uint32_t(have) * uint32_t(sizeof(T)));
                    g += have ? STEP * stride[v] : 0;
                }
                at[v] += have ? TC * stride[v] : 0;
            } else {
                const T *b = src[v] + (t_first + int64_t(k) * TC) * stride[v] + cbase;
                for (int i = tid; i < n * CT; i += NT) {
                    const int r = i / CT, o = i % CT;
                    tile[buf][v][r][o] = cbase + o < p.dim ? b[r * stride[v] + o] : T(0.f);
                }
            }
        }
        cp_async_commit();
    };
    // B and C of a chunk: loaded a chunk ahead as they are, widened to fp32
    // when they are stored
    constexpr int BV = kPackedBC, BN = (TC * 32 / BV + NT - 1) / NT;  // values per load, loads
    static_assert(BV == 4, "the pieces below are written out for four values");
    pair_t<T> bcw[BN][BV / 2];
    const auto bc_load = [&](int k) {
#pragma unroll
        for (int l = 0; l < BN; ++l) {
            const int i = (l * NT + tid) * BV, r = i / 32, o = i % 32;
            const int t = k * TC + r;
            const T *m = static_cast<const T *>(o < 16 ? p.B : p.C) +
                         (int64_t(t_first) + t) * (o < 16 ? p.sB : p.sC) + (o & 15);
            if (r >= TC || t >= n_all || (FIRST && !out && o >= 16)) {
                bcw[l][0] = bcw[l][1] = 0;
            } else if (p.bc_vec) {
                load_row<T, BV>(m, bcw[l]);
            } else {
                bcw[l][0] = PairOf<T>::make(m[0], m[1]);
                bcw[l][1] = PairOf<T>::make(m[2], m[3]);
            }
        }
    };
    const auto bc_put = [&](int k) {
#pragma unroll
        for (int l = 0; l < BN; ++l) {
            const uint64_t a = PairOf<T>::f2(bcw[l][0]), c2 = PairOf<T>::f2(bcw[l][1]);
            if ((l * NT + tid) * BV < TC * 32)
                *reinterpret_cast<float4 *>(&bcf[k & 1][0][0] + (l * NT + tid) * BV) =
                    make_float4(lo2(a), hi2(a), lo2(c2), hi2(c2));
        }
    };
    fetch(0, 0);
    bc_load(0);

    SpChannels<LPC> s;
    s.j = j;
    s.chans = chans;
    s.pair = chans == 2 && p.y_vec;
    bool pow = kFast;
    {
        float a0[2] = {0.f, 0.f}, bias[2] = {0.f, 0.f}, dskip[2] = {0.f, 0.f};
#pragma unroll
        for (int ch = 0; ch < 2; ++ch) {
#pragma unroll
            for (int k = 0; k < Q; ++k)
                s.h[ch][k] = s.a2[ch][k] = 0;
            if (ch >= chans)
                continue;
            const float *ar = p.A + int64_t(c + ch) * kDiagN;
            const float first = ar[0];
            a0[ch] = first * kLog2e;
#pragma unroll
            for (int k = 0; k < Q; ++k) {
                const float2 a = *reinterpret_cast<const float2 *>(ar + n0 + 2 * k);
                pow = pow && a.x == float(n0 + 2 * k + 1) * first &&
                      a.y == float(n0 + 2 * k + 2) * first;
                s.a2[ch][k] = pk2(a.x * kLog2e, a.y * kLog2e);
            }
            if (p.delta_bias)
                bias[ch] = p.delta_bias[c + ch];
            if (p.Dskip)
                dskip[ch] = p.Dskip[c + ch];
            // the second pass starts from what the first left, the first (and
            // a sequence of one segment) from the cache
            const bool left = !FIRST && many;
            if (left || (seg == 0 && !q.fresh)) {
                const float *from = (left ? agg(seg ? seg - 1 : nseg - 1) : st) + ch * kDiagN;
#pragma unroll
                for (int k = 0; k < Q; ++k) {
                    const float2 v = *reinterpret_cast<const float2 *>(from + 2 * k);
                    s.h[ch][k] = pk2(v.x, v.y);
                }
            }
            if (FIRST && !lead && seg == 0) {
                float *keep = agg(nseg - 1) + ch * kDiagN;
#pragma unroll
                for (int k = 0; k < Q; ++k)
                    *reinterpret_cast<float2 *>(keep + 2 * k) = make_float2(lo2(s.h[ch][k]), hi2(s.h[ch][k]));
            }
        }
        s.a0 = pk2(a0[0], a0[1]);
        s.bias = pk2(bias[0], bias[1]);
        s.dskip = pk2(dskip[0], dskip[1]);
        s.sum = 0;
    }
    pow = __all_sync(0xffffffffu, pow);
    bc_put(0);

    for (int k = 0; k < chunks; ++k) {
        const int buf = k & 1;
        cp_async_wait<0>();
        __syncthreads();  // chunk k is there; chunk k - 1 is done
        if (k + 1 < chunks) {
            fetch(k + 1, buf ^ 1);
            bc_load(k + 1);
        }
        const int n = min(TC, n_all - k * TC);
        const T *us = &tile[buf][0][0][tid / LPC * 2];
        const T *ds = &tile[buf][1][0][tid / LPC * 2], *zs = &tile[buf][NS - 1][0][tid / LPC * 2];
        const float *bc = &bcf[buf][0][n0];
        T *y = out ? static_cast<T *>(p.y) + (t_first + int64_t(k) * TC) * p.sy + c : nullptr;
        const auto scan = [&](auto o) {
            constexpr bool OUT = decltype(o)::value;
            if (kFast && pow && n == TC)
                packed_chunk<T, LPC, OUT, kFast, SOFT, GATE, kFast>(s, n, us, ds, zs, bc, y, p.sy);
            else if (n == TC)
                packed_chunk<T, LPC, OUT, false, SOFT, GATE, true>(s, n, us, ds, zs, bc, y, p.sy);
            else
                packed_chunk<T, LPC, OUT, false, SOFT, GATE, false>(s, n, us, ds, zs, bc, y, p.sy);
        };
        if constexpr (FIRST && LEADS)
            out ? scan(std::true_type()) : scan(std::false_type());
        else
            scan(std::bool_constant<!FIRST>());
        if (k + 1 < chunks)
            bc_put(k + 1);
    }
    if (!FIRST && !last)
        return;
    float sum[2] = {lo2(s.sum), hi2(s.sum)};
#pragma unroll
    for (int ch = 0; ch < 2; ++ch) {
        if (FIRST)
#pragma unroll
            for (int o = 1; o < LPC; o *= 2)
                sum[ch] += __shfl_xor_sync(0xffffffffu, sum[ch], o);
        if (ch >= chans)
            continue;
        float *dst = (last ? st : agg(seg)) + ch * kDiagN;
#pragma unroll
        for (int k = 0; k < Q; ++k)
            *reinterpret_cast<float2 *>(dst + 2 * k) = make_float2(lo2(s.h[ch][k]), hi2(s.h[ch][k]));
        if (FIRST && !last && j == 0)
            p.agg_sd[(ag + seg) * p.dim + c + ch] = sum[ch];
    }
}

// The states at the ends of the segments of sequences that have three or more,
// but for the first's and the last's, in place of what these scanned from zero:
// one thread per channel and state.
static __global__ void __launch_bounds__(256) scan_packed_fold_kernel(const __grid_constant__ ScanPackedParams p)
{
    const PackedIndex &ix = p.ix;
    const int s = int(blockIdx.y);
    const int i = int(blockIdx.x) * 256 + int(threadIdx.x);
    const int begin = ix.start[s], end = ix.start[s + 1];
    if (int64_t(end) - begin <= 2 * int64_t(p.seg_len))
        return;
    PackedSeq q;
    const PackedView view(ix, threadIdx.x & 31);
    if (!view.get(s, q) || i >= p.dim * kDiagN)
        return;
    const int c = i / kDiagN;
    const float a = p.A[i];
    const int nseg = (end - begin - 1) / p.seg_len + 1;
    const int64_t base = packed_agg(begin, p.seg_len);
    float *ag = p.agg + base * p.dim * kDiagN + i;
    const float *sd = p.agg_sd + base * p.dim + c;
    const int64_t hop = int64_t(p.dim) * kDiagN;
    float h = ag[0];
    // eight segments' numbers at a time: one after the other, each would cost a
    // trip to memory (37 segments of 2048 channels: 82 us, now 14; 293: 49)
    constexpr int AHEAD = 8;
    for (int k0 = 1; k0 < nseg - 1; k0 += AHEAD) {
        float E[AHEAD], S[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            const bool in = k0 + j < nseg - 1;
            E[j] = in ? ag[(k0 + j) * hop] : 0.f;
            S[j] = in ? sd[int64_t(k0 + j) * p.dim] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
            if (k0 + j < nseg - 1) {
                // a state of zero stays zero also where a positive A makes the
                // segment's decay infinite (0.3 % of 131072 x 2048)
                h = h == 0.f ? E[j] : fmaf(expf(a * S[j]), h, E[j]);
                ag[(k0 + j) * hop] = h;
            }
    }
}

}  // namespace selscan
