// layer_api.cu -- C entry points of the operators around the scan (see
// include/selscan.h): the short causal convolution (forward, backward, one
// token, packed prompts) and the scan over packed prompts.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdlib>
#include <cstdint>

#include "selscan.h"
#include "selscan_debug.h"
#include "api_common.cuh"
#include "conv.cuh"
#include "scan_packed.cuh"

using namespace selscan;

namespace {

constexpr int64_t kMaxLen = (int64_t(1) << 31) - 1024;
constexpr int64_t kMaxDim = int64_t(1) << 30;

bool mult16(int64_t stride, int64_t es) { return ((stride * es) & 15) == 0; }

// A (batch, dim, L) tensor of element type dt with any non-negative strides
// (an output's may not be zero where there is something to step over).
selscan_status check_bdl(const selscan_tensor *t, int64_t batch, int64_t dim, int64_t L,
                         int32_t dt, bool output)
{
    if (!present(t))
        return SELSCAN_ERR_NULL;
    if (t->ndim != 3 || t->shape[0] != batch || t->shape[1] != dim || t->shape[2] != L)
        return SELSCAN_ERR_SHAPE;
    if (t->dtype != dt)
        return SELSCAN_ERR_DTYPE;
    if (batch == 0 || dim == 0 || L == 0)
        return SELSCAN_OK;
    for (int i = 0; i < 3; ++i)
        if (t->stride[i] < 0 || (output && t->shape[i] > 1 && t->stride[i] == 0))
            return SELSCAN_ERR_STRIDE;
    if (reinterpret_cast<uintptr_t>(t->data) % elem_size(dt))
        return SELSCAN_ERR_ALIGN;
    return SELSCAN_OK;
}

// A contiguous state tensor of element type dt; NULL where there may be none.
selscan_status check_state(const selscan_tensor *t, int ndim, const int64_t *shape, int32_t dt,
                           bool nullable)
{
    if (!t || !t->data) {
        if (nullable && (!t || numel(t) != 0 || t->ndim < 1))
            return t ? SELSCAN_ERR_NULL : SELSCAN_OK;
        if (!present(t))
            return SELSCAN_ERR_NULL;
    }
    if (t->ndim != ndim)
        return SELSCAN_ERR_SHAPE;
    int64_t expect = 1;
    for (int i = ndim - 1; i >= 0; --i)
        if (t->shape[i] != shape[i])
            return SELSCAN_ERR_SHAPE;
    if (t->dtype != dt)
        return SELSCAN_ERR_DTYPE;
    if (numel(t) > 0)
        for (int i = ndim - 1; i >= 0; --i) {
            if (shape[i] > 1 && t->stride[i] != expect)
                return SELSCAN_ERR_STRIDE;
            expect *= shape[i];
        }
    if (reinterpret_cast<uintptr_t>(t->data) % elem_size(dt))
        return SELSCAN_ERR_ALIGN;
    return SELSCAN_OK;
}

// weight (dim, W) and bias (dim); returns W through *width.
selscan_status check_taps(const selscan_tensor *weight, const selscan_tensor *bias, int64_t dim,
                          int64_t *width)
{
    if (!present(weight))
        return SELSCAN_ERR_NULL;
    if (weight->ndim != 2)
        return SELSCAN_ERR_SHAPE;
    *width = weight->shape[1];
    const int64_t ws[2] = {dim, *width}, bs[1] = {dim};
    selscan_status st;
    if ((st = check_param(weight, 2, ws, false)) != SELSCAN_OK) return st;
    if ((st = check_param(bias, 1, bs, true)) != SELSCAN_OK) return st;
    return SELSCAN_OK;
}

// Whether the channels are the direction in which a tensor's elements are
// neighbours.
bool token_major(const selscan_tensor *t)
{
    return t->stride[1] == 1 && (t->stride[2] != 1 || t->shape[2] == 1);
}

ConvView view_of(const selscan_tensor *t, bool tok)
{
    const int64_t es = int64_t(elem_size(t->dtype));
    ConvView v{t->data, t->stride[0], t->stride[1], t->stride[2], 0};
    const bool base = aligned16(t->data) && (t->shape[0] <= 1 || mult16(v.sb, es));
    v.vec = tok ? base && v.sd == 1 && (t->shape[2] <= 1 || mult16(v.st, es))
                : base && v.st == 1 && (t->shape[1] <= 1 || mult16(v.sd, es));
    return v;
}

// Channel blocks of a warp (as a power of two): `want` for the layouts, fewer
// where the channels do not fill them, more where the tokens do not fill the
// rest.
int channel_blocks_log2(int want, int64_t cblocks, int64_t tblocks)
{
    int g = want;
    while (g > 0 && (int64_t(1) << (g - 1)) >= cblocks)
        --g;
    while (g < 5 && (32 >> (g + 1)) >= tblocks)
        ++g;
    return g;
}

template <typename T, int W>
void launch_conv(const ConvParams &p, bool xt, bool yt, dim3 grid, cudaStream_t s)
{
    if (xt)
        yt ? conv_fwd_kernel<T, W, true, true><<<grid, 128, 0, s>>>(p)
           : conv_fwd_kernel<T, W, true, false><<<grid, 128, 0, s>>>(p);
    else
        yt ? conv_fwd_kernel<T, W, false, true><<<grid, 128, 0, s>>>(p)
           : conv_fwd_kernel<T, W, false, false><<<grid, 128, 0, s>>>(p);
}

template <typename T, int W>
void launch_conv_bwd(const ConvBwdParams &p, bool xt, bool yt, dim3 grid, cudaStream_t s)
{
    if (xt)
        yt ? conv_bwd_kernel<T, W, true, true><<<grid, 128, 0, s>>>(p)
           : conv_bwd_kernel<T, W, true, false><<<grid, 128, 0, s>>>(p);
    else
        yt ? conv_bwd_kernel<T, W, false, true><<<grid, 128, 0, s>>>(p)
           : conv_bwd_kernel<T, W, false, false><<<grid, 128, 0, s>>>(p);
}

// Rows of a block of the convolution's single-token kernel: as many as let one
// wave of blocks (four per SM) hold the batch, at most kConvStepRows.  A
// block's taps are read once for its rows.
int conv_step_rows(int64_t batch, int64_t gx, int64_t sms)
{
    const int64_t rows = (batch * gx + 4 * sms - 1) / (4 * sms);
    return int(std::min<int64_t>(std::max<int64_t>(rows, 1), kConvStepRows));
}

// kConvRun rows at a time, how many times a warp of the packed convolution
// takes them: as few as let one wave of blocks (three per SM, whose 168 registers
// hold the next rows: 21.6 us for 8192 x 2560 bf16; four 25.4, five 29.1) hold
// the rows.
int conv_packed_subs(int64_t tokens, int64_t ctiles, int64_t sms)
{
    const int64_t blocks = (tokens + 4 * kConvRun - 1) / (4 * kConvRun) * ctiles;
    return int(std::min<int64_t>(std::max<int64_t>((blocks + 3 * sms - 1) / (3 * sms), 1),
                                 kConvSubs));
}

int g_dbg_packed_seg = 0;    // test hooks, see selscan_debug_packed_segment
int g_dbg_packed_lanes = 0;

struct PackedPlan {
    int lanes;    // per channel
    bool lead;    // outputs of first segments in the first pass
    int seg_len;  // tokens of a segment
};

// Lanes per channel and tokens per segment of packed prompts, from the numbers
// of rows, sequences and channels (the lengths are on the device).  All figures
// bf16 with gate, general A where none is named, us, both sides measured when the
// rule was chosen (the kernels have become up to 2 % slower since, all alike).
// Lanes: eight up to 2^20 elements, where the longest sequence's own time counts
// (257 x 64 fp32 in five prompts 18, four lanes 27; 300 x 768 in one 19 against
// 24; but 16000 x 256 in 16 78 against 70).  One, which does the least work,
// where the average sequence would be cut up in any case and the rows fill the
// GPU (131072 x 2048 in one prompt, A[n] = (n+1) A[0], 1840 against 2600; 16384
// x 2048 in one 377 against 399; but 8192 x 2048 in 16 234 against 197).  Four
// otherwise (16384 x 2048 in 32 prompts 362, one lane 472).
// Segments: the rows' share of some waves of warps.  One lane: 16 warps per SM,
// a wave and a third, and twice, four times, ... as many where segments would be
// longer than 512, several sequences' than 192, whose ends leave gaps that
// shorter ones fill (131072 x 2048 1840, unhalved 1872; 32768 x 5120 in two
// 1720 against 1965; 16384 x 2048 in four 382 against 424).  Four lanes: 44
// warps per SM; with `lead` 60, since first segments cost no second scan (256
// tokens 357, 336 364, 512 376).
// lead: where the rows fill the GPU (32768 x 2048 in 64 prompts 633, without 700;
// 8192 x 2048 in 16 197 against 205); short of that, the first pass takes as long
// as its slowest segment, which outputs make slower (16000 x 256 in 16 73 against
// 70).
PackedPlan packed_plan(int64_t tokens, int64_t seqs, int64_t dim, int64_t sms)
{
    const int64_t warps1 = (dim + 63) / 64, warps4 = 4 * warps1;
    const auto seg_of = [&](int64_t warps, int64_t slots) {
        return std::max<int64_t>(64, ((tokens * warps + slots - 1) / slots + 15) / 16 * 16);
    };
    // short calls in one launch: cut up, they would take three
    const bool brief = tokens <= 128 || (tokens <= 512 && tokens <= 64 * seqs);
    const int64_t seg4 = brief ? tokens + 1 : seg_of(warps4, 44 * sms);
    const int dbg = g_dbg_packed_lanes;
    PackedPlan plan;
    plan.lanes = dbg                                       ? std::abs(dbg)
                 : tokens * dim <= (int64_t(1) << 20)      ? 8
                 : tokens > 2 * seqs * seg4 && seg4 >= 256 ? 1
                                                           : 4;
    plan.lead = dbg ? dbg < 0 : plan.lanes == 4 && !brief && seg4 > 128;
    int64_t seg = plan.lead ? seg_of(warps4, 60 * sms) : seg4;
    if (plan.lanes == 1) {
        int64_t slots = 16 * sms;
        while ((seg = seg_of(warps1, slots)) > (seqs == 1 ? 512 : 192))
            slots *= 2;
    }
    plan.seg_len = g_dbg_packed_seg ? g_dbg_packed_seg : int(std::min(seg, kMaxLen));
    return plan;
}

template <bool FIRST, bool GATE, bool SOFT>
void launch_packed(const ScanPackedParams &p, bool bf, int lanes, unsigned grid, cudaStream_t s)
{
    const auto go = [&](auto tag, auto l) {
        using T = decltype(tag);
        constexpr int LPC = decltype(l)::value;
        scan_packed_kernel<T, LPC, FIRST, SOFT, GATE>
            <<<grid, SpShape<T, LPC>::kThreads, 0, s>>>(p);
    };
    const auto with = [&](auto tag) {
        if constexpr (!(FIRST && GATE)) {
            if (lanes == 1)
                return go(tag, std::integral_constant<int, 1>());
            if (lanes == 8)
                return go(tag, std::integral_constant<int, 8>());
        }
        go(tag, std::integral_constant<int, 4>());
    };
    bf ? with(__nv_bfloat16()) : with(float());
}

template <bool FIRST>
cudaError_t launch_packed(const ScanPackedParams &p, bool bf, int lanes, unsigned grid, cudaStream_t s)
{
    if (p.z && (!FIRST || p.lead))
        p.softplus ? launch_packed<FIRST, true, true>(p, bf, lanes, grid, s)
                   : launch_packed<FIRST, true, false>(p, bf, lanes, grid, s);
    else
        p.softplus ? launch_packed<FIRST, false, true>(p, bf, lanes, grid, s)
                   : launch_packed<FIRST, false, false>(p, bf, lanes, grid, s);
    return counted_launch();
}

// f(T tag, integral constant W) for the element type and tap count at hand.
template <typename F>
void dispatch(int32_t dt, int64_t width, F f)
{
    const auto with = [&](auto tag) {
        if (width == 2)
            f(tag, std::integral_constant<int, 2>());
        else if (width == 3)
            f(tag, std::integral_constant<int, 3>());
        else
            f(tag, std::integral_constant<int, 4>());
    };
    if (dt == SELSCAN_BF16)
        with(__nv_bfloat16());
    else
        with(float());
}

// Packed prompts: the rows' and the sequences' index arrays.
selscan_status check_packed(const selscan_tensor *state, const selscan_tensor *start,
                            const selscan_tensor *slots, const selscan_tensor *seen,
                            int64_t tokens, PackedIndex *ix)
{
    if (!present(state) || !present(start) || !slots)
        return SELSCAN_ERR_NULL;
    if (slots->ndim != 1 || slots->shape[0] < 0)
        return SELSCAN_ERR_SHAPE;
    const int64_t seqs = slots->shape[0];
    selscan_status st;
    if ((st = check_index(slots, seqs, false)) != SELSCAN_OK) return st;
    if ((st = check_index(start, seqs + 1, false)) != SELSCAN_OK) return st;
    if ((st = check_index(seen, seqs, true)) != SELSCAN_OK) return st;
    if (tokens > kMaxLen || seqs > 65535 || state->shape[0] > 0x7fffffffll)
        return SELSCAN_ERR_UNSUPPORTED;
    ix->tokens = int(tokens);
    ix->seqs = int(seqs);
    ix->slot_count = int(state->shape[0]);
    ix->start = static_cast<const int *>(start->data);
    ix->slots = static_cast<const int *>(slots->data);
    ix->seen = seen ? static_cast<const int *>(seen->data) : nullptr;
    return SELSCAN_OK;
}

// A (tokens, cols) operand of packed prompts: contiguous columns, any row
// stride (an output's rows may not lie on one another).
selscan_status check_rows(const selscan_tensor *t, int64_t tokens, int64_t cols, int32_t dt,
                          bool output)
{
    selscan_status st = check_tok(t, tokens, cols, dt);
    if (st != SELSCAN_OK || tokens == 0 || cols == 0)
        return st;
    if (cols > 1 && t->stride[1] != 1)
        return SELSCAN_ERR_STRIDE;
    if (output && tokens > 1 && t->stride[0] < cols)
        return SELSCAN_ERR_STRIDE;
    return SELSCAN_OK;
}

bool rows_vec(const selscan_tensor *t, int64_t es)
{
    return aligned16(t->data) && (t->shape[0] <= 1 || mult16(t->stride[0], es));
}

// Bytes of one load of B or C of packed prompts: a piece of kPackedBC values (8
// in bf16, 16 in fp32) where every row's pieces are aligned to that, else 0
// (value by value).
int64_t packed_piece_bytes(const selscan_tensor *t)
{
    const int64_t es = int64_t(elem_size(t->dtype)), piece = kPackedBC * es;
    const bool ok = reinterpret_cast<uintptr_t>(t->data) % uintptr_t(piece) == 0 &&
                    (t->shape[0] <= 1 || (t->stride[0] * es) % piece == 0);
    return ok ? piece : 0;
}

}  // namespace

extern "C" selscan_status selscan_conv(const selscan_tensor *x, const selscan_tensor *weight,
                                       const selscan_tensor *bias, int silu,
                                       const selscan_tensor *h0, selscan_tensor *y,
                                       selscan_tensor *last_state, cudaStream_t stream)
{
    if (!present(x) || !weight || !y)
        return SELSCAN_ERR_NULL;
    if (x->ndim != 3)
        return SELSCAN_ERR_SHAPE;
    const int32_t dt = x->dtype;
    if (dt != SELSCAN_F32 && dt != SELSCAN_BF16)
        return SELSCAN_ERR_DTYPE;
    const int64_t batch = x->shape[0], dim = x->shape[1], L = x->shape[2];
    if (batch < 0 || dim < 0 || L < 0)
        return SELSCAN_ERR_SHAPE;
    selscan_status st;
    int64_t W = 0;
    if ((st = check_bdl(x, batch, dim, L, dt, false)) != SELSCAN_OK) return st;
    if ((st = check_bdl(y, batch, dim, L, dt, true)) != SELSCAN_OK) return st;
    if ((st = check_taps(weight, bias, dim, &W)) != SELSCAN_OK) return st;
    const int64_t sshape[3] = {batch, dim, W - 1};
    if ((st = check_state(h0, 3, sshape, dt, true)) != SELSCAN_OK) return st;
    if ((st = check_state(last_state, 3, sshape, dt, true)) != SELSCAN_OK) return st;
    if (W < 2 || W > 4 || batch > 65535 || dim > kMaxDim || L > kMaxLen)
        return SELSCAN_ERR_UNSUPPORTED;
    if (batch == 0 || dim == 0)
        return SELSCAN_OK;
    if (L == 0) {
        // no input: the final state is the initial one (zero if none)
        if (!last_state || !last_state->data || last_state->data == opt_data(h0))
            return SELSCAN_OK;
        const size_t bytes = size_t(batch * dim * (W - 1)) * elem_size(dt);
        const cudaError_t e =
            opt_data(h0) ? cudaMemcpyAsync(last_state->data, h0->data, bytes,
                                           cudaMemcpyDeviceToDevice, stream)
                         : cudaMemsetAsync(last_state->data, 0, bytes, stream);
        return e == cudaSuccess ? SELSCAN_OK : SELSCAN_ERR_CUDA;
    }

    const bool xt = token_major(x), yt = token_major(y);
    const int64_t blk = 16 / int64_t(elem_size(dt));  // channels and tokens of a thread
    const int64_t cblocks = (dim + blk - 1) / blk, tblocks = (L + blk - 1) / blk;
    ConvParams p{};
    p.batch = int(batch);
    p.dim = int(dim);
    p.L = int(L);
    p.cg_log2 = channel_blocks_log2(xt ? (yt ? 5 : 2) : (yt ? 2 : 0), cblocks, tblocks);
    p.ctiles = int((cblocks + (1 << p.cg_log2) - 1) >> p.cg_log2);
    const int ngr = 32 >> p.cg_log2;
    p.ttiles = int((tblocks + ngr - 1) / ngr);
    p.x = view_of(x, xt);
    p.y = view_of(y, yt);
    p.weight = static_cast<const float *>(weight->data);
    p.bias = static_cast<const float *>(opt_data(bias));
    p.h0 = opt_data(h0);
    p.last = last_state ? last_state->data : nullptr;
    p.silu = silu ? 1 : 0;
    const int64_t gx = int64_t(p.ctiles) * ((p.ttiles + 3) / 4);
    if (gx > 0x7fffffffll)
        return SELSCAN_ERR_UNSUPPORTED;
    const dim3 grid{unsigned(gx), unsigned(batch)};
    dispatch(dt, W, [&](auto tag, auto w) {
        launch_conv<decltype(tag), decltype(w)::value>(p, xt, yt, grid, stream);
    });
    return counted_launch() == cudaSuccess ? SELSCAN_OK : SELSCAN_ERR_CUDA;
}

extern "C" selscan_status selscan_conv_bwd(const selscan_tensor *x, const selscan_tensor *weight,
                                           const selscan_tensor *bias, int silu,
                                           const selscan_tensor *h0, const selscan_tensor *dy,
                                           const selscan_tensor *dlast, selscan_tensor *dx,
                                           selscan_tensor *dweight, selscan_tensor *dbias,
                                           selscan_tensor *dh0, cudaStream_t stream)
{
    if (!present(x) || !weight || !dy || !dx || !dweight)
        return SELSCAN_ERR_NULL;
    if (x->ndim != 3)
        return SELSCAN_ERR_SHAPE;
    const int32_t dt = x->dtype;
    if (dt != SELSCAN_F32 && dt != SELSCAN_BF16)
        return SELSCAN_ERR_DTYPE;
    const int64_t batch = x->shape[0], dim = x->shape[1], L = x->shape[2];
    if (batch < 0 || dim < 0 || L < 0)
        return SELSCAN_ERR_SHAPE;
    selscan_status st;
    int64_t W = 0;
    if ((st = check_bdl(x, batch, dim, L, dt, false)) != SELSCAN_OK) return st;
    if ((st = check_bdl(dy, batch, dim, L, dt, false)) != SELSCAN_OK) return st;
    if ((st = check_bdl(dx, batch, dim, L, dt, true)) != SELSCAN_OK) return st;
    if ((st = check_taps(weight, bias, dim, &W)) != SELSCAN_OK) return st;
    const int64_t sshape[3] = {batch, dim, W - 1}, wshape[2] = {dim, W}, bshape[1] = {dim};
    if ((st = check_param(dweight, 2, wshape, false)) != SELSCAN_OK) return st;
    if ((st = check_param(dbias, 1, bshape, true)) != SELSCAN_OK) return st;
    for (const selscan_tensor *t : {h0, dlast, static_cast<const selscan_tensor *>(dh0)})
        if ((st = check_state(t, 3, sshape, dt, true)) != SELSCAN_OK) return st;
    if (W < 2 || W > 4 || batch > 65535 || dim > kMaxDim || L > kMaxLen)
        return SELSCAN_ERR_UNSUPPORTED;
    if (dim == 0)
        return SELSCAN_OK;
    if (batch == 0 || L == 0) {
        // nothing to sum over; the initial state is the final one
        if (cudaMemsetAsync(dweight->data, 0, size_t(dim * W) * 4, stream) != cudaSuccess ||
            (dbias && dbias->data &&
             cudaMemsetAsync(dbias->data, 0, size_t(dim) * 4, stream) != cudaSuccess))
            return SELSCAN_ERR_CUDA;
        if (batch == 0 || !dh0 || !dh0->data)
            return SELSCAN_OK;
        const size_t bytes = size_t(batch * dim * (W - 1)) * elem_size(dt);
        const cudaError_t e =
            opt_data(dlast) ? cudaMemcpyAsync(dh0->data, dlast->data, bytes,
                                              cudaMemcpyDeviceToDevice, stream)
                            : cudaMemsetAsync(dh0->data, 0, bytes, stream);
        return e == cudaSuccess ? SELSCAN_OK : SELSCAN_ERR_CUDA;
    }

    int dev = 0;
    DeviceInfo *di = nullptr;
    if ((st = device_setup(&dev, &di)) != SELSCAN_OK)
        return st;
    const bool xt = token_major(x), yt = token_major(dy);
    const int64_t ch = kConvBwdCh, blk = 16 / int64_t(elem_size(dt));
    const int64_t cblocks = (dim + ch - 1) / ch, tblocks = (L + blk - 1) / blk;
    ConvBwdParams p{};
    p.batch = int(batch);
    p.dim = int(dim);
    p.L = int(L);
    p.cg_log2 = channel_blocks_log2(xt ? (yt ? 5 : 4) : (yt ? 4 : 0), cblocks, tblocks);
    p.ctiles = int((cblocks + (1 << p.cg_log2) - 1) >> p.cg_log2);
    const int ngr = 32 >> p.cg_log2;
    const int64_t tiles = (tblocks + ngr - 1) / ngr;
    // Runs: the fewest steps in sequence, with whole waves of blocks (five per
    // SM) and about half a step for a run's start and the W-1 tokens above it.
    p.across = p.cg_log2 <= 4;
    const int64_t per_run = p.across ? (p.ctiles + 3) / 4 * batch : int64_t(p.ctiles) * batch;
    const auto blocks_of = [&](int64_t r) { return p.across ? per_run * r : per_run * ((r + 3) / 4); };
    double best = 1e300;
    int64_t runs = 1;
    for (int64_t r = 1; r <= std::min<int64_t>(tiles, 256); ++r) {
        const int64_t steps = (tiles + r - 1) / r, rr = (tiles + steps - 1) / steps;
        const double waves = double((blocks_of(rr) + 5 * di->sm_count - 1) / (5 * di->sm_count));
        const double t = waves * (double(steps) + 0.5);
        if (t < best * 0.999) {
            best = t;
            runs = rr;
        }
    }
    p.steps = int((tiles + runs - 1) / runs);
    p.runs = int(runs);
    p.x = view_of(x, xt);
    p.dy = view_of(dy, yt);
    p.dx = view_of(dx, xt);
    p.weight = static_cast<const float *>(weight->data);
    p.bias = static_cast<const float *>(opt_data(bias));
    p.h0 = opt_data(h0);
    p.dlast = opt_data(dlast);
    p.dh0 = dh0 ? dh0->data : nullptr;
    p.silu = silu ? 1 : 0;
    const int64_t gx = blocks_of(runs) / batch;
    const int64_t rows = batch * runs;
    if (gx > 0x7fffffffll || rows > 0x7fffffffll || dim * (W + 1) > 0x7fffffffll)
        return SELSCAN_ERR_UNSUPPORTED;
    void *ws = nullptr;
    if (scratch_alloc(&ws, size_t(rows) * size_t(dim * (W + 1)) * 4, stream) != cudaSuccess)
        return SELSCAN_ERR_CUDA;
    p.part = static_cast<float *>(ws);
    const dim3 grid{unsigned(gx), unsigned(batch)};
    cudaError_t le = cudaSuccess;
    dispatch(dt, W, [&](auto tag, auto w) {
        constexpr int WW = decltype(w)::value;
        launch_conv_bwd<decltype(tag), WW>(p, xt, yt, grid, stream);
        if ((le = counted_launch()) != cudaSuccess)
            return;
        conv_bwd_sum_kernel<WW><<<unsigned((dim * (W + 1) + 31) / 32), 256, 0, stream>>>(
            p.part, int(rows), int(dim), static_cast<float *>(dweight->data),
            dbias ? static_cast<float *>(dbias->data) : nullptr);
        le = counted_launch();
    });
    cudaFreeAsync(ws, stream);
    return le == cudaSuccess ? SELSCAN_OK : SELSCAN_ERR_CUDA;
}

extern "C" selscan_status selscan_conv_step(selscan_tensor *state, const selscan_tensor *slots,
                                            const selscan_tensor *x, const selscan_tensor *weight,
                                            const selscan_tensor *bias, int silu,
                                            selscan_tensor *y, cudaStream_t stream)
{
    if (!present(state) || !present(x) || !weight || !present(y))
        return SELSCAN_ERR_NULL;
    if (x->ndim != 2 || state->ndim != 3)
        return SELSCAN_ERR_SHAPE;
    const int32_t dt = x->dtype;
    if (dt != SELSCAN_F32 && dt != SELSCAN_BF16)
        return SELSCAN_ERR_DTYPE;
    const int64_t batch = x->shape[0], dim = x->shape[1];
    if (batch < 0 || dim < 0 || state->shape[0] < 0)
        return SELSCAN_ERR_SHAPE;
    selscan_status st;
    int64_t W = 0;
    if ((st = check_tok(x, batch, dim, dt)) != SELSCAN_OK) return st;
    if ((st = check_tok(y, batch, dim, dt)) != SELSCAN_OK) return st;
    if ((st = check_taps(weight, bias, dim, &W)) != SELSCAN_OK) return st;
    const int64_t count = slots ? state->shape[0] : batch;
    if (slots && (st = check_index(slots, batch, false)) != SELSCAN_OK) return st;
    const int64_t sshape[3] = {count, dim, W - 1};
    if ((st = check_state(state, 3, sshape, dt, false)) != SELSCAN_OK) return st;
    if ((batch > 1 && y->stride[0] == 0) || (dim > 1 && y->stride[1] == 0))
        return SELSCAN_ERR_STRIDE;
    if (W < 2 || W > 4 || batch > 65535 || dim > kMaxDim || count > 0x7fffffffll)
        return SELSCAN_ERR_UNSUPPORTED;
    if (batch == 0 || dim == 0)
        return SELSCAN_OK;

    ConvStepParams p{};
    int dev = 0;
    DeviceInfo *di = nullptr;
    if ((st = device_setup(&dev, &di)) != SELSCAN_OK)
        return st;
    const int64_t sms = di->sm_count;
    if (slots) {
        p.slots = static_cast<const int *>(slots->data);
        p.err = di->err;
    }
    const int64_t es = int64_t(elem_size(dt)), blk = 16 / es;
    const auto vec_ok = [&](const selscan_tensor *t) {
        return (dim == 1 || t->stride[1] == 1) && rows_vec(t, es);
    };
    p.vec = dim % blk == 0 && vec_ok(x) && vec_ok(y) && aligned16(state->data);
    p.wvec = aligned16(weight->data);
    p.batch = int(batch);
    p.dim = int(dim);
    p.x = x->data;
    p.sx0 = x->stride[0];
    p.sx1 = x->stride[1];
    p.y = y->data;
    p.sy0 = y->stride[0];
    p.sy1 = y->stride[1];
    p.weight = static_cast<const float *>(weight->data);
    p.bias = static_cast<const float *>(opt_data(bias));
    p.state = state->data;
    p.slot_count = int(count);
    p.silu = silu ? 1 : 0;
    const int64_t threads = p.vec ? dim / blk : dim;
    const int64_t gx = (threads + 127) / 128;
    p.rows = conv_step_rows(batch, gx, sms);
    const dim3 grid{unsigned(gx), unsigned((batch + p.rows - 1) / p.rows)};
    dispatch(dt, W, [&](auto tag, auto w) {
        using T = decltype(tag);
        constexpr int WW = decltype(w)::value;
        p.vec ? conv_step_kernel<T, WW, true><<<grid, 128, 0, stream>>>(p)
              : conv_step_kernel<T, WW, false><<<grid, 128, 0, stream>>>(p);
    });
    return counted_launch() == cudaSuccess ? SELSCAN_OK : SELSCAN_ERR_CUDA;
}

extern "C" selscan_status selscan_conv_packed(selscan_tensor *state, const selscan_tensor *x,
                                              const selscan_tensor *weight,
                                              const selscan_tensor *bias, int silu,
                                              const selscan_tensor *start,
                                              const selscan_tensor *slots,
                                              const selscan_tensor *seen, selscan_tensor *y,
                                              cudaStream_t stream)
{
    if (!present(state) || !present(x) || !weight || !present(y))
        return SELSCAN_ERR_NULL;
    if (x->ndim != 2 || state->ndim != 3)
        return SELSCAN_ERR_SHAPE;
    const int32_t dt = x->dtype;
    if (dt != SELSCAN_F32 && dt != SELSCAN_BF16)
        return SELSCAN_ERR_DTYPE;
    const int64_t tokens = x->shape[0], dim = x->shape[1];
    if (tokens < 0 || dim < 0 || state->shape[0] < 0)
        return SELSCAN_ERR_SHAPE;
    selscan_status st;
    int64_t W = 0;
    if ((st = check_rows(x, tokens, dim, dt, false)) != SELSCAN_OK) return st;
    if ((st = check_rows(y, tokens, dim, dt, true)) != SELSCAN_OK) return st;
    if ((st = check_taps(weight, bias, dim, &W)) != SELSCAN_OK) return st;
    const int64_t sshape[3] = {state->shape[0], dim, W - 1};
    if ((st = check_state(state, 3, sshape, dt, false)) != SELSCAN_OK) return st;
    ConvPackedParams p{};
    if ((st = check_packed(state, start, slots, seen, tokens, &p.ix)) != SELSCAN_OK) return st;
    if (W < 2 || W > 4 || dim > kMaxDim)
        return SELSCAN_ERR_UNSUPPORTED;
    if (dim == 0 || p.ix.seqs == 0)
        return SELSCAN_OK;

    int dev = 0;
    DeviceInfo *di = nullptr;
    if ((st = device_setup(&dev, &di)) != SELSCAN_OK)
        return st;
    p.ix.err = di->err;
    const int64_t es = int64_t(elem_size(dt)), blk = 16 / es;
    p.vec = dim % blk == 0 && rows_vec(x, es) && rows_vec(y, es);
    p.svec = p.vec && aligned16(state->data);
    p.dim = int(dim);
    p.x = x->data;
    p.sx = x->stride[0];
    p.y = y->data;
    p.sy = y->stride[0];
    p.weight = static_cast<const float *>(weight->data);
    p.bias = static_cast<const float *>(opt_data(bias));
    p.state = state->data;
    p.silu = silu ? 1 : 0;
    const int64_t per = 32 * (p.vec ? blk : 4);
    p.ctiles = int((dim + per - 1) / per);
    p.subs = conv_packed_subs(tokens, p.ctiles, di->sm_count);
    p.runs = int((tokens + p.subs * kConvRun - 1) / (p.subs * kConvRun));
    const int64_t blocks = (int64_t(p.runs) + 1 + 3) / 4 * p.ctiles;
    if (blocks > 0x7fffffffll)
        return SELSCAN_ERR_UNSUPPORTED;
    dispatch(dt, W, [&](auto tag, auto w) {
        using T = decltype(tag);
        constexpr int WW = decltype(w)::value;
        p.vec ? conv_packed_kernel<T, WW, true><<<unsigned(blocks), 128, 0, stream>>>(p)
              : conv_packed_kernel<T, WW, false><<<unsigned(blocks), 128, 0, stream>>>(p);
    });
    return counted_launch() == cudaSuccess ? SELSCAN_OK : SELSCAN_ERR_CUDA;
}

extern "C" long long selscan_debug_packed_piece(const selscan_tensor *t)
{
    return packed_piece_bytes(t);
}

extern "C" void selscan_debug_packed_segment(int tokens, int lanes)
{
    g_dbg_packed_seg = tokens <= 0 ? 0 : (tokens + 15) / 16 * 16;
    g_dbg_packed_lanes = lanes == 1 || lanes == 4 || lanes == -4 || lanes == 8 ? lanes : 0;
}

extern "C" selscan_status selscan_fwd_packed(
    selscan_tensor *state, const selscan_tensor *u, const selscan_tensor *delta,
    const selscan_tensor *delta_bias, int delta_softplus, const selscan_tensor *A,
    const selscan_tensor *B, const selscan_tensor *C, const selscan_tensor *D,
    const selscan_tensor *z, const selscan_tensor *start, const selscan_tensor *slots,
    const selscan_tensor *seen, selscan_tensor *y, cudaStream_t stream)
{
    if (!present(state) || !present(u) || !present(A) || !present(y))
        return SELSCAN_ERR_NULL;
    if (u->ndim != 2 || A->ndim != 2 || state->ndim != 3)
        return SELSCAN_ERR_SHAPE;
    const int32_t dt = u->dtype;
    if (dt != SELSCAN_F32 && dt != SELSCAN_BF16)
        return SELSCAN_ERR_DTYPE;
    const int64_t tokens = u->shape[0], dim = u->shape[1], N = A->shape[1];
    if (tokens < 0 || dim < 0 || state->shape[0] < 0 || A->shape[0] != dim)
        return SELSCAN_ERR_SHAPE;
    selscan_status st;
    if ((st = check_rows(u, tokens, dim, dt, false)) != SELSCAN_OK) return st;
    if ((st = check_rows(delta, tokens, dim, dt, false)) != SELSCAN_OK) return st;
    const bool gate = z && (z->data || tokens == 0);
    if (z && !z->data && tokens > 0 && dim > 0)
        return SELSCAN_ERR_NULL;
    if (gate && (st = check_rows(z, tokens, dim, dt, false)) != SELSCAN_OK) return st;
    if ((st = check_rows(B, tokens, N, dt, false)) != SELSCAN_OK) return st;
    if ((st = check_rows(C, tokens, N, dt, false)) != SELSCAN_OK) return st;
    if ((st = check_rows(y, tokens, dim, dt, true)) != SELSCAN_OK) return st;
    {
        const int64_t ashape[2] = {dim, N}, vshape[1] = {dim};
        if ((st = check_param(A, 2, ashape, false)) != SELSCAN_OK) return st;
        if ((st = check_param(delta_bias, 1, vshape, true)) != SELSCAN_OK) return st;
        if ((st = check_param(D, 1, vshape, true)) != SELSCAN_OK) return st;
        const int64_t sshape[3] = {state->shape[0], dim, N};
        if ((st = check_param(state, 3, sshape, false)) != SELSCAN_OK) return st;
    }
    if (!aligned16(A->data) || !aligned16(state->data))
        return SELSCAN_ERR_ALIGN;
    ScanPackedParams p{};
    if ((st = check_packed(state, start, slots, seen, tokens, &p.ix)) != SELSCAN_OK) return st;
    if (N != kDiagN || dim > kMaxDim / kDiagN)
        return SELSCAN_ERR_UNSUPPORTED;
    if (dim == 0 || p.ix.seqs == 0)
        return SELSCAN_OK;

    int dev = 0;
    DeviceInfo *di = nullptr;
    if ((st = device_setup(&dev, &di)) != SELSCAN_OK)
        return st;
    p.ix.err = di->err;
    const int64_t es = int64_t(elem_size(dt));
    p.dim = int(dim);
    p.vec = rows_vec(u, es) && rows_vec(delta, es) && (!gate || rows_vec(z, es));
    p.bc_vec = packed_piece_bytes(B) && packed_piece_bytes(C);
    p.u = u->data;
    p.su = u->stride[0];
    p.delta = delta->data;
    p.sd = delta->stride[0];
    p.z = gate ? z->data : nullptr;
    p.sz = gate ? z->stride[0] : 0;
    p.B = B->data;
    p.sB = B->stride[0];
    p.C = C->data;
    p.sC = C->stride[0];
    p.y = y->data;
    p.sy = y->stride[0];
    p.A = static_cast<const float *>(A->data);
    p.delta_bias = static_cast<const float *>(opt_data(delta_bias));
    p.Dskip = static_cast<const float *>(opt_data(D));
    p.state = static_cast<float *>(state->data);
    p.softplus = delta_softplus ? 1 : 0;

    p.y_vec = reinterpret_cast<uintptr_t>(y->data) % uintptr_t(2 * es) == 0 &&
              (tokens <= 1 || y->stride[0] % 2 == 0);
    const PackedPlan plan = packed_plan(tokens, p.ix.seqs, dim, di->sm_count);
    const int64_t ct = plan.lanes == 8 ? 32 : 64;
    p.tiles = int((dim + ct - 1) / ct);
    p.seg_len = plan.seg_len;
    const int64_t units = tokens / p.seg_len + p.ix.seqs;
    if (units * p.tiles > 0x7fffffffll)
        return SELSCAN_ERR_UNSUPPORTED;
    const unsigned grid = unsigned(units * p.tiles);
    const bool bf = dt == SELSCAN_BF16;
    void *ws = nullptr;
    cudaError_t le = cudaSuccess;
    if (tokens > p.seg_len) {  // some sequence may have several segments
        const size_t entries = 2 * size_t(tokens / p.seg_len) + 2;
        if (scratch_alloc(&ws, entries * size_t(dim) * (kDiagN + 1) * 4, stream) != cudaSuccess)
            return SELSCAN_ERR_CUDA;
        p.agg = static_cast<float *>(ws);
        p.agg_sd = p.agg + entries * size_t(dim) * kDiagN;
    }
    p.lead = ws && plan.lead;
    if (ws)
        le = launch_packed<true>(p, bf, plan.lanes, grid, stream);
    if (ws && le == cudaSuccess && tokens > 2 * int64_t(p.seg_len)) {
        const dim3 fg{unsigned((dim * kDiagN + 255) / 256), unsigned(p.ix.seqs)};
        scan_packed_fold_kernel<<<fg, 256, 0, stream>>>(p);
        le = counted_launch();
    }
    if (le == cudaSuccess)
        le = launch_packed<false>(p, bf, plan.lanes, grid, stream);
    if (ws)
        cudaFreeAsync(ws, stream);
    return le == cudaSuccess ? SELSCAN_OK : SELSCAN_ERR_CUDA;
}
