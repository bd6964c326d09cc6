"""GPU parity of the operators on packed prompts and slotted caches
(selscan_fwd_packed, selscan_conv_packed, selscan_step with slots) with plain
fp64 numpy, sequence by sequence, and their runs together as a serving loop and
a training layer make them.

Tolerances: those of the dense scan's tests for y and the states, relative L2
(fp32 1e-5; bf16 y 5e-3: rounding to bf16 is off by at most 2^-8 = 3.9e-3 of
each value, the rest is left for fp32 arithmetic; fp32 states 1e-5), and per
element for the convolution (one bf16 rounding, 2^-8, over fp32 arithmetic,
2^-20 of the sum of absolute terms)."""
import numpy as np
import pytest

import plain_layer
import synthetic

pytestmark = pytest.mark.gpu

N = 16


def rel(a, b):
    a, b = np.asarray(a, np.float64), np.asarray(b, np.float64)
    return float(np.linalg.norm(a - b) / max(np.linalg.norm(b), 1e-30))


def rnd(rng, *shape, dtype="f32", scale=1.0):
    a = (scale * rng.standard_normal(shape)).astype(np.float32)
    return synthetic.round_bf16(a) if dtype == "bf16" else a


def dev(a, dtype="f32"):
    import torch
    if a is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(a))
    return t.to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()


def i32(a):
    import torch
    return torch.from_numpy(np.asarray(a, np.int32)).cuda()


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


class Packed:
    """A packed batch: lengths, starts, slots of a cache, tokens seen."""

    def __init__(self, rng, lens, tail=0, lead=0):
        self.lens = list(lens)
        self.start = lead + np.concatenate([[0], np.cumsum(lens)])
        self.tokens = int(self.start[-1]) + tail
        self.count = len(lens) + 3
        self.slots = rng.permutation(self.count)[:len(lens)]
        self.seen = rng.integers(0, 2, len(lens)) * 7
        self.owned = np.zeros(self.tokens, bool)
        self.owned[self.start[0]:self.start[-1]] = True

    def args(self):
        return i32(self.start), i32(self.slots)

    def each(self):
        for i in range(len(self.lens)):
            yield i, slice(int(self.start[i]), int(self.start[i + 1])), int(self.slots[i])


def scan_inputs(rng, T, D, dtype, real=False):
    step = np.exp(rng.uniform(np.log(1e-3), np.log(1e-1), D))
    A = np.tile(-np.arange(1, N + 1, dtype=np.float32), (D, 1))
    if not real:
        A = (A * np.exp(0.3 * rng.standard_normal((D, N)))).astype(np.float32)
    return dict(u=rnd(rng, T, D, dtype=dtype), delta=rnd(rng, T, D, dtype=dtype, scale=0.5),
                z=rnd(rng, T, D, dtype=dtype), B=rnd(rng, T, N, dtype=dtype),
                C=rnd(rng, T, N, dtype=dtype), A=A, D=rnd(rng, D),
                delta_bias=np.log(np.expm1(step)).astype(np.float32))


def scan_reference(pk, inp, state0, y0, gate=True, seen=True, **kw):
    y, state = y0.astype(np.float64), state0.astype(np.float64)
    for i, rows, slot in pk.each():
        h0 = state[slot] if (not seen or pk.seen[i]) else None
        y[rows], state[slot] = plain_layer.scan(
            inp["u"][rows], inp["delta"][rows], inp["A"], inp["B"][rows], inp["C"][rows],
            D=inp["D"], z=inp["z"][rows] if gate else None, delta_bias=inp["delta_bias"], h0=h0,
            **kw)
    return y, state


def scan_call(pk, inp, state, out, dtype, gate=True, seen=True, **kw):
    import selective_state_space_selscan_b200 as ss
    g = {k: dev(inp[k], dtype if k in ("u", "delta", "z", "B", "C") else "f32") for k in inp}
    return ss.selscan_fwd_packed(state, g["u"], g["delta"], g["A"], g["B"], g["C"], *pk.args(),
                                 D=g["D"], z=g["z"] if gate else None,
                                 delta_bias=g["delta_bias"],
                                 seen=i32(pk.seen) if seen else None, out=out, **kw)


LENGTHS = [  # sequences of a batch
    [1], [17], [1, 1, 1], [0, 5, 0, 0, 3, 0], [16, 32, 64], [7, 130, 1, 65, 2, 0, 40],
    [300, 2, 70], [1] * 40, [63, 64, 65, 127, 128, 129], [700],
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 200, 7])
def test_scan_packed_matches_plain(dtype, D):
    import selective_state_space_selscan_b200 as ss
    rng = np.random.default_rng(20)
    for j, lens in enumerate(LENGTHS):
        pk = Packed(rng, lens, tail=3 * (j % 2), lead=2 * (j % 3))
        gate, real, seen = j % 4 != 3, j % 2 == 0, j % 3 != 2
        inp = scan_inputs(rng, pk.tokens, D, dtype, real)
        state0 = rnd(rng, pk.count, D, N)
        y0 = rnd(rng, pk.tokens, D, dtype=dtype)
        y_ref, s_ref = scan_reference(pk, inp, state0, y0, gate, seen)
        state, out = dev(state0), dev(y0, dtype)
        y = scan_call(pk, inp, state, out, dtype, gate, seen)
        ss.check()
        assert y is out
        got, st = host(y), host(state)
        assert np.array_equal(got[~pk.owned], y0[~pk.owned]), lens  # rows of no sequence
        others = [s for s in range(pk.count) if s not in pk.slots]
        assert np.array_equal(st[others], state0[others]), lens
        for i, rows, slot in pk.each():
            assert rel(st[slot], s_ref[slot]) <= 1e-5, (lens, i)
            if rows.stop > rows.start:
                assert rel(got[rows], y_ref[rows]) <= (1e-5 if dtype == "f32" else 5e-3), (lens, i)


@pytest.mark.parametrize("lanes", [1, 4, -4, 8])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scan_packed_forms(lanes, dtype):
    """All splits of a channel's states over lanes, in segments of 16 to 48
    tokens, with A of every kind: powers, general, partly positive, wide
    (decays that underflow)."""
    import selective_state_space_selscan_b200 as ss
    rng = np.random.default_rng(33)
    D = 136
    try:
        for j, (seg, lens) in enumerate([(16, [100, 3, 33]), (32, [64, 0, 65, 1]), (48, [200]),
                                         (0, [37, 5])]):
            ss.debug_packed_segment(seg, lanes)
            for kind in ("real", "free", "positive", "wide"):
                pk = Packed(rng, lens, tail=j)
                inp = scan_inputs(rng, pk.tokens, D, dtype, kind == "real")
                if kind == "positive":
                    inp["A"][::3, ::5] *= -0.5
                if kind == "wide":
                    inp["A"] *= 100.0
                    inp["delta"][::7] += 12.0
                    inp["delta"] = synthetic.round_bf16(inp["delta"])
                state0, y0 = rnd(rng, pk.count, D, N), rnd(rng, pk.tokens, D, dtype=dtype)
                y_ref, s_ref = scan_reference(pk, inp, state0, y0, gate=j != 1)
                state, out = dev(state0), dev(y0, dtype)
                scan_call(pk, inp, state, out, dtype, gate=j != 1)
                ss.check()
                for i, rows, slot in pk.each():
                    # A positive A grows a state by exp(sum delta A): past 3e38
                    # it leaves fp32, and the exponents' sum X carries a
                    # relative error of X 2^-23.  Up to 1e4, X < 10 and that
                    # is about 1e-6; larger states, and the outputs of their
                    # channels, are not compared.
                    small = np.abs(s_ref[slot]) <= 1e4
                    chan = small.all(1)
                    assert kind == "positive" or small.all()
                    assert chan.sum() >= D // 2
                    assert rel(host(state)[slot][small], s_ref[slot][small]) <= 1e-5, (seg, kind, i)
                    if rows.stop > rows.start:
                        err = rel(host(out)[rows][:, chan], y_ref[rows][:, chan])
                        assert err <= (1e-5 if dtype == "f32" else 5e-3), (seg, kind, i)
    finally:
        ss.debug_packed_segment(0)


def test_scan_packed_many_segments():
    """One long prompt among short ones, few channels: tens of segments per
    sequence, folded between two passes."""
    import selective_state_space_selscan_b200 as ss
    rng = np.random.default_rng(21)
    for dtype, D, lens in (("f32", 32, [9000, 5, 3000]), ("bf16", 160, [1, 12000, 64, 0, 900])):
        pk = Packed(rng, lens)
        inp = scan_inputs(rng, pk.tokens, D, dtype, real=dtype == "bf16")
        state0, y0 = rnd(rng, pk.count, D, N), rnd(rng, pk.tokens, D, dtype=dtype)
        y_ref, s_ref = scan_reference(pk, inp, state0, y0)
        state, out = dev(state0), dev(y0, dtype)
        scan_call(pk, inp, state, out, dtype)
        ss.check()
        for i, rows, slot in pk.each():
            assert rel(host(state)[slot], s_ref[slot]) <= 1e-5, (dtype, i)
            if rows.stop > rows.start:
                assert rel(host(out)[rows], y_ref[rows]) <= (1e-5 if dtype == "f32" else 5e-3)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,lens", [
    (2040, [1500, 100, 2, 900, 0, 430, 700, 1300, 64, 65, 350, 800, 1000, 1, 600, 385]),
    (1100, [21000, 2, 5800]),
    (1100, [26000]),
])
def test_scan_packed_fills_the_gpu(D, lens, dtype):
    """Sizes whose automatic split takes first segments' outputs in the first
    pass, and long prompts with one lane per channel, several and alone; the
    first and last channels and two in between against fp64."""
    import selective_state_space_selscan_b200 as ss
    rng = np.random.default_rng(len(lens))
    pk = Packed(rng, lens, tail=3, lead=1)
    inp = scan_inputs(rng, pk.tokens, D, dtype, real=len(lens) == 3)
    state0, y0 = rnd(rng, pk.count, D, N), rnd(rng, pk.tokens, D, dtype=dtype)
    ch = np.array([0, 1, 63, 64, D // 2, D - 2, D - 1])
    part = {k: v if k in "BC" else v[ch] if k in ("A", "D", "delta_bias") else v[:, ch]
            for k, v in inp.items()}
    y_ref, s_ref = scan_reference(pk, part, state0[:, ch], y0[:, ch])
    state, out = dev(state0), dev(y0, dtype)
    scan_call(pk, inp, state, out, dtype)
    ss.check()
    st, y = host(state)[:, ch], host(out)
    assert np.array_equal(y[~pk.owned], y0[~pk.owned].astype(np.float64))
    for i, rows, slot in pk.each():
        assert rel(st[slot], s_ref[slot]) <= 1e-5, i
        if rows.stop > rows.start:
            assert rel(y[rows][:, ch], y_ref[rows]) <= (1e-5 if dtype == "f32" else 5e-3), i


def test_scan_packed_without_options_and_strided():
    """No bias, D, gate, softplus (negative steps too); operands as column
    slices of wider rows, at odd offsets as well."""
    import torch
    import selective_state_space_selscan_b200 as ss
    rng = np.random.default_rng(22)
    D = 72
    for dtype in ("f32", "bf16"):
        for pad in (0, 1, 8):
            pk = Packed(rng, [20, 1, 90])
            inp = scan_inputs(rng, pk.tokens, D, dtype)
            inp["delta"] = np.abs(inp["delta"]) * 0.1
            inp["delta"] = synthetic.round_bf16(inp["delta"].astype(np.float32)) \
                if dtype == "bf16" else inp["delta"]
            state0 = rnd(rng, pk.count, D, N)
            y_ref, s_ref = np.zeros((pk.tokens, D)), state0.astype(np.float64)
            for i, rows, slot in pk.each():
                y_ref[rows], s_ref[slot] = plain_layer.scan(
                    inp["u"][rows], inp["delta"][rows], inp["A"], inp["B"][rows],
                    inp["C"][rows], softplus=False, h0=s_ref[slot])

            def cols(a):
                t = torch.full((pk.tokens, 2 * a.shape[1] + pad), float("nan"), device="cuda",
                               dtype=torch.bfloat16 if dtype == "bf16" else torch.float32)
                t[:, pad:pad + a.shape[1]] = dev(a, dtype)
                return t[:, pad:pad + a.shape[1]]

            state = dev(state0)
            out = cols(np.zeros((pk.tokens, D), np.float32))
            ss.selscan_fwd_packed(state, cols(inp["u"]), cols(inp["delta"]), dev(inp["A"]),
                                  cols(inp["B"]), cols(inp["C"]), *pk.args(),
                                  delta_softplus=False, out=out)
            ss.check()
            assert rel(host(state)[pk.slots], s_ref[pk.slots]) <= 1e-5
            assert rel(host(out), y_ref) <= (1e-5 if dtype == "f32" else 5e-3)


def test_scan_packed_keeps_nan_to_its_sequence_and_channel():
    import torch
    import selective_state_space_selscan_b200 as ss
    rng = np.random.default_rng(23)
    D = 40
    pk = Packed(rng, [30, 50, 20])
    for dtype in ("f32", "bf16"):
        inp = scan_inputs(rng, pk.tokens, D, dtype)
        state0 = rnd(rng, pk.count, D, N)
        a_state, b_state = dev(state0), dev(state0)
        a = scan_call(pk, inp, a_state, None, dtype)
        inp["u"][45, 3] = np.nan
        b = scan_call(pk, inp, b_state, None, dtype)
        ss.check()
        hit = torch.zeros(pk.tokens, D, dtype=torch.bool, device="cuda")
        hit[45:80, 3] = True
        assert torch.equal(a[~hit], b[~hit]) and b[hit].isnan().all()
        keep = torch.ones_like(a_state, dtype=torch.bool)
        keep[int(pk.slots[1]), 3] = False
        assert torch.equal(a_state[keep], b_state[keep])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 512, 200, 7])
def test_conv_packed_matches_plain(dtype, D):
    import selective_state_space_selscan_b200 as ss
    rng = np.random.default_rng(24)
    for j, lens in enumerate(LENGTHS + [[2] * 9, [3, 1, 2, 3, 1], [8, 8, 7, 1, 9]]):
        W = (4, 3, 2)[j % 3]
        pk = Packed(rng, lens, tail=3 * (j % 2), lead=2 * (j % 3))
        x, w, bias = rnd(rng, pk.tokens, D, dtype=dtype), rnd(rng, D, W), rnd(rng, D)
        st0 = rnd(rng, pk.count, D, W - 1, dtype=dtype)
        y0 = rnd(rng, pk.tokens, D, dtype=dtype)
        seen = j % 3 != 2
        state, out = dev(st0, dtype), dev(y0, dtype)
        ss.selscan_conv_packed(state, dev(x, dtype), dev(w), *pk.args(), bias=dev(bias),
                               seen=i32(pk.seen) if seen else None, out=out)
        ss.check()
        got, st = host(out), host(state)
        want = st0.astype(np.float64)
        assert np.array_equal(got[~pk.owned], y0[~pk.owned])
        for i, rows, slot in pk.each():
            h0 = want[slot] if (not seen or pk.seen[i]) else None
            ref, last, size = plain_layer.conv(x[rows].T, w, bias, True, h0)
            want[slot] = last
            tol = (2.0 ** -8 if dtype == "bf16" else 0) * np.abs(ref) + 2.0 ** -20 * (size + np.abs(ref))
            assert (np.abs(got[rows].T - ref) <= tol).all(), (lens, W, i)
        assert np.array_equal(st, want), (lens, W)


def test_packed_operators_skip_and_refuse_on_the_device():
    """Padding sequences (negative slots) are skipped; a slot twice, a slot past
    the cache, and rows outside the buffer are refused, reported by check(), and
    nothing of them is written; the other sequences are computed."""
    import torch
    import selective_state_space_selscan_b200 as ss
    rng = np.random.default_rng(25)
    D, lens = 136, [10, 30, 5, 200]
    base = Packed(rng, lens)
    inp = scan_inputs(rng, base.tokens, D, "f32")
    x, w = inp["u"], rnd(rng, D, 4)
    state0, cst0 = rnd(rng, 6, D, N), rnd(rng, 6, D, 3)
    y0 = rnd(rng, base.tokens, D)
    start = list(base.start)
    cases = [  # slots, starts, sequences left out, whether check() reports
        ([0, -1, 2, 3], start, {1}, False),
        ([-1, -1, -1, -2], start, {0, 1, 2, 3}, False),
        ([0, 1, 0, 3], start, {2}, True),
        ([0, 6, 2, 3], start, {1}, True),
        ([0, 1, 2, 2 ** 31 - 1], start, {3}, True),
        ([0, 1, 2, 3], start[:4] + [base.tokens + 1], {3}, True),
        ([0, 1, 2, 3], [-1] + start[1:], {0}, True),
    ]
    for slots, st, out_of, reports in cases:
        pk = Packed(rng, lens)
        pk.slots, pk.start, pk.seen = np.array(slots), np.array(st), np.array([1, 1, 0, 1])
        for conv in (False, True):
            out = dev(y0)
            state = dev(cst0 if conv else state0)
            if conv:
                ss.selscan_conv_packed(state, dev(x), dev(w), *pk.args(), seen=i32(pk.seen), out=out)
            else:
                scan_call(pk, inp, state, out, "f32")
            if reports:
                with pytest.raises(ss.SelscanError, match="SELSCAN_ERR_INDEX"):
                    ss.check()
            ss.check()
            got, sg = host(out), host(state)
            want = (cst0 if conv else state0).astype(np.float64)
            for i in range(4):
                rows = slice(max(0, int(base.start[i])), int(base.start[i + 1]))
                if i in out_of:
                    assert np.array_equal(got[rows], y0[rows]), (slots, st, conv)
                    continue
                h0 = want[slots[i]] if pk.seen[i] else None
                if conv:
                    ref, last, _ = plain_layer.conv(x[rows].T, w, None, True, h0)
                    ref = ref.T
                else:
                    ref, last = plain_layer.scan(
                        inp["u"][rows], inp["delta"][rows], inp["A"], inp["B"][rows],
                        inp["C"][rows], D=inp["D"], z=inp["z"][rows],
                        delta_bias=inp["delta_bias"], h0=h0)
                assert rel(got[rows], ref) <= 1e-5, (slots, st, conv)
                want[slots[i]] = last
            assert rel(sg, want) <= 1e-5
            kept = [s for s in range(6) if s not in [slots[i] for i in range(4) if i not in out_of]]
            assert np.array_equal(sg[kept], (cst0 if conv else state0)[kept])


def test_packed_starts_in_disorder_stay_inside():
    """Starts that go back, or lie far outside, are reported and touch nothing
    outside the buffers (guard rows around y and the state)."""
    import torch
    import selective_state_space_selscan_b200 as ss
    rng = np.random.default_rng(26)
    D, T = 128, 600
    inp = scan_inputs(rng, T, D, "bf16")
    w = rnd(rng, D, 4)
    for start in ([0, 500, 100, 600], [600, 0, 0, 600], [0, 2 ** 31 - 1, -2 ** 31, 600],
                  [-2 ** 31, -5, 700, 2 ** 31 - 1], [300, 200, 100, 0]):
        pk = Packed(rng, [1, 1, 1])
        pk.start, pk.slots, pk.seen = np.array(start), np.array([0, 1, 2]), np.array([1, 0, 1])
        for conv in (False, True):
            buf = torch.full((T + 64, D), 3.0, dtype=torch.bfloat16, device="cuda")
            if conv:
                cache = torch.full((5, D, 3), 3.0, dtype=torch.bfloat16, device="cuda")
                ss.selscan_conv_packed(cache[1:4], dev(inp["u"], "bf16"), dev(w), *pk.args(),
                                       seen=i32(pk.seen), out=buf[32:T + 32])
            else:
                cache = torch.full((5, D, N), 3.0, device="cuda")
                scan_call(pk, inp, cache[1:4], buf[32:T + 32], "bf16")
            with pytest.raises(ss.SelscanError, match="SELSCAN_ERR_INDEX"):
                ss.check()
            assert (buf[:32] == 3).all() and (buf[T + 32:] == 3).all()
            assert (cache[0] == 3).all() and (cache[4] == 3).all()


# ------------------------------------------------ decode step through slots
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scalar", [False, True])
def test_step_with_slots_equals_the_gathered_step(dtype, scalar):
    """Row by row the same kernel arithmetic as selscan_step on the gathered
    states: bit for bit; untouched slots and padding rows stay."""
    import torch
    import selective_state_space_selscan_b200 as ss
    rng = np.random.default_rng(27)
    for batch, dim, NS in ((1, 64, 16), (5, 192, 32), (300, 64, 16), (40, 128, 128)):
        count = batch + batch // 2 + 1
        slots = rng.permutation(count)[:batch].astype(np.int32)
        padded = rng.random(batch) < 0.2
        slots[padded] = -1
        live = np.flatnonzero(~padded)
        A = -np.abs(rnd(rng, dim // 64)) if scalar else -np.abs(rnd(rng, dim, NS))
        x, z = (dev(rnd(rng, batch, dim, dtype=dtype), dtype) for _ in range(2))
        B, C = (dev(rnd(rng, batch, NS, dtype=dtype), dtype) for _ in range(2))
        units = dim // 64 if scalar else dim
        dt = dev(rnd(rng, batch, units, dtype=dtype), "f32" if scalar else dtype)
        shape = (count, dim // 64, 64, NS) if scalar else (count, dim, NS)
        cache = dev(rnd(rng, *shape))
        before = cache.clone()
        Dv, bias = dev(rnd(rng, units)), dev(rnd(rng, units))
        out = torch.full_like(x, 9.0)

        def step(state, r, **kw):
            if scalar:
                return ss.selscan_step_scalarA(state, x[r], dt[r], dev(A), B[r], C[r], 64, D=Dv,
                                               z=z[r], dt_bias=bias, dt_softplus=True, **kw)
            return ss.selscan_step(state, x[r], dt[r], dev(A), B[r], C[r], D=Dv, z=z[r],
                                   delta_bias=bias, **kw)

        y = step(cache, slice(None), slots=i32(slots), out=out)
        ss.check()
        assert y is out and (out[torch.from_numpy(padded).cuda()] == 9).all()
        if len(live):
            rows = torch.from_numpy(live).cuda()
            at = torch.from_numpy(slots[live].astype(np.int64)).cuda()
            part = before[at].contiguous()
            ref = step(part, rows)
            assert torch.equal(out[rows], ref) and torch.equal(cache[at], part)
            before[at] = part
        assert torch.equal(cache, before)


def test_step_refuses_slots_on_the_device():
    import torch
    import selective_state_space_selscan_b200 as ss
    rng = np.random.default_rng(28)
    D = 520
    A = dev(-np.abs(rnd(rng, D, N)))
    x, B = dev(rnd(rng, 4, D)), dev(rnd(rng, 4, N))
    for bad, skipped in (([0, 1, 0, 2], 2), ([0, 3, 1, 2], 1)):
        cache = dev(rnd(rng, 3, D, N))
        keep = [i for i in range(4) if i != skipped]
        at = torch.tensor([bad[i] for i in keep], device="cuda")
        part = cache[at].contiguous()
        out = torch.full((4, D), 9.0, device="cuda")
        ss.selscan_step(cache, x, x, A, B, B, slots=i32(bad), out=out)
        with pytest.raises(ss.SelscanError, match="SELSCAN_ERR_INDEX"):
            ss.check()
        ref = ss.selscan_step(part, x[keep], x[keep], A, B[keep], B[keep])
        ss.check()
        assert (out[skipped] == 9).all() and torch.equal(out[keep], ref)
        assert torch.equal(cache[at], part)


# ------------------------------------------------------- as they are used
def test_many_sequences():
    """More sequences than one probe of a warp sees (32) and more than its
    square, single tokens among them."""
    import selective_state_space_selscan_b200 as ss
    rng = np.random.default_rng(36)
    D = 24
    for count in (33, 200, 1500):
        lens = rng.integers(0, 4, count)
        lens[rng.integers(0, count, 3)] = 90
        pk = Packed(rng, lens, tail=2)
        inp = scan_inputs(rng, pk.tokens, D, "f32")
        x, w = inp["u"], rnd(rng, D, 4)
        state0, cst0 = rnd(rng, pk.count, D, N), rnd(rng, pk.count, D, 3)
        y0 = np.zeros((pk.tokens, D), np.float32)
        y_ref, s_ref = scan_reference(pk, inp, state0, y0)
        state, out = dev(state0), dev(y0)
        scan_call(pk, inp, state, out, "f32")
        cst, yc = dev(cst0), dev(y0)
        ss.selscan_conv_packed(cst, dev(x), dev(w), *pk.args(), seen=i32(pk.seen), out=yc)
        ss.check()
        assert rel(host(out), y_ref) <= 1e-5 and rel(host(state), s_ref) <= 1e-5
        c_ref, st_ref = np.zeros_like(y_ref), cst0.astype(np.float64)
        for i, rows, slot in pk.each():
            y, st_ref[slot], _ = plain_layer.conv(x[rows].T, w, None, True,
                                                  st_ref[slot] if pk.seen[i] else None)
            c_ref[rows] = y.T
        assert rel(host(yc), c_ref) <= 1e-5 and np.array_equal(host(cst), st_ref)


def test_packed_calls_in_two_graphs():
    """Two captured graphs of the same calls (each with its own scratch in the
    capture), replayed in turn with new inputs, equal the eager calls."""
    import torch
    import selective_state_space_selscan_b200 as ss
    rng = np.random.default_rng(29)
    D = 128
    pk = Packed(rng, [900, 1, 3000, 40])
    inp = scan_inputs(rng, pk.tokens, D, "bf16")
    g = {k: dev(inp[k], "bf16" if k in ("u", "delta", "z", "B", "C") else "f32") for k in inp}
    w = dev(rnd(rng, D, 4))
    start, slots = pk.args()
    cache0, conv0 = dev(rnd(rng, pk.count, D, N)), dev(rnd(rng, pk.count, D, 3, dtype="bf16"), "bf16")
    tok = dev(rnd(rng, 4, D, dtype="bf16"), "bf16")
    tb = dev(rnd(rng, 4, N, dtype="bf16"), "bf16")

    def calls(x, cache, conv):
        y = ss.selscan_conv_packed(conv, x, w, start, slots)
        y = ss.selscan_fwd_packed(cache, y, g["delta"], g["A"], g["B"], g["C"], start, slots,
                                  D=g["D"], z=g["z"], delta_bias=g["delta_bias"])
        v = ss.selscan_conv_step(conv, tok, w, slots=slots)
        return y, ss.selscan_step(cache, v, tok, g["A"], tb, tb, slots=slots)

    graphs = []
    for i in range(2):
        x, cache, conv = g["u"].clone(), cache0.clone(), conv0.clone()
        calls(x, cache, conv)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            y, v = calls(x, cache, conv)
        graphs.append((gr, x, cache, conv, y, v))
    for k in range(3):
        for gr, x, cache, conv, y, v in graphs:
            x.copy_(torch.randn_like(x))
            cache.copy_(cache0)
            conv.copy_(conv0)
            gr.replay()
            c2, k2 = cache0.clone(), conv0.clone()
            y2, v2 = calls(x, c2, k2)
            torch.cuda.synchronize()
            assert torch.equal(y, y2) and torch.equal(v, v2)
            assert torch.equal(cache, c2) and torch.equal(conv, k2)
    ss.check()


def test_both_bindings_make_the_same_calls(monkeypatch):
    """The C++ binding and the ctypes one, on every entry point they share."""
    import torch
    import selective_state_space_selscan_b200 as ss
    rng = np.random.default_rng(37)
    D = 64
    pk = Packed(rng, [9, 70, 1])
    inp = scan_inputs(rng, pk.tokens, D, "bf16")
    x, w, b = dev(rnd(rng, 2, D, 50)), dev(rnd(rng, D, 4)), dev(rnd(rng, D))
    h0, tok, bc = dev(rnd(rng, 2, D, 3)), dev(rnd(rng, 2, D)), dev(rnd(rng, 2, N))
    dt = dev(rnd(rng, 2, 1))
    bc128 = dev(rnd(rng, 2, 128))
    assert ss._binding(), "_bind.so is not built"
    results = []
    for bind in (ss._binding(), False):
        monkeypatch.setattr(ss, "_bound", bind)
        rng = np.random.default_rng(38)
        state, conv = dev(rnd(rng, pk.count, D, N)), dev(rnd(rng, pk.count, D, 3))
        scal = dev(rnd(rng, 4, 1, 64, 128))
        out = [scan_call(pk, inp, state, None, "bf16"), *ss.selscan_conv(x, w, bias=b, h0=h0)]
        g = ss.selscan_conv_bwd(x, w, x, bias=b, h0=h0, dlast=h0)
        out += [g[k] for k in ("dx", "dweight", "dbias", "dh0")]
        out.append(ss.selscan_conv_packed(conv, dev(inp["u"]), w, *pk.args(), bias=b,
                                          seen=i32(pk.seen)))
        out.append(ss.selscan_conv_step(conv, tok, w, slots=i32([1, 0]),
                                        stream=torch.cuda.current_stream()))
        out.append(ss.selscan_step(state, tok, tok, dev(inp["A"]), bc, bc, D=b, slots=i32([0, 2])))
        out.append(ss.selscan_step_scalarA(scal, tok, dt, -b[:1].abs(), bc128, bc128, 64, D=b[:1],
                                           z=tok, dt_bias=b[:1], dt_softplus=True,
                                           slots=i32([3, 1])))
        ss.check()
        results.append(out + [state, conv, scal])
    for a, c in zip(*results):
        assert torch.equal(a, c)


@pytest.mark.parametrize("which", ["conv_bwd", "packed", "step"])
def test_first_call_inside_a_capture(which):
    """In a fresh process the library's first call on a device, which makes
    its scratch pool, may be a captured one."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = f"""
import sys
sys.path.insert(0, {root!r})
import torch
import selective_state_space_selscan_b200 as ss
r = lambda *s: torch.randn(*s, device="cuda")
i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
x, w, A, cache, bc = r(2, 64, 40), r(64, 4), -r(64, 16).abs(), r(3, 64, 16), r(2000, 16)
t, start, slots, row = r(2000, 64), i(0, 1900, 2000), i(0, 2), r(2, 64)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    if {which!r} == "conv_bwd":
        ss.selscan_conv_bwd(x, w, x)
    elif {which!r} == "packed":
        ss.selscan_fwd_packed(cache, t, t, A, bc, bc, start, slots)
    else:
        ss.selscan_step(cache, row, row, A, bc[:2], bc[:2], slots=slots)
g.replay()
ss.check()
print("captured")
"""
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert "captured" in out.stdout, out.stdout + out.stderr


def test_rows_of_no_sequence_may_hold_anything():
    """NaN in the rows behind the last sequence and before the first, in slots
    that no sequence owns, and in the state of a sequence that starts from
    zero, reaches nothing."""
    import torch
    import selective_state_space_selscan_b200 as ss
    rng = np.random.default_rng(34)
    D = 136
    for dtype in ("f32", "bf16"):
        for lens in ([5, 0, 40], [0, 0], [300, 1]):
            pk = Packed(rng, lens, tail=9, lead=6)
            pk.seen = np.array([0, 3, 0][:len(lens)])
            inp = scan_inputs(rng, pk.tokens, D, dtype)
            state0 = rnd(rng, pk.count, D, N)
            y0 = rnd(rng, pk.tokens, D, dtype=dtype)
            w = rnd(rng, D, 4)
            cst0 = rnd(rng, pk.count, D, 3, dtype=dtype)
            results = []
            for bad in (0.0, np.nan):
                x = {k: v.copy() for k, v in inp.items()}
                for k in ("u", "delta", "z", "B", "C"):
                    x[k][~pk.owned] = bad
                st, cst = state0.copy(), cst0.copy()
                loose = [s for s in range(pk.count)
                         if s not in pk.slots or pk.seen[list(pk.slots).index(s)] == 0]
                st[loose] = bad
                cst[loose] = bad
                state, conv, out, yc = dev(st), dev(cst, dtype), dev(y0, dtype), dev(y0, dtype)
                scan_call(pk, x, state, out, dtype)
                ss.selscan_conv_packed(conv, dev(x["u"], dtype), dev(w), *pk.args(),
                                       seen=i32(pk.seen), out=yc)
                ss.check()
                at = torch.from_numpy(pk.slots.astype(np.int64)).cuda()
                results.append((out, yc, state[at], conv[at]))
            for a, b in zip(*results):
                assert torch.equal(a, b)


def test_no_rows_at_all():
    """Sequences without rows: states stay, or are zeroed where nothing was
    seen."""
    import torch
    import selective_state_space_selscan_b200 as ss
    rng = np.random.default_rng(35)
    D = 40
    for dtype in ("f32", "bf16"):
        empty = dev(np.zeros((0, D), np.float32), dtype)
        bc = dev(np.zeros((0, N), np.float32), dtype)
        state0, conv0 = rnd(rng, 4, D, N), rnd(rng, 4, D, 3, dtype=dtype)
        state, conv = dev(state0), dev(conv0, dtype)
        start, slots, seen = i32([0, 0, 0]), i32([2, 0]), i32([0, 4])
        y = ss.selscan_fwd_packed(state, empty, empty, dev(-np.ones((D, N), np.float32)), bc, bc,
                                  start, slots, seen=seen)
        yc = ss.selscan_conv_packed(conv, empty, dev(rnd(rng, D, 4)), start, slots, seen=seen)
        ss.check()
        assert y.shape == yc.shape == (0, D)
        state0[2], conv0[2] = 0, 0
        assert np.array_equal(host(state), state0) and np.array_equal(host(conv), conv0)


def test_serving_loop_equals_the_whole_sequences():
    """Prefill in chunks of unequal lengths mixed with single tokens, then
    decode steps, through one cache, against the plain layer (convolution, then
    scan, with B, C and the step size given per token) over whole sequences."""
    import torch
    import selective_state_space_selscan_b200 as ss
    rng = np.random.default_rng(30)
    D, dtype = 96, "f32"
    total = [57, 131, 9, 64]
    slots = [3, 0, 4, 1]
    seqs = [scan_inputs(rng, n, D, dtype) for n in total]
    for s in seqs:
        s.update({k: seqs[0][k] for k in ("A", "D", "delta_bias")})
    w, bias = rnd(rng, D, 4), rnd(rng, D)
    refs = []
    for s in seqs:
        x, _, _ = plain_layer.conv(s["u"].T, w, bias)
        refs.append(plain_layer.scan(x.T, s["delta"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"],
                                     delta_bias=s["delta_bias"]))
    cache = torch.full((6, D, N), 5.0, device="cuda")  # stale: the first chunk starts from zero
    conv = torch.full((6, D, 3), 5.0, device="cuda")
    A, Dv, db = dev(seqs[0]["A"]), dev(seqs[0]["D"]), dev(seqs[0]["delta_bias"])
    done, got = [0] * 4, [[] for _ in total]
    for chunk in ([20, 3, 0, 64], [1, 100, 2, 0], [30, 1, 1, 0], [1, 20, 1, 0]):
        part = {k: np.concatenate([seqs[i][k][done[i]:done[i] + n] for i, n in enumerate(chunk)])
                for k in ("u", "delta", "z", "B", "C")}
        start = i32(np.concatenate([[0], np.cumsum(chunk)]))
        at, seen = i32(slots), i32(done)
        x = ss.selscan_conv_packed(conv, dev(part["u"]), dev(w), start, at, bias=dev(bias), seen=seen)
        y = ss.selscan_fwd_packed(cache, x, dev(part["delta"]), A, dev(part["B"]), dev(part["C"]),
                                  start, at, D=Dv, z=dev(part["z"]), delta_bias=db, seen=seen)
        off = 0
        for i, n in enumerate(chunk):
            got[i].append(host(y[off:off + n]))
            off += n
            done[i] += n
    while any(d < n for d, n in zip(done, total)):
        row = [i for i in range(4) if done[i] < total[i]]
        tok = {k: np.stack([seqs[i][k][done[i]] for i in row]) for k in ("u", "delta", "z", "B", "C")}
        at = i32([slots[i] for i in row] + [-1, -1])  # a padded batch
        tok = {k: dev(np.concatenate([v, np.zeros((2, v.shape[1]), np.float32)])) for k, v in tok.items()}
        x = ss.selscan_conv_step(conv, tok["u"], dev(w), bias=dev(bias), slots=at,
                                 out=torch.zeros_like(tok["u"]))
        y = ss.selscan_step(cache, x, tok["delta"], A, tok["B"], tok["C"], D=Dv, z=tok["z"],
                            delta_bias=db, slots=at, out=torch.zeros_like(x))
        for j, i in enumerate(row):
            got[i].append(host(y[j:j + 1]))
            done[i] += 1
    ss.check()
    for i, (y_ref, h_ref) in enumerate(refs):
        assert rel(np.concatenate(got[i]), y_ref) <= 1e-5, i
        assert rel(host(cache[slots[i]]), h_ref) <= 1e-5, i


def test_training_layer_gradients():
    """Projection half (token-major) -> convolution -> channels-first scan, and
    back through both, against torch's own differentiation of the plain layer
    in fp64.  fp32 throughout: relative L2 1e-4 as in the scan's gradient
    tests (fp32 sums over all tokens)."""
    import torch
    import selective_state_space_selscan_b200 as ss
    rng = np.random.default_rng(31)
    b, D, L = 2, 48, 120
    f = lambda *s, scale=1.0: torch.from_numpy(rnd(rng, *s, scale=scale)).cuda()
    xz, w, bias = f(b, L, 2 * D), f(D, 4), f(D)
    delta, B, C, Dv = f(b, D, L, scale=0.5), f(b, N, L), f(b, N, L), f(D)
    A = -torch.exp(f(D, N, scale=0.3))
    dy = f(b, D, L)
    x, z = xz[..., :D].transpose(1, 2), xz[..., D:].transpose(1, 2).contiguous()
    u, _ = ss.selscan_conv(x, w, bias=bias)
    y, _ = ss.selscan_fwd(u, delta, A, B, C, D=Dv, z=z)
    gs = ss.selscan_bwd(u, delta, A, B, C, dy, D=Dv, z=z)
    gxz = torch.zeros_like(xz)
    gc = ss.selscan_conv_bwd(x, w, gs["du"], bias=bias, dx=gxz[..., :D].transpose(1, 2))
    ss.check()

    p = {k: v.double().detach().clone().requires_grad_() for k, v in
         dict(xz=xz, w=w, bias=bias, delta=delta, A=A, B=B, C=C, D=Dv).items()}
    xx = torch.nn.functional.pad(p["xz"][..., :D].transpose(1, 2), (3, 0))
    v = sum(p["w"][:, k:k + 1] * xx[..., k:k + L] for k in range(4)) + p["bias"][:, None]
    uu = v * torch.sigmoid(v)
    d = torch.nn.functional.softplus(p["delta"])
    h, ys = torch.zeros(b, D, N, dtype=torch.float64, device="cuda"), []
    for t in range(L):
        h = torch.exp(d[:, :, t, None] * p["A"]) * h + (d * uu)[:, :, t, None] * p["B"][:, None, :, t]
        ys.append((h * p["C"][:, None, :, t]).sum(-1))
    yy = (torch.stack(ys, -1) + p["D"][:, None] * uu) * torch.nn.functional.silu(
        p["xz"][..., D:].transpose(1, 2))
    yy.backward(dy.double())
    assert rel(host(y), host(yy)) <= 1e-5
    gxz[..., D:] = gs["dz"].transpose(1, 2)
    for name, got, ref in (("xz", gxz, p["xz"]), ("w", gc["dweight"], p["w"]),
                           ("bias", gc["dbias"], p["bias"]), ("delta", gs["ddelta"], p["delta"]),
                           ("A", gs["dA"], p["A"]), ("B", gs["dB"], p["B"])):
        assert rel(host(got), host(ref.grad)) <= 1e-4, name
