"""Infinities, NaN and overflow in scans of packed prompts: what they reach is
what the formula says, whatever form and number of segments the call takes.

Tolerances: those of the packed scan's other tests, relative L2 over the finite
values (fp32 1e-5, bf16 y 5e-3, states 1e-5)."""
import numpy as np
import pytest

import selective_state_space_selscan_b200 as ss
from test_packed import N, Packed, dev, host, rel, rnd, scan_call, scan_inputs, scan_reference

pytestmark = pytest.mark.gpu

# tokens per segment and lanes per channel: the library's own choice, and every
# form with sequences of one, two, three and more segments
FORMS = [(0, 0)] + [(seg, lanes) for lanes in (1, 4, -4, 8) for seg in (16, 32, 112)]


def same(got, want, tol, what):
    """NaN and infinities where the reference has them, the rest within tol."""
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), what
    ok = np.isfinite(want)
    assert rel(got[ok], want[ok]) <= tol, what


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("real", [False, True])
def test_infinite_decay_rates_reset_the_state(dtype, real):
    """A = -inf (exp of a large log): every token starts its state anew, and the
    tokens that fill up a sequence's last chunk leave it alone."""
    rng = np.random.default_rng(60)
    D = 40
    pk = Packed(rng, [5, 1, 100, 33], tail=3)
    inp = scan_inputs(rng, pk.tokens, D, dtype, real)
    inp["A"][3, :] = -np.inf
    inp["A"][17, 5] = -np.inf
    inp["A"][18, 9:] = -np.inf
    state0, y0 = rnd(rng, pk.count, D, N), rnd(rng, pk.tokens, D, dtype=dtype)
    y_ref, s_ref = scan_reference(pk, inp, state0, y0)
    assert np.isfinite(y_ref).all() and np.isfinite(s_ref).all()
    try:
        for form in FORMS:
            ss.debug_packed_segment(*form)
            state, out = dev(state0), dev(y0, dtype)
            scan_call(pk, inp, state, out, dtype)
            ss.check()
            same(host(state), s_ref, 1e-5, form)
            same(host(out), y_ref, 1e-5 if dtype == "f32" else 5e-3, form)
    finally:
        ss.debug_packed_segment(0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("where", ["u", "delta", "z", "B", "C", "A", "D", "delta_bias", "state"])
def test_nan_reaches_what_it_should(where, dtype):
    """One NaN in an operand, in sequences of one and more segments: the outputs
    and states that the fp64 form makes NaN, and no others."""
    rng = np.random.default_rng(61)
    D = 40
    pk = Packed(rng, [5, 30, 100, 1], tail=3)
    pk.seen[:] = 7
    inp = scan_inputs(rng, pk.tokens, D, dtype)
    state0, y0 = rnd(rng, pk.count, D, N), rnd(rng, pk.tokens, D, dtype=dtype)
    for at in (0, 17, 96):  # a token in the first, an inner and the last segment
        bad, st = {k: v.copy() for k, v in inp.items()}, state0.copy()
        for i in (1, 2):
            t = int(pk.start[i]) + min(at, pk.lens[i] - 1)
            if where in ("u", "delta", "z"):
                bad[where][t, 21 + i] = np.nan
            elif where in ("B", "C"):
                bad[where][t, 9 + i] = np.nan
            elif where == "A":
                bad[where][21 + i, at % N] = np.nan
            elif where == "state":
                st[pk.slots[i], 21 + i, at % N] = np.nan
            else:
                bad[where][21 + i] = np.nan
        y_ref, s_ref = scan_reference(pk, bad, st, y0)
        assert np.isnan(y_ref).any()
        try:
            for form in FORMS:
                ss.debug_packed_segment(*form)
                state, out = dev(st), dev(y0, dtype)
                scan_call(pk, bad, state, out, dtype)
                ss.check()
                same(host(state), s_ref, 1e-5, (where, at, form))
                same(host(out), y_ref, 1e-5 if dtype == "f32" else 5e-3, (where, at, form))
        finally:
            ss.debug_packed_segment(0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decays_up_to_the_largest_number(dtype):
    """Positive A: exp(delta A) up to 2^128 is a number, from there infinity.

    One step takes a state of 1e-30 to exp(x) of it, and zero steps keep it.  The
    exponent x = 2 A goes through A log2 e (constant and product) and the product
    with the step, 1.3e-8 + 2 x 2^-24 = 1.4e-7 of it at most, so exp(x) is off by
    1.4e-7 x of itself, and by 2^-20 for the exponential and the products."""
    rng = np.random.default_rng(62)
    x = np.array([60.0, 87.0, 87.9, 88.3, 88.6, 88.7, 88.8, 89.0, 95.0, 120.0, 1e4, np.inf])
    D = len(x)
    pk = Packed(rng, [1, 20, 60])
    pk.seen[:] = 1
    zero = np.zeros((pk.tokens, D), np.float32)
    inp = dict(u=zero, delta=zero.copy(), B=rnd(rng, pk.tokens, N, dtype=dtype),
               C=rnd(rng, pk.tokens, N, dtype=dtype), z=zero, D=np.zeros(D, np.float32),
               A=np.repeat((x / 2).astype(np.float32)[:, None], N, 1),
               delta_bias=np.zeros(D, np.float32))
    inp["delta"][pk.start[:-1]] = 2.0
    state0 = (1e-30 * (1 + np.abs(rng.standard_normal((pk.count, D, N))))).astype(np.float32)
    e = np.float64(2) * inp["A"][:, 0]
    big = e >= 128 * np.log(2)
    assert big.sum() == 6 and not (np.abs(e - 128 * np.log(2)) < 1e-2).any()
    finite = np.isfinite(e)  # exp(0 A) is NaN where A is infinite
    try:
        for form in FORMS:
            ss.debug_packed_segment(*form)
            state = dev(state0)
            scan_call(pk, inp, state, None, dtype, gate=False, delta_softplus=False)
            ss.check()
            got = host(state)
            for i, rows, slot in pk.each():
                if pk.lens[i] > 1:
                    assert np.isnan(got[slot][~finite]).all(), (form, i)
                else:
                    assert np.isinf(got[slot][~finite]).all(), (form, i)
                assert np.isposinf(got[slot][big & finite]).all(), (form, i)
                want = state0[slot].astype(np.float64)[~big] * np.exp(e[~big])[:, None]
                off = np.abs(got[slot][~big] / want - 1)
                assert (off <= (1.4e-7 * e[~big] + 2.0 ** -20)[:, None]).all(), (form, i, off.max())
    finally:
        ss.debug_packed_segment(0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_growing_decays_leave_an_empty_state_empty(dtype):
    """A = +1 and a sum of steps of about 96 per segment of 48 tokens, whose
    exponential is infinite: the state of a fresh sequence is zero until its first
    input, in the last segment, and a number from there."""
    rng = np.random.default_rng(63)
    D = 40
    pk = Packed(rng, [200, 3, 240])
    pk.seen[:] = 0
    inp = scan_inputs(rng, pk.tokens, D, dtype)
    inp["A"][::2, ::3] = 1.0
    inp["delta"][:] = 2.0
    inp["delta_bias"][:] = 0.0
    for i in (0, 2):
        inp["u"][pk.start[i]:pk.start[i + 1] - 6] = 0
    state0, y0 = rnd(rng, pk.count, D, N), rnd(rng, pk.tokens, D, dtype=dtype)
    y_ref, s_ref = scan_reference(pk, inp, state0, y0, softplus=False)
    assert np.isfinite(s_ref).all()
    try:
        for lanes in (1, 4, -4, 8):
            ss.debug_packed_segment(48, lanes)
            state, out = dev(state0), dev(y0, dtype)
            scan_call(pk, inp, state, out, dtype, delta_softplus=False)
            ss.check()
            same(host(state), s_ref, 1e-5, lanes)
            same(host(out), y_ref, 1e-5 if dtype == "f32" else 5e-3, lanes)
    finally:
        ss.debug_packed_segment(0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_steps_forget_large_states(dtype):
    """A step of delta |A| >= 100 leaves nothing of a state of 1e36 (exp(-100) of
    it is 4e-8, and from 104 on the decay is zero in fp32): the state is the step's
    own input, whichever form the call takes."""
    rng = np.random.default_rng(64)
    D = 40
    pk = Packed(rng, [1, 60, 33])
    pk.seen[:] = 1
    inp = scan_inputs(rng, pk.tokens, D, dtype)
    inp["A"] = np.repeat(np.linspace(-110, -4000, D, dtype=np.float32)[:, None], N, 1)
    inp["delta"][:], inp["delta_bias"][:] = 1.0, 0.0
    inp["B"] = np.where(np.abs(inp["B"]) < 0.25, np.float32(0.5), inp["B"])
    inp["u"] = np.where(np.abs(inp["u"]) < 0.25, np.float32(0.5), inp["u"])
    state0 = (1e36 * (1 + rng.random((pk.count, D, N)))).astype(np.float32)
    try:
        for form in FORMS:
            ss.debug_packed_segment(*form)
            state = dev(state0)
            scan_call(pk, inp, state, None, dtype, delta_softplus=False)
            ss.check()
            for i, rows, slot in pk.each():
                t = rows.stop - 1
                want = inp["u"][t].astype(np.float64)[:, None] * inp["B"][t].astype(np.float64)
                off = np.abs(host(state)[slot] - want)
                # what is left of the state after the one step of the first sequence
                kept = np.abs(state0[slot].astype(np.float64)) * np.exp(inp["A"].astype(np.float64))
                assert (off <= 2.0 ** -22 * np.abs(want) + kept).all(), (form, i, off.max())
    finally:
        ss.debug_packed_segment(0)
