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
