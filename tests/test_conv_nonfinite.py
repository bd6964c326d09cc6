"""Infinities and NaN in the convolution's operands reach the outputs, states
and gradients that the formula gives them to, and no others.

Tolerances, per element, those of the convolution's other tests: one rounding to
bf16 (2^-8) of the outputs in x's type; fp32 arithmetic, 2^-20 of the sum of
absolute terms for outputs, twice that for gradients; and n 2^-24 of it for sums
over n terms."""
import numpy as np
import pytest

import plain_layer
import selective_state_space_selscan_b200 as ss
from test_packed import dev, host, rnd

pytestmark = pytest.mark.gpu


def same(got, want, tol, what):
    """NaN and infinities where the reference has them, the rest within tol."""
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), what
    ok = np.isfinite(want)
    assert (np.abs(got - want)[ok] <= tol[ok]).all(), what


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tokens_first", [False, True])
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("value", [np.inf, np.nan])
def test_conv_gradients(value, silu, tokens_first, dtype):
    """One bad input at the end, in the middle and at the start of a channel's
    sequence: without SiLU the taps that do not meet it keep their gradients."""
    rng = np.random.default_rng(80)
    D = 24
    for W in (2, 3, 4):
        for L in (1, 2, 7, 8, 64, 101):
            x, dy = rnd(rng, 2, D, L, dtype=dtype), rnd(rng, 2, D, L, dtype=dtype)
            w, bias = rnd(rng, D, W), rnd(rng, D)
            for c, t in ((3, L - 1), (6, L - 2), (10, L - W + 1), (13, L // 2), (17, 0)):
                x[0, c, max(0, t)] = value
            with np.errstate(invalid="ignore"):
                ref = plain_layer.conv_grads(x, w, dy, bias, silu)
                y_ref, last, size = plain_layer.conv(x, w, bias, silu)
            xt = dev(x.transpose(0, 2, 1), dtype).transpose(1, 2) if tokens_first else dev(x, dtype)
            got = ss.selscan_conv_bwd(xt, dev(w), dev(dy, dtype), bias=dev(bias), silu=silu)
            y, _ = ss.selscan_conv(xt, dev(w), bias=dev(bias), silu=silu)
            ss.check()
            eps = 2.0 ** -8 if dtype == "bf16" else 0.0
            what, n = (W, L), (2 * L + 16) * 2.0 ** -24 + 2.0 ** -19
            with np.errstate(invalid="ignore"):
                same(host(got["dx"]), ref["dx"],
                     eps * np.abs(ref["dx"]) + 2.0 ** -19 * ref["dxsize"], what)
                same(host(got["dweight"]), ref["dweight"], n * ref["dwsize"], what)
                same(host(got["dbias"]), ref["dbias"], n * ref["dbsize"], what)
                if np.isnan(value):  # torch and numpy differ on inf * sigmoid(-inf)
                    same(host(y), y_ref, eps * np.abs(y_ref) + 2.0 ** -20 * (size + np.abs(y_ref)),
                         what)
