"""Padding sequences of a packed batch whose starts go back (a buffer of zeros
behind the live ones) can hide live sequences from the search for a row's owner:
such a call is reported, a padded batch in order is not and is right.

Tolerance: relative L2 1e-5 for fp32, as in the packed operators' other tests."""
import numpy as np
import pytest

import plain_layer
import selective_state_space_selscan_b200 as ss
from test_packed import N, Packed, dev, host, i32, rel, rnd, scan_inputs, scan_reference

pytestmark = pytest.mark.gpu


def batch(rng, pads):
    """Two live sequences of rows [0, 10) and [10, 40), then ``pads`` padding
    ones."""
    pk = Packed(rng, [10, 30])
    pk.starts = np.concatenate([pk.start, np.full(pads, pk.start[-1])])
    pk.all_slots = np.concatenate([pk.slots, np.full(pads, -1)])
    pk.seen_all = np.concatenate([pk.seen, np.zeros(pads, int)])
    return pk


def call(conv, pk, inp, w, state, out):
    start, slots, seen = i32(pk.starts), i32(pk.all_slots), i32(pk.seen_all)
    if conv:
        return ss.selscan_conv_packed(state, dev(inp["u"]), dev(w), start, slots, seen=seen, out=out)
    g = {k: dev(v) for k, v in inp.items()}
    return ss.selscan_fwd_packed(state, g["u"], g["delta"], g["A"], g["B"], g["C"], start, slots,
                                 D=g["D"], z=g["z"], delta_bias=g["delta_bias"], seen=seen, out=out)


@pytest.mark.parametrize("conv", [False, True])
@pytest.mark.parametrize("pads", [3, 60])
def test_starts_of_padding_that_go_back_are_reported(conv, pads):
    rng = np.random.default_rng(70)
    D = 40
    pk = batch(rng, pads)
    inp, w = scan_inputs(rng, pk.tokens, D, "f32"), rnd(rng, D, 4)
    state0 = rnd(rng, pk.count, D, 3) if conv else rnd(rng, pk.count, D, N)
    y0 = rnd(rng, pk.tokens, D)
    for first in (3, 4, len(pk.starts) - 2):
        # the starts from here on are zero; the last one begins no sequence
        keep = pk.starts.copy()
        pk.starts[first:] = 0
        call(conv, pk, inp, w, dev(state0), dev(y0))
        with pytest.raises(ss.SelscanError, match="SELSCAN_ERR_INDEX"):
            ss.check()
        pk.starts = keep


@pytest.mark.parametrize("conv", [False, True])
@pytest.mark.parametrize("pads", [1, 3, 60])
@pytest.mark.parametrize("end", [40, 0])
def test_padded_batches_in_order(conv, pads, end):
    """``end``: the start behind the last sequence, which is padding."""
    rng = np.random.default_rng(71)
    D = 40
    pk = batch(rng, pads)
    pk.starts[-1] = end
    inp, w = scan_inputs(rng, pk.tokens, D, "f32"), rnd(rng, D, 4)
    state0 = rnd(rng, pk.count, D, 3) if conv else rnd(rng, pk.count, D, N)
    y0 = rnd(rng, pk.tokens, D)
    state, out = dev(state0), dev(y0)
    call(conv, pk, inp, w, state, out)
    ss.check()
    if conv:
        y_ref, s_ref = y0.astype(np.float64), state0.astype(np.float64)
        for i, rows, slot in pk.each():
            y, s_ref[slot], _ = plain_layer.conv(inp["u"][rows].T, w, None, True,
                                                 s_ref[slot] if pk.seen[i] else None)
            y_ref[rows] = y.T
    else:
        y_ref, s_ref = scan_reference(pk, inp, state0, y0)
    assert rel(host(out), y_ref) <= 1e-5 and rel(host(state), s_ref) <= 1e-5
