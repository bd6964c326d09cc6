"""B and C of packed prompts as slices of a projection, at every alignment that
a slice can have: the scan's inner pieces are loads of several values, which
need their whole size as alignment.

The CPU test asks the library which loads it would make.  The GPU test's
tolerances are those of the packed scan's other tests: relative L2, fp32 1e-5;
bf16 y 5e-3 (one rounding of each value by at most 2^-8 = 3.9e-3 of it, the rest
for fp32 arithmetic), states 1e-5."""
import numpy as np
import pytest

import plain_layer
import selective_state_space_selscan_b200 as ss
from test_packed import N, Packed, dev, host, i32, rel, rnd, scan_inputs

FAKE = 0x7f0000000000
SIZE = {ss.SELSCAN_F32: 4, ss.SELSCAN_BF16: 2}


@pytest.mark.parametrize("dtype", list(SIZE))
def test_pieces_of_b_and_c_are_aligned(dtype):
    """For every offset and row stride: the loads' size divides every row's
    address, and rows that are aligned to four values are read in pieces."""
    es = SIZE[dtype]
    for offset in range(17):
        for extra in range(17):
            for tokens in (1, 2, 300):
                data, stride = FAKE + offset * es, 2 * N + extra
                t = ss._DESC.pack(data, dtype, 2, tokens, N, 0, 0, stride, 1, 0, 0)
                piece = ss.debug_packed_piece(t)
                rows = [data + r * stride * es for r in range(min(tokens, 5))]
                assert piece in (0, 4 * es)
                if piece:
                    assert all(a % piece == 0 for a in rows), (offset, extra, tokens)
                assert bool(piece) == all(a % (4 * es) == 0 for a in rows)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lanes", [0, 1, 4, -4, 8])
def test_scan_packed_slices_of_a_projection(lanes, dtype):
    """B and C behind R columns of a (tokens, R + 2 N + tail) projection, its
    rows 4, 8 or 16 bytes from a whole piece; one, two and more segments."""
    import torch
    rng = np.random.default_rng(50)
    D = 40
    tt = torch.bfloat16 if dtype == "bf16" else torch.float32
    pk = Packed(rng, [5, 1, 70, 33])
    inp = scan_inputs(rng, pk.tokens, D, dtype)
    state0 = rnd(rng, pk.count, D, N)
    y_ref, s_ref = np.zeros((pk.tokens, D)), state0.astype(np.float64)
    for i, rows, slot in pk.each():
        y_ref[rows], s_ref[slot] = plain_layer.scan(
            inp["u"][rows], inp["delta"][rows], inp["A"], inp["B"][rows], inp["C"][rows],
            delta_bias=inp["delta_bias"], h0=s_ref[slot])
    try:
        for seg in (0, 16, 48) if lanes else (0,):
            ss.debug_packed_segment(seg, lanes)
            for first, tail in ((0, 0), (2, 0), (6, 0), (4, 0), (0, 2), (2, 2), (6, 2), (4, 6),
                                (1, 0), (1, 3)):
                proj = torch.full((pk.tokens, first + 2 * N + tail), float("nan"), device="cuda",
                                  dtype=tt)
                B, C = proj[:, first:first + N], proj[:, first + N:first + 2 * N]
                B.copy_(dev(inp["B"], dtype))
                C.copy_(dev(inp["C"], dtype))
                state = dev(state0)
                y = ss.selscan_fwd_packed(state, dev(inp["u"], dtype), dev(inp["delta"], dtype),
                                          dev(inp["A"]), B, C, *pk.args(),
                                          delta_bias=dev(inp["delta_bias"]))
                ss.check()
                assert rel(host(state)[pk.slots], s_ref[pk.slots]) <= 1e-5, (seg, first, tail)
                assert rel(host(y), y_ref) <= (1e-5 if dtype == "f32" else 5e-3), (seg, first, tail)
    finally:
        ss.debug_packed_segment(0)
