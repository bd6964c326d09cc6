"""Offsets past 2^32 elements: rows of packed prompts in a buffer of long rows,
and slots far inside large caches, for every operator that reads through them.

Tolerances: those of the packed operators' other tests, relative L2 (bf16 y 5e-3,
fp32 states 1e-5; the convolution's bf16 y one rounding, 2^-8)."""
import numpy as np
import pytest

import plain_layer
import selective_state_space_selscan_b200 as ss
from test_packed import N, Packed, dev, host, i32, rel, rnd, scan_inputs

pytestmark = pytest.mark.gpu

D = 64


@pytest.fixture
def room():
    import torch
    if torch.cuda.mem_get_info()[0] < 48 << 30:
        pytest.skip("needs 48 GB of device memory")
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("seg", [0, 16])
def test_far_rows_and_far_slots(room, seg):
    import torch
    rng = np.random.default_rng(90)
    pk = Packed(rng, [34, 1, 0, 1])
    pk.seen[:] = [3, 0, 0, 2]
    pitch = 1 << 27
    count = (1 << 22) + 8
    pk.slots = np.array([count - 1, (1 << 21) + 1, 5, count - 7])
    inp = scan_inputs(rng, pk.tokens, D, "bf16")
    assert (pk.tokens - 1) * pitch > 1 << 32 and (count - 7) * D * N > 1 << 32
    buf = torch.empty(pk.tokens, pitch, dtype=torch.bfloat16, device="cuda")
    cols = {}
    for j, k in enumerate(("u", "delta", "z", "B", "C")):
        cols[k] = buf[:, j * 72:j * 72 + inp[k].shape[1]]
        cols[k].copy_(dev(inp[k], "bf16"))
    out = buf[:, 400:400 + D]
    cache = torch.empty(count, D, N, device="cuda")
    state0 = {int(s): rnd(rng, D, N) for s in pk.slots}
    for s, v in state0.items():
        cache[s] = dev(v)
    y_ref, s_ref = np.zeros((pk.tokens, D)), {}
    for i, rows, slot in pk.each():
        h0 = state0[slot] if pk.seen[i] else None
        y_ref[rows], s_ref[slot] = plain_layer.scan(
            inp["u"][rows], inp["delta"][rows], inp["A"], inp["B"][rows], inp["C"][rows],
            D=inp["D"], z=inp["z"][rows], delta_bias=inp["delta_bias"], h0=h0)
    try:
        ss.debug_packed_segment(seg, 4 if seg else 0)
        ss.selscan_fwd_packed(cache, cols["u"], cols["delta"], dev(inp["A"]), cols["B"], cols["C"],
                              *pk.args(), D=dev(inp["D"]), z=cols["z"],
                              delta_bias=dev(inp["delta_bias"]), seen=i32(pk.seen), out=out)
    finally:
        ss.debug_packed_segment(0)
    ss.check()
    assert rel(host(out), y_ref) <= 5e-3
    for s, ref in s_ref.items():
        assert rel(host(cache[s]), ref) <= 1e-5 or not np.any(ref) and not np.any(host(cache[s]))

    # the decode step on the same slots, a row of each; rows far apart too
    rows = buf[::(pk.tokens - 1) // 3][:4]
    assert rows.stride(0) * 3 > 1 << 32
    tok = {k: rows[:, j * 72:j * 72 + inp[k].shape[1]] for j, k in enumerate(("u", "delta", "z", "B", "C"))}
    at = torch.from_numpy(pk.slots).cuda()
    part = cache[at].contiguous()
    y = ss.selscan_step(cache, tok["u"], tok["delta"], dev(inp["A"]), tok["B"], tok["C"], z=tok["z"],
                        slots=i32(pk.slots))
    ref = ss.selscan_step(part, *(tok[k].contiguous() for k in ("u", "delta")), dev(inp["A"]),
                          *(tok[k].contiguous() for k in ("B", "C")), z=tok["z"].contiguous())
    ss.check()
    assert torch.equal(y, ref) and torch.equal(cache[at], part)


@pytest.mark.parametrize("dim,dtype", [(D, "bf16"), (D - 1, "bf16"), (D, "f32")])
def test_convolution_of_far_rows_and_far_slots(room, dim, dtype):
    import torch
    rng = np.random.default_rng(91)
    pk = Packed(rng, [30, 2, 0, 3])
    pk.seen[:] = [3, 0, 0, 2]
    es = 2 if dtype == "bf16" else 4
    tt = torch.bfloat16 if dtype == "bf16" else torch.float32
    pitch = 1 << 27
    count = ((1 << 32) // (dim * 3)) + 9
    pk.slots = np.array([count - 1, count // 2 + 5, 5, count - 7])
    x, w, b = rnd(rng, pk.tokens, dim, dtype=dtype), rnd(rng, dim, 4), rnd(rng, dim)
    buf = torch.empty(pk.tokens, pitch, dtype=tt, device="cuda")
    xs, out = buf[:, :dim], buf[:, 128:128 + dim]
    xs.copy_(dev(x, dtype))
    cache = torch.empty(count, dim, 3, dtype=tt, device="cuda")
    assert (pk.tokens - 1) * pitch > 1 << 32 and (count - 7) * dim * 3 > 1 << 32
    st0 = {int(s): rnd(rng, dim, 3, dtype=dtype) for s in pk.slots}
    for s, v in st0.items():
        cache[s] = dev(v, dtype)
    ss.selscan_conv_packed(cache, xs, dev(w), *pk.args(), bias=dev(b), seen=i32(pk.seen), out=out)
    ss.check()
    got = host(out)
    for i, rows, slot in pk.each():
        ref, last, size = plain_layer.conv(x[rows].T, w, b, True, st0[slot] if pk.seen[i] else None)
        tol = (2.0 ** -8 if es == 2 else 0) * np.abs(ref) + 2.0 ** -20 * (size + np.abs(ref))
        assert (np.abs(got[rows].T - ref) <= tol).all(), i
        assert np.array_equal(host(cache[slot]), last), i

    tok = xs[::(pk.tokens - 1) // 3][:4]
    at = torch.from_numpy(pk.slots).cuda()
    part = cache[at].contiguous()
    y = ss.selscan_conv_step(cache, tok, dev(w), bias=dev(b), slots=i32(pk.slots))
    ref = ss.selscan_conv_step(part, tok.contiguous(), dev(w), bias=dev(b))
    ss.check()
    assert torch.equal(y, ref) and torch.equal(cache[at], part)
