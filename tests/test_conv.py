"""GPU parity of the short causal convolution (selscan_conv, its gradients
selscan_conv_bwd, its single-token step) with plain fp64 numpy.

Tolerances, per element.  A bf16 result is rounded once: 2^-8 of its value.
Below that, fp32 arithmetic: the W + 1 <= 5 additions of a pre-activation are
off by at most 5 * 2^-24 of the sum S of its absolute terms, SiLU (slope at
most 1.1, special-function error below 2^-20 of its value) keeps that, so
|y - ref| <= 2^-20 (S + |ref|) covers it.  A gradient g has slope error below
2^-19 (1 + S) |dy| (SiLU' changes by at most 0.5 per unit of v), and dx adds at
most four of them.  dweight sums n = batch * L terms: each addition is off by
at most 2^-24 of the partial sum, and a sum of n terms in any order has at most
n additions in a chain."""
import numpy as np
import pytest

import plain_layer
import synthetic

pytestmark = pytest.mark.gpu

F32 = 2.0 ** -20


def half_step(dtype):
    return 2.0 ** -8 if dtype == "bf16" else 0.0


def rnd(rng, *shape, dtype="f32", scale=1.0):
    a = (scale * rng.standard_normal(shape)).astype(np.float32)
    return synthetic.round_bf16(a) if dtype == "bf16" else a


def tdt(dtype):
    import torch
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def dev(a, dtype="f32", layout="channels"):
    """On the GPU; (b, D, L) arrays as channels-first, or as the view of a
    token-major tensor, of the first half of a (b, L, 2D) one, or of rows at
    odd offsets."""
    import torch
    if a is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(a)).to(tdt(dtype)).cuda()
    if layout == "channels":
        return t
    b, D, L = t.shape
    if layout == "tokens":
        return t.transpose(1, 2).contiguous().transpose(1, 2)
    if layout == "half":
        buf = torch.full((b, L, 2 * D), float("nan"), dtype=t.dtype, device="cuda")
        buf[..., :D] = t.transpose(1, 2)
        return buf[..., :D].transpose(1, 2)
    if layout == "odd":  # rows that no 16-byte vector fits
        buf = torch.full((b, D, L + 3), float("nan"), dtype=t.dtype, device="cuda")
        buf[..., 1:L + 1] = t
        return buf[..., 1:L + 1]
    assert layout == "strange"  # neither direction contiguous
    buf = torch.full((b, L, D, 2), float("nan"), dtype=t.dtype, device="cuda")
    buf[..., 1] = t.transpose(1, 2)
    return buf[..., 1].transpose(1, 2)


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def near(got, ref, tol, what=""):
    got = host(got)
    assert got.shape == ref.shape, what
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(),
                           got[bad][:3], ref[bad][:3])


SHAPES = [  # batch, D, L
    (2, 64, 256), (1, 8, 8), (3, 40, 77), (2, 5, 33), (1, 1, 1), (2, 24, 2), (1, 300, 129),
    (2, 136, 1), (1, 16, 1030),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("xl,yl", [("channels", "channels"), ("tokens", "channels"),
                                   ("half", "channels"), ("channels", "tokens"),
                                   ("half", "tokens"), ("odd", "odd"), ("strange", "strange")])
def test_conv_matches_plain(dtype, xl, yl):
    import torch
    import selective_state_space_selscan_b200 as ss
    rng = np.random.default_rng(5)
    for i, (b, D, L) in enumerate(SHAPES):
        for W in (2, 3, 4):
            x, w = rnd(rng, b, D, L, dtype=dtype), rnd(rng, D, W)
            bias = rnd(rng, D) if (i + W) % 3 else None
            h0 = rnd(rng, b, D, W - 1, dtype=dtype) if (i + W) % 2 else None
            silu = (i + W) % 4 != 0
            ref, last_ref, size = plain_layer.conv(x, w, bias, silu, h0)
            out = dev(np.zeros_like(x), dtype, yl)
            y, last = ss.selscan_conv(dev(x, dtype, xl), dev(w), bias=dev(bias), silu=silu,
                                      h0=dev(h0, dtype), out=out)
            ss.check()
            assert y is out
            near(y, ref, half_step(dtype) * np.abs(ref) + F32 * (size + np.abs(ref)), (b, D, L, W))
            assert np.array_equal(host(last), last_ref)
    assert torch.isfinite(y.float()).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("xl,yl", [("channels", "channels"), ("tokens", "channels"),
                                   ("half", "channels"), ("channels", "tokens"),
                                   ("half", "tokens"), ("odd", "odd"), ("strange", "strange")])
def test_conv_gradients_match_plain(dtype, xl, yl):
    import selective_state_space_selscan_b200 as ss
    rng = np.random.default_rng(6)
    for i, (b, D, L) in enumerate(SHAPES):
        for W in (2, 3, 4):
            x, w, dy = (rnd(rng, b, D, L, dtype=dtype), rnd(rng, D, W),
                        rnd(rng, b, D, L, dtype=dtype))
            bias = rnd(rng, D) if (i + W) % 3 else None
            states = (i + W) % 2
            h0 = rnd(rng, b, D, W - 1, dtype=dtype) if states else None
            dlast = rnd(rng, b, D, W - 1, dtype=dtype) if states else None
            silu = (i + W) % 4 != 0
            ref = plain_layer.conv_grads(x, w, dy, bias, silu, h0, dlast)
            g = ss.selscan_conv_bwd(dev(x, dtype, xl), dev(w), dev(dy, dtype, yl),
                                    bias=dev(bias), silu=silu, h0=dev(h0, dtype),
                                    dlast=dev(dlast, dtype))
            ss.check()
            what = (b, D, L, W)
            near(g["dx"], ref["dx"], half_step(dtype) * np.abs(ref["dx"]) + 2 * F32 * ref["dxsize"],
                 what + ("dx",))
            n = b * L + 16
            near(g["dweight"], ref["dweight"], (n * 2.0 ** -24 + 2 * F32) * ref["dwsize"],
                 what + ("dweight",))
            if bias is None:
                assert g["dbias"] is None
            else:
                near(g["dbias"], ref["dbias"], (n * 2.0 ** -24 + 2 * F32) * ref["dbsize"],
                     what + ("dbias",))
            if states:
                near(g["dh0"], ref["dh0"],
                     half_step(dtype) * np.abs(ref["dh0"]) + 2 * F32 * ref["dh0size"],
                     what + ("dh0",))
            else:
                assert g["dh0"] is None


@pytest.mark.parametrize("W", [2, 3, 4])
def test_conv_gradients_by_differences(W):
    """The kernel's gradients against central differences of the plain
    forward's loss, entry by entry.  Step 1e-4: the truncation error is about
    1e-8 times third derivatives of order one, the fp64 rounding 1e-12."""
    import selective_state_space_selscan_b200 as ss
    rng = np.random.default_rng(7)
    b, D, L = 2, 3, 5
    x, w, bias = rnd(rng, b, D, L), rnd(rng, D, W), rnd(rng, D)
    h0, dy, dlast = rnd(rng, b, D, W - 1), rnd(rng, b, D, L), rnd(rng, b, D, W - 1)
    g = ss.selscan_conv_bwd(dev(x), dev(w), dev(dy), bias=dev(bias), h0=dev(h0), dlast=dev(dlast))
    ss.check()

    def loss(x, w, bias, h0):
        y, last, _ = plain_layer.conv(x, w, bias, True, h0)
        return (dy * y).sum() + (dlast * last).sum()

    args = [a.astype(np.float64) for a in (x, w, bias, h0)]
    for i, key in enumerate(("dx", "dweight", "dbias", "dh0")):
        num = np.zeros(args[i].shape)
        for j in np.ndindex(num.shape):
            for sign in (1, -1):
                moved = [a.copy() for a in args]
                moved[i][j] += sign * 1e-4
                num[j] += sign * loss(*moved) / 2e-4
        near(g[key], num, 1e-5 * (1 + np.abs(num)), key)


def test_conv_without_tokens_or_rows():
    import torch
    import selective_state_space_selscan_b200 as ss
    w = torch.ones(16, 4, device="cuda")
    for dt in (torch.float32, torch.bfloat16):
        x = torch.empty(2, 16, 0, device="cuda", dtype=dt)
        h0 = torch.randn(2, 16, 3, device="cuda").to(dt)
        y, last = ss.selscan_conv(x, w, h0=h0)
        assert y.shape == (2, 16, 0) and torch.equal(last, h0)
        y, last = ss.selscan_conv(x, w)
        assert (last == 0).all()
        g = ss.selscan_conv_bwd(x, w, x, bias=w[:, 0].contiguous(), h0=h0, dlast=2 * h0)
        assert torch.equal(g["dh0"], 2 * h0) and (g["dweight"] == 0).all() and (g["dbias"] == 0).all()
        e = torch.empty(0, 16, 8, device="cuda", dtype=dt)
        y, last = ss.selscan_conv(e, w)
        assert y.shape == (0, 16, 8) and last.shape == (0, 16, 3)
        g = ss.selscan_conv_bwd(e, w, e)
        assert (g["dweight"] == 0).all()
    ss.check()


def test_conv_continues_in_place():
    """Chunks of a sequence, the state in one buffer, equal the whole."""
    import torch
    import selective_state_space_selscan_b200 as ss
    rng = np.random.default_rng(8)
    x, w = rnd(rng, 2, 48, 200, dtype="bf16"), rnd(rng, 48, 4)
    whole, last = ss.selscan_conv(dev(x, "bf16"), dev(w))
    state = torch.zeros(2, 48, 3, dtype=torch.bfloat16, device="cuda")
    parts, at = [], 0
    for n in (64, 1, 2, 5, 128):
        y, st = ss.selscan_conv(dev(x[..., at:at + n], "bf16"), dev(w), h0=state, last_state=state)
        assert st is state
        parts.append(y)
        at += n
    ss.check()
    assert torch.equal(torch.cat(parts, 2), whole) and torch.equal(state, last)


def test_conv_is_causal_next_to_nan_and_infinity():
    """A NaN or an infinity reaches the W tokens from its own on, and in the
    gradients the tokens whose windows hold it: nothing else."""
    import torch
    import selective_state_space_selscan_b200 as ss
    rng = np.random.default_rng(9)
    for layout in ("channels", "tokens"):
        for bad in (float("nan"), float("inf")):
            for at in (0, 3, 40, 76):
                x, w, dy = rnd(rng, 1, 24, 77), rnd(rng, 24, 4), rnd(rng, 1, 24, 77)
                clean, _ = ss.selscan_conv(dev(x, layout=layout), dev(w))
                gclean = ss.selscan_conv_bwd(dev(x, layout=layout), dev(w), dev(dy))
                x[0, 7, at] = bad
                y, _ = ss.selscan_conv(dev(x, layout=layout), dev(w))
                g = ss.selscan_conv_bwd(dev(x, layout=layout), dev(w), dev(dy))
                ss.check()
                hit = torch.zeros(1, 24, 77, dtype=torch.bool, device="cuda")
                hit[0, 7, at:at + 4] = True
                assert torch.equal(y[~hit], clean[~hit])
                hit[0, 7, max(0, at - 3):at + 4] = True
                assert torch.equal(g["dx"][~hit], gclean["dx"][~hit])
                rows = torch.arange(24, device="cuda") != 7
                assert torch.equal(g["dweight"][rows], gclean["dweight"][rows])


def test_conv_extreme_values():
    """Large pre-activations: SiLU and its slope saturate without overflow."""
    import selective_state_space_selscan_b200 as ss
    for dtype in ("f32", "bf16"):
        x = np.array([[[-1e4, -200.0, -90.0, -30.0, 0.0, 30.0, 90.0, 1e4, 1e30, -1e30]]],
                     np.float32)
        x = synthetic.round_bf16(x) if dtype == "bf16" else x
        w = np.array([[0.0, 1.0]], np.float32)
        y, _ = ss.selscan_conv(dev(x, dtype), dev(w))
        g = ss.selscan_conv_bwd(dev(x, dtype), dev(w), dev(np.ones_like(x), dtype))
        ss.check()
        ref, _, size = plain_layer.conv(x, w)
        # below 2^-126 results may be flushed to zero
        near(y, ref, half_step(dtype) * np.abs(ref) + F32 * np.abs(ref) + 1e-30)
        gr = plain_layer.conv_grads(x, w, np.ones_like(x))
        near(g["dx"], gr["dx"], half_step(dtype) * np.abs(gr["dx"]) + 2 * F32 + 1e-30)


def test_conv_backward_repeats_bit_for_bit():
    import torch
    import selective_state_space_selscan_b200 as ss
    rng = np.random.default_rng(10)
    x, w, dy = (rnd(rng, 3, 96, 700, dtype="bf16"), rnd(rng, 96, 4), rnd(rng, 3, 96, 700, dtype="bf16"))
    args = (dev(x, "bf16", "half"), dev(w), dev(dy, "bf16"))
    bias = dev(rnd(rng, 96))
    a = ss.selscan_conv_bwd(*args, bias=bias)
    for _ in range(3):
        b = ss.selscan_conv_bwd(*args, bias=bias)
        assert all(torch.equal(a[k], b[k]) for k in ("dx", "dweight", "dbias"))
    ss.check()
    assert a["dx"].stride(1) == 1  # x's layout


def test_conv_offsets_past_32_bits():
    """Rows more than 2^31 elements apart."""
    import torch
    import selective_state_space_selscan_b200 as ss
    far = (1 << 31) + 64
    buf = torch.empty(far + 64 * 64, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(11)
    x, w = rnd(rng, 2, 32, 64, dtype="bf16"), rnd(rng, 32, 4)
    for strides in ((far, 64, 1), (far, 1, 32)):
        v = torch.as_strided(buf, (2, 32, 64), strides)
        v.copy_(dev(x, "bf16"))
        ref, last = ss.selscan_conv(dev(x, "bf16"), dev(w))
        y, l2 = ss.selscan_conv(v, dev(w))
        assert torch.equal(y, ref) and torch.equal(last, l2)
        g = ss.selscan_conv_bwd(v, dev(w), ref)
        gr = ss.selscan_conv_bwd(dev(x, "bf16"), dev(w), ref)
        assert torch.equal(g["dx"], gr["dx"])
        out = torch.as_strided(buf, (2, 32, 64), strides)
        out.zero_()
        ss.selscan_conv(dev(x, "bf16"), dev(w), out=out)
        assert torch.equal(out, ref)
    ss.check()


def test_conv_sizes_of_every_launch_form():
    """Sizes at which the kernels take another split: channels that fill a
    warp, part of it, or several; runs of one tile, of many, of a part."""
    import selective_state_space_selscan_b200 as ss
    rng = np.random.default_rng(16)
    for b, D, L in ((1, 2, 3000), (1, 1024, 9), (2, 260, 515), (1, 32, 4100), (5, 72, 64)):
        for dtype in ("f32", "bf16"):
            for layout in ("channels", "tokens", "half"):
                x, w, dy = rnd(rng, b, D, L, dtype=dtype), rnd(rng, D, 4), rnd(rng, b, D, L, dtype=dtype)
                ref, last, size = plain_layer.conv(x, w)
                y, st = ss.selscan_conv(dev(x, dtype, layout), dev(w))
                near(y, ref, half_step(dtype) * np.abs(ref) + F32 * (size + np.abs(ref)), (b, D, L))
                gr = plain_layer.conv_grads(x, w, dy)
                g = ss.selscan_conv_bwd(dev(x, dtype, layout), dev(w), dev(dy, dtype))
                ss.check()
                near(g["dx"], gr["dx"], half_step(dtype) * np.abs(gr["dx"]) + 2 * F32 * gr["dxsize"])
                near(g["dweight"], gr["dweight"],
                     ((b * L + 16) * 2.0 ** -24 + 2 * F32) * gr["dwsize"])


# ------------------------------------------------------------ single tokens
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("batch,D", [(1, 64), (3, 40), (5, 7), (33, 1), (2, 1030), (300, 16)])
def test_conv_step_matches_plain(dtype, batch, D):
    import torch
    import selective_state_space_selscan_b200 as ss
    rng = np.random.default_rng(12)
    for W in (2, 3, 4):
        for slotted in (False, True):
            count = batch + 4 if slotted else batch
            st0 = rnd(rng, count, D, W - 1, dtype=dtype)
            x, w, bias = rnd(rng, batch, D, dtype=dtype), rnd(rng, D, W), rnd(rng, D)
            rows = rng.permutation(count)[:batch] if slotted else np.arange(batch)
            state = dev(st0, dtype)
            slots = torch.from_numpy(rows.astype(np.int32)).cuda() if slotted else None
            y = ss.selscan_conv_step(state, dev(x, dtype), dev(w), bias=dev(bias), slots=slots)
            ss.check()
            ref, last, size = plain_layer.conv(x[..., None], w, bias, True, st0[rows])
            near(y, ref[..., 0], half_step(dtype) * np.abs(ref[..., 0]) +
                 F32 * (size + np.abs(ref))[..., 0])
            want = st0.astype(np.float64)
            want[rows] = last
            assert np.array_equal(host(state), want)


def test_conv_step_strides_in_place_and_padding():
    import torch
    import selective_state_space_selscan_b200 as ss
    rng = np.random.default_rng(13)
    B, D = 6, 32
    w, x = rnd(rng, D, 4), rnd(rng, B, D, dtype="bf16")
    st0 = rnd(rng, 9, D, 3, dtype="bf16")
    slots = torch.tensor([4, -1, 8, 0, -7, 2], dtype=torch.int32, device="cuda")
    want_state = dev(st0, "bf16")
    want = ss.selscan_conv_step(want_state, dev(x, "bf16"), dev(w), slots=slots,
                                out=torch.full((B, D), 9.0, dtype=torch.bfloat16, device="cuda"))
    assert (want[[1, 4]] == 9).all()  # padding rows stay
    keep = [1, 3, 5, 6, 7]
    assert torch.equal(want_state[keep], dev(st0, "bf16")[keep])
    # x and y as columns of wider tensors, and y over x
    for wide in (2 * D, 2 * D + 1):
        buf = torch.full((B, wide), 9.0, dtype=torch.bfloat16, device="cuda")
        buf[:, 1:D + 1] = dev(x, "bf16")
        state = dev(st0, "bf16")
        out = torch.full((B, 2 * D), 9.0, dtype=torch.bfloat16, device="cuda")[:, ::2]
        ss.selscan_conv_step(state, buf[:, 1:D + 1], dev(w), slots=slots, out=out)
        assert torch.equal(out, want) and torch.equal(state, want_state)
    xd, state = dev(x, "bf16"), dev(st0, "bf16")
    ss.selscan_conv_step(state, xd, dev(w), slots=slots, out=xd)
    ss.check()
    live = [0, 2, 3, 5]
    assert torch.equal(xd[live], want[live]) and torch.equal(state, want_state)


def test_conv_step_refuses_slots_on_the_device():
    import torch
    import selective_state_space_selscan_b200 as ss
    rng = np.random.default_rng(14)
    D = 300
    w, x, st0 = rnd(rng, D, 4), rnd(rng, 4, D), rnd(rng, 3, D, 3)
    for bad, skipped in (([0, 1, 0, 2], 2), ([0, 3, 1, 2], 1), ([2, 1, 1 << 30, 0], 2)):
        state = dev(st0)
        out = torch.full((4, D), 9.0, device="cuda")
        slots = torch.tensor(bad, dtype=torch.int32, device="cuda")
        ss.selscan_conv_step(state, dev(x), dev(w), slots=slots, out=out)
        with pytest.raises(ss.SelscanError, match="SELSCAN_ERR_INDEX"):
            ss.check()
        ss.check()  # the record is cleared
        assert (out[skipped] == 9).all()
        keep = [i for i in range(4) if i != skipped]
        ref, last, _ = plain_layer.conv(x[keep][..., None], w, None, True, st0[[bad[i] for i in keep]])
        near(out[keep], ref[..., 0], 1e-5 * (1 + np.abs(ref[..., 0])))
        assert np.array_equal(host(state)[[bad[i] for i in keep]], last)


def test_conv_on_another_stream_and_in_a_graph():
    import torch
    import selective_state_space_selscan_b200 as ss
    rng = np.random.default_rng(15)
    x, w, dy = rnd(rng, 2, 64, 300, dtype="bf16"), rnd(rng, 64, 4), rnd(rng, 2, 64, 300, dtype="bf16")
    xd, wd, dyd = dev(x, "bf16", "half"), dev(w), dev(dy, "bf16")
    want, _ = ss.selscan_conv(xd, wd)
    gwant = ss.selscan_conv_bwd(xd, wd, dyd)
    st0 = dev(rnd(rng, 2, 64, 3, dtype="bf16"), "bf16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, _ = ss.selscan_conv(xd, wd, stream=side)
    g = ss.selscan_conv_bwd(xd, wd, dyd, stream=side)
    side.synchronize()
    assert torch.equal(y, want) and torch.equal(g["dweight"], gwant["dweight"])
    # two captured graphs, replayed in turn after other work on the scratch pool
    graphs = []
    for scale in (1.0, -1.0):
        xs, dys, state = (xd * scale).clone(), dyd.clone(), st0.clone()
        tok = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            y, _ = ss.selscan_conv(xs, wd)
            g = ss.selscan_conv_bwd(xs, wd, dys)
            ss.selscan_conv_step(state, xs[..., 0], wd, out=tok)
        graphs.append((gr, xs, dys, y, g, state, tok))
    for _ in range(3):
        for gr, xs, dys, y, g, state, tok in graphs:
            dys.copy_(torch.randn_like(dys))
            state.copy_(st0)
            gr.replay()
            again = ss.selscan_conv_bwd(xs, wd, dys)
            torch.cuda.synchronize()
            assert torch.equal(again["dx"], g["dx"]) and torch.equal(again["dweight"], g["dweight"])
            assert torch.equal(y, ss.selscan_conv(xs, wd)[0])
            st = st0.clone()
            assert torch.equal(tok, ss.selscan_conv_step(st, xs[..., 0], wd))
            assert torch.equal(st, state)
    ss.check()
