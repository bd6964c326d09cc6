"""The operators around the scan, as a model's layer meets them: the short
causal convolution in front of it (prompts, training, single tokens), the scan
of packed prompts of unequal lengths over a cache of states, and the decode
step through that cache.  Each has a plain form in elementary torch operations
(``own = False``) and the library's calls (``own = True``) on the same inputs.

Layouts as the layer has them: the input projection gives x and z as the two
halves of a token-major (tokens, 2 D) product, the scan's projection gives
B and C as slices of (tokens, R + 2 N); weights, A, D and biases are fp32.
"""
import math

import torch

own = False

N = 16  # states per channel of the diagonal scan


def listed():
    return [
        # a training or prefill layer of a 2.8B-sized model: x is the first half
        # of the input projection, y goes on to the channels-first scan
        dict(name="conv prompt bf16", op="conv", batch=4, dim=5120, L=4096, width=4,
             dtype="bf16", layout="tokens", h0=False),
        # the smallest layer, fp32, continued from a saved state
        dict(name="conv small fp32", op="conv", batch=1, dim=64, L=256, width=4,
             dtype="f32", layout="channels", h0=True),
        # a prefill batch of a serving loop: unequal prompts and chunks of prompts
        dict(name="conv packed bf16", op="conv_packed", seqs=24, tokens=8192, dim=2560,
             width=4, dtype="bf16", pad=0),
        # the backward pass of a training layer
        dict(name="conv backward bf16", op="conv_bwd", batch=8, dim=2560, L=2048, width=4,
             dtype="bf16", layout="tokens", h0=False),
        # odd sizes, three taps, fp32, with the gradients of both states
        dict(name="conv backward odd fp32", op="conv_bwd", batch=3, dim=200, L=999, width=3,
             dtype="f32", layout="channels", h0=True),
        # one token of one request: latency
        dict(name="conv step one", op="conv_step", batch=1, dim=2560, width=4, dtype="bf16",
             pad=0),
        # one token of each request of a large decode batch, padded rows at its end
        dict(name="conv step batch", op="conv_step", batch=1024, dim=5120, width=4,
             dtype="bf16", pad=24),
        # a prefill batch: prompts of unequal lengths, some continued; a trained A
        dict(name="scan packed bf16", op="scan_packed", seqs=32, tokens=16384, dim=2048,
             dtype="bf16", gate=True, A="free", pad=0),
        # one long prompt, A as models are initialised
        dict(name="scan packed long", op="scan_packed", seqs=1, tokens=131072, dim=2048,
             dtype="bf16", gate=True, A="real", pad=0),
        # a few short prompts in fp32
        dict(name="scan packed fp32", op="scan_packed", seqs=5, tokens=257, dim=64,
             dtype="f32", gate=True, A="free", pad=7),
        # decode batches through a cache with more slots than requests: diagonal ...
        dict(name="step slots", op="step_slots", form="diag", batch=256, dim=5120,
             dtype="bf16", pad=6),
        # ... and one scalar A per head (32 heads of 64 channels, 128 states)
        dict(name="step slots scalar", op="step_slots", form="scalar", batch=64, dim=2048,
             dtype="bf16", pad=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "conv_packed", "conv_bwd", "conv_step", "scan_packed",
                     "step_slots"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("conv", "conv_bwd"):
        most = 20_000_000 if op == "conv" else 10_000_000
        batch, dim = _log(rng, 1, 8), _log(rng, 16, 5120)
        if rng.random() < 0.5:
            dim = max(16, dim // 16 * 16)
        L = max(1, min(_log(rng, 1, 8192), most // (batch * dim)))
        return dict(op=op, batch=batch, dim=dim, L=L, width=rng.choice([2, 3, 4, 4]),
                    dtype=dtype, layout=rng.choice(["tokens", "channels"]),
                    h0=rng.random() < 0.5)
    if op == "conv_packed":
        seqs, dim, tokens = _log(rng, 1, 200), _log(rng, 16, 2560), _log(rng, 1, 8192)
        return dict(op=op, seqs=seqs, tokens=tokens, dim=dim, width=rng.choice([2, 3, 4, 4]),
                    dtype=dtype, pad=rng.choice([0, 0, 5]) if tokens > 20 else 0)
    if op == "conv_step":
        return dict(op=op, batch=_log(rng, 1, 1024), dim=_log(rng, 16, 2560),
                    width=rng.choice([2, 3, 4, 4]), dtype=dtype, pad=rng.choice([0, 0, 9]))
    if op == "scan_packed":
        dim = _log(rng, 16, 2048)
        if rng.random() < 0.5:
            dim = max(16, dim // 16 * 16)
        tokens = min(_log(rng, 1, 32768), 16_000_000 // dim)
        return dict(op=op, seqs=_log(rng, 1, 64), tokens=tokens, dim=dim, dtype=dtype,
                    gate=rng.random() < 0.7, A=rng.choice(["free", "real"]),
                    pad=rng.choice([0, 0, 3]) if tokens > 20 else 0)
    form = rng.choice(["diag", "scalar"])
    if form == "diag":
        return dict(op=op, form=form, batch=_log(rng, 1, 256), dim=_log(rng, 16, 5120),
                    dtype=dtype, pad=rng.choice([0, 0, 4]))
    return dict(op=op, form=form, batch=_log(rng, 1, 64), dim=64 * rng.randint(1, 32),
                dtype=dtype, pad=rng.choice([0, 0, 4]))


def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


class _Random:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(self, *shape, dtype=torch.float32, scale=1.0):
        t = torch.randn(*shape, device="cuda", generator=self.g, dtype=torch.float32)
        return t.mul_(scale).to(dtype)

    def uniform(self, lo, hi, *shape):
        return torch.rand(*shape, device="cuda", generator=self.g).mul_(hi - lo).add_(lo)

    def order(self, n):
        return torch.randperm(n, device="cuda", generator=self.g)


def _lengths(r, seqs, tokens, pad):
    """Sequence starts of ``seqs`` prompts of log-normal lengths (the shortest
    may be empty) that fill ``tokens`` rows but for ``pad`` rows at the end."""
    share = torch.cumsum(torch.exp(1.2 * r.normal(seqs)).double(), 0)
    ends = torch.round(share / share[-1] * max(0, tokens - pad)).to(torch.int32)
    return torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), ends])


def _cache(r, s, rows, pad):
    """Slots of ``rows`` requests in a cache with room for half as many more;
    the last ``pad`` rows of a decode batch hold none."""
    s["count"] = rows + rows // 2 + 1
    slots = r.order(s["count"])[:rows].to(torch.int32)
    s["live"] = max(1, rows - pad)
    slots[s["live"]:] = -1
    s["slots"] = slots


def _conv_weights(r, s, dim, width):
    s["weight"] = r.uniform(-1, 1, dim, width) / math.sqrt(width)
    s["bias"] = r.uniform(-0.5, 0.5, dim)


def _scan_weights(r, s, dim, free):
    A = -torch.arange(1, N + 1, device="cuda", dtype=torch.float32).expand(dim, N)
    s["A"] = (A * torch.exp(0.2 * r.normal(dim, N)) if free else A).contiguous()
    step = torch.exp(r.uniform(math.log(1e-3), math.log(1e-1), dim))
    s["delta_bias"] = torch.log(torch.expm1(step))
    s["D"] = r.normal(dim)


def prepare(case, seed):
    r, dt, op = _Random(seed), _type(case), case["op"]
    dim = case["dim"]
    s = dict(op=op, case=case)
    if op in ("conv", "conv_bwd"):
        b, L, w = case["batch"], case["L"], case["width"]
        _conv_weights(r, s, dim, w)
        if case["layout"] == "tokens":
            s["x"] = r.normal(b, L, 2 * dim, dtype=dt)[..., :dim].transpose(1, 2)
        else:
            s["x"] = r.normal(b, dim, L, dtype=dt)
            if L % 2:  # rows longer than the sequence, as a padded buffer has them
                s["x"] = r.normal(b, dim, L + 1, dtype=dt)[..., :L]
        s["h0"] = r.normal(b, dim, w - 1, dtype=dt) if case["h0"] else None
        if op == "conv_bwd":
            s["dy"] = r.normal(b, dim, L, dtype=dt)
            s["dlast"] = r.normal(b, dim, w - 1, dtype=dt) if case["h0"] else None
    elif op == "conv_packed":
        T = case["tokens"]
        _conv_weights(r, s, dim, case["width"])
        s["x"] = r.normal(T, 2 * dim, dtype=dt)[:, :dim]
        s["start"] = _lengths(r, case["seqs"], T, case["pad"])
        _cache(r, s, case["seqs"], 0)
        s["seen"] = (r.uniform(0, 1, case["seqs"]) < 0.4).to(torch.int32) * 100
        s["state"] = r.normal(s["count"], dim, case["width"] - 1, dtype=dt)
        s["y"] = torch.zeros(T, dim, device="cuda", dtype=dt)
    elif op == "conv_step":
        b = case["batch"]
        _conv_weights(r, s, dim, case["width"])
        _cache(r, s, b, case["pad"])
        s["x"] = r.normal(b, 2 * dim, dtype=dt)[:, :dim]
        s["state"] = r.normal(s["count"], dim, case["width"] - 1, dtype=dt)
        s["y"] = torch.zeros(b, dim, device="cuda", dtype=dt)
    elif op == "scan_packed":
        T, rank = case["tokens"], -(-dim // 16)
        _scan_weights(r, s, dim, case["A"] == "free")
        s["u"] = r.normal(T, dim, dtype=dt)
        s["delta"] = r.normal(T, dim, dtype=dt, scale=0.5)
        s["z"] = r.normal(T, 2 * dim, dtype=dt)[:, dim:] if case["gate"] else None
        proj = r.normal(T, rank + 2 * N, dtype=dt)
        s["B"], s["C"] = proj[:, rank:rank + N], proj[:, rank + N:]
        s["start"] = _lengths(r, case["seqs"], T, case["pad"])
        _cache(r, s, case["seqs"], 0)
        s["seen"] = (r.uniform(0, 1, case["seqs"]) < 0.4).to(torch.int32) * 100
        s["state"] = r.normal(s["count"], dim, N)
        s["y"] = torch.zeros(T, dim, device="cuda", dtype=dt)
    elif case["form"] == "diag":
        b, rank = case["batch"], -(-dim // 16)
        _scan_weights(r, s, dim, True)
        _cache(r, s, b, case["pad"])
        s["u"] = r.normal(b, dim, dtype=dt)
        s["delta"] = r.normal(b, dim, dtype=dt, scale=0.5)
        s["z"] = r.normal(b, 2 * dim, dtype=dt)[:, dim:]
        proj = r.normal(b, rank + 2 * N, dtype=dt)
        s["B"], s["C"] = proj[:, rank:rank + N], proj[:, rank + N:]
        s["state"] = r.normal(s["count"], dim, N)
        s["y"] = torch.zeros(b, dim, device="cuda", dtype=dt)
    else:
        b, H, P, NS = case["batch"], dim // 64, 64, 128
        _cache(r, s, b, case["pad"])
        s["A"] = -torch.exp(r.uniform(0, math.log(16), H))
        s["D"] = r.normal(H)
        step = torch.exp(r.uniform(math.log(1e-3), math.log(1e-1), H))
        s["delta_bias"] = torch.log(torch.expm1(step))
        xbc = r.normal(b, dim + 2 * NS, dtype=dt)
        s["u"] = xbc[:, :dim]
        s["B"], s["C"] = xbc[:, dim:dim + NS], xbc[:, dim + NS:]
        s["delta"] = r.normal(b, H, scale=0.5)
        s["z"] = r.normal(b, dim, dtype=dt)
        s["state"] = r.normal(s["count"], H, P, NS)
        s["y"] = torch.zeros(b, dim, device="cuda", dtype=dt)
    return s


def work(case):
    e, dim, op = (2 if case["dtype"] == "bf16" else 4), case["dim"], case["op"]
    if op in ("conv", "conv_bwd"):
        n, w = case["batch"] * dim * case["L"], case["width"]
        ends = case["batch"] * dim * (w - 1) * e * ((2 if case["h0"] else 1))
        if op == "conv":
            return dict(bytes=2 * n * e + ends + dim * (w + 1) * 4, flops=n * (2 * w + 6))
        return dict(bytes=3 * n * e + (2 * ends if case["h0"] else 0) + 2 * dim * (w + 1) * 4,
                    flops=n * (6 * w + 12))
    if op == "conv_packed":
        n, w = case["tokens"] * dim, case["width"]
        return dict(bytes=2 * n * e + 2 * case["seqs"] * dim * (w - 1) * e + dim * (w + 1) * 4,
                    flops=n * (2 * w + 6))
    if op == "conv_step":
        n, w = case["batch"] * dim, case["width"]
        return dict(bytes=n * (2 + 2 * (w - 1)) * e + dim * (w + 1) * 4, flops=n * (2 * w + 6))
    if op == "scan_packed":
        n = case["tokens"] * dim
        return dict(bytes=n * (4 if case["gate"] else 3) * e + case["tokens"] * 2 * N * e +
                    2 * case["seqs"] * dim * N * 4 + dim * (N + 2) * 4, flops=n * (7 * N + 12))
    n, ns = case["batch"] * dim, N if case["form"] == "diag" else 128
    return dict(bytes=n * ns * 8 + n * 4 * e + case["batch"] * 2 * ns * e, flops=n * (6 * ns + 12))


def run(s):
    return (_own if own else _plain)[s["op"]](s)


# ------------------------------------------------------------ plain forms
def _silu(v):
    return v / (1 + torch.exp(-v))


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _with_past(s):
    """x in 32 bits with the width - 1 inputs before it (zeros, or h0)."""
    x, w = s["x"].float(), s["weight"].shape[1]
    past = s["h0"].float() if s["h0"] is not None else x.new_zeros(*x.shape[:2], w - 1)
    return torch.cat([past, x], dim=2)


def _taps(e, weight, bias):
    """sum_k weight[:, k] e[:, :, t + k] + bias."""
    return (e.unfold(2, weight.shape[1], 1) * weight[:, None, :]).sum(-1) + bias[:, None]


def _plain_conv(s):
    e = _with_past(s)
    y = _silu(_taps(e, s["weight"], s["bias"]))
    return dict(y=y.to(s["x"].dtype),
                last_state=e[:, :, e.shape[2] - s["weight"].shape[1] + 1:].to(s["x"].dtype))


def _plain_conv_bwd(s):
    w, dt = s["weight"], s["x"].dtype
    past = w.shape[1] - 1
    e = _with_past(s)
    v = _taps(e, w, s["bias"])
    sg = 1 / (1 + torch.exp(-v))
    g = s["dy"].float() * sg * (1 + v * (1 - sg))
    dw = (e.unfold(2, past + 1, 1) * g[..., None]).sum((0, 2))
    # the gradient of e[i] sums w[k] g[i - k]
    gp = torch.nn.functional.pad(g, (past, past))
    de = (gp.unfold(2, past + 1, 1) * w.flip(1)[:, None, :]).sum(-1)
    if s["dlast"] is not None:
        de[:, :, de.shape[2] - past:] += s["dlast"].float()
    out = dict(dx=de[:, :, past:].to(dt), dweight=dw, dbias=g.sum((0, 2)))
    if s["h0"] is not None:
        out["dh0"] = de[:, :, :past].to(dt)
    return out


def _sequence_of(start, tokens):
    """The sequence of each row, and whether the row belongs to one."""
    t = torch.arange(tokens, device="cuda")
    seq = torch.searchsorted(start, t, right=True) - 1
    return t, torch.clamp(seq, max=start.numel() - 2), t < start[-1]


def _plain_conv_packed(s):
    w, slots = s["weight"], s["slots"].long()
    past, x = w.shape[1] - 1, s["x"].float()
    old = s["state"][slots].float() * (s["seen"] > 0)[:, None, None]
    # every sequence's rows behind its past, one after the other
    t, seq, inside = _sequence_of(s["start"], x.shape[0])
    e = x.new_zeros(x.shape[0] + slots.numel() * past, x.shape[1])
    first = s["start"][:-1] + torch.arange(slots.numel(), device="cuda") * past
    e[first[:, None] + torch.arange(past, device="cuda")] = old.transpose(1, 2)
    at = t + (seq + 1) * past
    e[at] = x
    v = (e.unfold(0, past + 1, 1)[at - past] * w).sum(-1) + s["bias"]
    s["y"].copy_(torch.where(inside[:, None], _silu(v).to(s["y"].dtype), s["y"]))
    last = first + s["start"][1:] - s["start"][:-1]
    s["state"][slots] = e[last[:, None] + torch.arange(past, device="cuda")].transpose(
        1, 2).to(s["state"].dtype)
    return dict(y=s["y"], state=s["state"])


def _plain_conv_step(s):
    n, slots = s["live"], s["slots"][:s["live"]].long()
    e = torch.cat([s["state"][slots].float(), s["x"][:n, :, None].float()], dim=2)
    s["y"][:n] = _silu((e * s["weight"]).sum(-1) + s["bias"]).to(s["y"].dtype)
    s["state"][slots] = e[:, :, 1:].to(s["state"].dtype)
    return dict(y=s["y"], state=s["state"])


def _plain_scan_packed(s):
    """All rows as one recurrence h_t = a_t h_{t-1} + b_t, whose a is zero at
    each first row and whose b holds that sequence's initial state there; over
    blocks of rows, by doubling inside a block."""
    T, dim = s["u"].shape
    slots = s["slots"].long()
    t, seq, inside = _sequence_of(s["start"], T)
    first = t == s["start"][seq]
    old = s["state"][slots] * (s["seen"] > 0)[:, None, None]
    block = max(64, min(T, 33554432 // (dim * N)))
    h = old.new_zeros(dim, N)
    # a sequence without rows keeps its initial state
    s["state"][slots] = old
    for lo in range(0, T, block):  # the recurrence over blocks of rows
        rows = slice(lo, min(T, lo + block))
        u = s["u"][rows].float()
        d = _softplus(s["delta"][rows].float() + s["delta_bias"])
        a = torch.exp(d[:, :, None] * s["A"])
        b = (d * u)[:, :, None] * s["B"][rows].float()[:, None, :]
        begin = first[rows, None, None]
        b = torch.where(begin, b + a * old[seq[rows]], b)
        a = torch.where(begin, a.new_zeros(()), a)
        b[0] += a[0] * h
        k = 1
        while k < a.shape[0]:  # rows already joined: 1, 2, 4, ...
            b = torch.cat([b[:k], b[k:] + a[k:] * b[:-k]])
            a = torch.cat([a[:k], a[k:] * a[:-k]])
            k *= 2
        h = b[-1]
        v = (b * s["C"][rows].float()[:, None, :]).sum(-1) + s["D"] * u
        if s["z"] is not None:
            v = v * _silu(s["z"][rows].float())
        s["y"][rows] = torch.where(inside[rows, None], v.to(s["y"].dtype), s["y"][rows])
        # the states behind the last rows of the sequences that end here
        end = s["start"][1:].long() - 1
        here = (end >= lo) & (end < lo + u.shape[0]) & (s["start"][1:] > s["start"][:-1])
        new = b[torch.clamp(end - lo, 0, u.shape[0] - 1)]
        s["state"][slots] = torch.where(here[:, None, None], new, s["state"][slots])
    return dict(y=s["y"], state=s["state"])


def _plain_step_slots(s):
    n, slots = s["live"], s["slots"][:s["live"]].long()
    u, z, old = s["u"][:n].float(), s["z"][:n].float(), s["state"][slots]
    B, C = s["B"][:n].float(), s["C"][:n].float()
    d = _softplus(s["delta"][:n].float() + s["delta_bias"])
    if s["case"]["form"] == "diag":
        new = torch.exp(d[:, :, None] * s["A"]) * old + (d * u)[:, :, None] * B[:, None, :]
        v = (new * C[:, None, :]).sum(-1) + s["D"] * u
    else:
        x = u.view(n, old.shape[1], old.shape[2])
        new = (torch.exp(d * s["A"])[:, :, None, None] * old +
               (d[:, :, None] * x)[..., None] * B[:, None, None, :])
        v = ((new * C[:, None, None, :]).sum(-1) + s["D"][:, None] * x).reshape(n, -1)
    s["y"][:n] = (v * _silu(z)).to(s["y"].dtype)
    s["state"][slots] = new
    return dict(y=s["y"], state=s["state"])


_plain = dict(conv=_plain_conv, conv_bwd=_plain_conv_bwd, conv_packed=_plain_conv_packed,
              conv_step=_plain_conv_step, scan_packed=_plain_scan_packed,
              step_slots=_plain_step_slots)


# ---------------------------------------------------------- the library's
def _own_conv(s):
    import selective_state_space_selscan_b200 as ss
    y, last = ss.selscan_conv(s["x"], s["weight"], bias=s["bias"], h0=s["h0"],
                              return_last_state=True)
    return dict(y=y, last_state=last)


def _own_conv_bwd(s):
    import selective_state_space_selscan_b200 as ss
    g = ss.selscan_conv_bwd(s["x"], s["weight"], s["dy"], bias=s["bias"], h0=s["h0"],
                            dlast=s["dlast"])
    keys = ("dx", "dweight", "dbias") + (("dh0",) if s["h0"] is not None else ())
    return {k: g[k] for k in keys}


def _own_conv_packed(s):
    import selective_state_space_selscan_b200 as ss
    ss.selscan_conv_packed(s["state"], s["x"], s["weight"], s["start"], s["slots"],
                           bias=s["bias"], seen=s["seen"], out=s["y"])
    return dict(y=s["y"], state=s["state"])


def _own_conv_step(s):
    import selective_state_space_selscan_b200 as ss
    ss.selscan_conv_step(s["state"], s["x"], s["weight"], bias=s["bias"], slots=s["slots"],
                         out=s["y"])
    return dict(y=s["y"], state=s["state"])


def _own_scan_packed(s):
    import selective_state_space_selscan_b200 as ss
    ss.selscan_fwd_packed(s["state"], s["u"], s["delta"], s["A"], s["B"], s["C"], s["start"],
                          s["slots"], D=s["D"], z=s["z"], delta_bias=s["delta_bias"],
                          seen=s["seen"], out=s["y"])
    return dict(y=s["y"], state=s["state"])


def _own_step_slots(s):
    import selective_state_space_selscan_b200 as ss
    kw = dict(D=s["D"], z=s["z"], slots=s["slots"], out=s["y"])
    if s["case"]["form"] == "diag":
        ss.selscan_step(s["state"], s["u"], s["delta"], s["A"], s["B"], s["C"],
                        delta_bias=s["delta_bias"], **kw)
    else:
        ss.selscan_step_scalarA(s["state"], s["u"], s["delta"], s["A"], s["B"], s["C"], 64,
                                dt_bias=s["delta_bias"], dt_softplus=True, **kw)
    return dict(y=s["y"], state=s["state"])


_own = dict(conv=_own_conv, conv_bwd=_own_conv_bwd, conv_packed=_own_conv_packed,
            conv_step=_own_conv_step, scan_packed=_own_scan_packed,
            step_slots=_own_step_slots)


# ------------------------------------------------------ in 64 bits, apart
def _x_conv(past, x, weight, bias):
    """One row of channels (dim, n) behind its past (dim, width - 1): the
    sums before the SiLU, tap by tap."""
    e, n = torch.cat([past, x], 1), x.shape[1]
    v = bias.double()[:, None].expand(-1, n)
    for k in range(weight.shape[1]):
        v = v + weight[:, k:k + 1].double() * e[:, k:k + n]
    return v, e[:, n:]


def exact(case, seed):
    s = prepare(case, seed)
    op, dim = case["op"], case["dim"]
    f = lambda t: None if t is None else t.double()
    if op in ("conv", "conv_bwd"):
        w = case["width"]
        zero = torch.zeros(dim, w - 1, device="cuda", dtype=torch.float64)
        if op == "conv":
            ys, lasts = [], []
            for b in range(case["batch"]):
                v, last = _x_conv(f(s["h0"][b]) if case["h0"] else zero, f(s["x"][b]),
                                  s["weight"], s["bias"])
                ys.append(v * torch.sigmoid(v))
                lasts.append(last)
            return dict(y=torch.stack(ys), last_state=torch.stack(lasts))
        dxs, dhs = [], []
        dw = torch.zeros(dim, w, device="cuda", dtype=torch.float64)
        db = torch.zeros(dim, device="cuda", dtype=torch.float64)
        for b in range(case["batch"]):
            past, x = f(s["h0"][b]) if case["h0"] else zero, f(s["x"][b])
            v, _ = _x_conv(past, x, s["weight"], s["bias"])
            sg = torch.sigmoid(v)
            g = f(s["dy"][b]) * (sg + v * sg * torch.sigmoid(-v))
            e = torch.cat([past, x], 1)
            de = torch.zeros_like(e)
            n = x.shape[1]
            for k in range(w):
                dw[:, k] += (g * e[:, k:k + n]).sum(1)
                de[:, k:k + n] += s["weight"][:, k:k + 1].double() * g
            if case["h0"]:
                de[:, n:] += f(s["dlast"][b])
            db += g.sum(1)
            dxs.append(de[:, w - 1:])
            dhs.append(de[:, :w - 1])
        out = dict(dx=torch.stack(dxs), dweight=dw, dbias=db)
        if case["h0"]:
            out["dh0"] = torch.stack(dhs)
        return out
    y, state = f(s["y"]), f(s["state"])
    slots, seen = s["slots"].tolist(), None
    if op in ("conv_packed", "scan_packed"):
        start, seen = s["start"].tolist(), s["seen"].tolist()
    if op == "conv_packed":
        for i, slot in enumerate(slots):
            x = f(s["x"][start[i]:start[i + 1]]).t()
            v, last = _x_conv(state[slot] * (1 if seen[i] else 0), x, s["weight"], s["bias"])
            y[start[i]:start[i + 1]] = (v * torch.sigmoid(v)).t()
            state[slot] = last
        return dict(y=y, state=state)
    if op == "conv_step":
        for i in range(s["live"]):
            v, last = _x_conv(state[slots[i]], f(s["x"][i])[:, None], s["weight"], s["bias"])
            y[i] = (v * torch.sigmoid(v))[:, 0]
            state[slots[i]] = last
        return dict(y=y, state=state)
    soft = torch.nn.functional.softplus
    A, D, bias = f(s["A"]), f(s["D"]), f(s["delta_bias"])
    if op == "scan_packed":
        some = max(1, min(2048, (1 << 28) // (dim * N)))
        for i, slot in enumerate(slots):
            h = state[slot] * (1 if seen[i] else 0)
            for lo in range(start[i], start[i + 1], some):
                hi = min(start[i + 1], lo + some)
                u = f(s["u"][lo:hi])
                d = soft(f(s["delta"][lo:hi]) + bias, threshold=1000.0)
                a, hs = torch.exp(d[..., None] * A), (d * u)[..., None] * f(s["B"][lo:hi])[:, None]
                for j in range(hi - lo):
                    h = hs[j].addcmul_(a[j], h)
                v = torch.einsum("tdn,tn->td", hs, f(s["C"][lo:hi])) + D * u
                if s["z"] is not None:
                    z = f(s["z"][lo:hi])
                    v = v * z * torch.sigmoid(z)
                y[lo:hi] = v
            state[slot] = h
        return dict(y=y, state=state)
    for i in range(s["live"]):
        u, d, z = f(s["u"][i]), soft(f(s["delta"][i]) + bias, threshold=1000.0), f(s["z"][i])
        Dx = D
        if case["form"] == "scalar":
            d, Dx = d.repeat_interleave(64), D.repeat_interleave(64)
            a = torch.exp(d * A.repeat_interleave(64))[:, None]
        else:
            a = torch.exp(d[:, None] * A)
        h = a * state[slots[i]].reshape(dim, -1) + (d * u)[:, None] * f(s["B"][i])
        y[i] = (h @ f(s["C"][i]) + Dx * u) * z * torch.sigmoid(z)
        state[slots[i]] = h.reshape(state.shape[1:])
    return dict(y=y, state=state)
