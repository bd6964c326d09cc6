"""Plain fp64 numpy forms of the operators around the scan, for the tests:
the short causal convolution (forward, gradients, one sequence after its past)
and the diagonal scan of one sequence, token by token."""
import numpy as np


def sigmoid(v):
    """Without cancellation on either side."""
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


def conv(x, weight, bias=None, silu=True, h0=None):
    """x (..., D, L), weight (D, W), h0 (..., D, W-1).  Returns y, the last
    W-1 inputs, and the sum of absolute terms of each pre-activation (what
    fp32 rounding errors scale with)."""
    x = np.asarray(x, np.float64)
    D, W = weight.shape
    w = np.asarray(weight, np.float64)
    past = np.zeros(x.shape[:-1] + (W - 1,)) if h0 is None else np.asarray(h0, np.float64)
    e = np.concatenate([past, x], -1)
    L = x.shape[-1]
    b = np.zeros(D) if bias is None else np.asarray(bias, np.float64)
    v = np.zeros_like(x) + b[:, None]
    size = np.zeros_like(x) + np.abs(b)[:, None]
    for k in range(W):
        v = v + w[:, k:k + 1] * e[..., k:k + L]
        size = size + np.abs(w[:, k:k + 1] * e[..., k:k + L])
    y = v * sigmoid(v) if silu else v
    return y, e[..., L:], size


def conv_grads(x, weight, dy, bias=None, silu=True, h0=None, dlast=None):
    """Gradients of sum(dy y) + sum(dlast last): dx, dh0, dweight, dbias, and
    the sums of absolute terms of dx|dh0 and dweight."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    D, W = weight.shape
    w = np.asarray(weight, np.float64)
    L = x.shape[-1]
    past = np.zeros(x.shape[:-1] + (W - 1,)) if h0 is None else np.asarray(h0, np.float64)
    e = np.concatenate([past, x], -1)
    g, gsize = dy, np.abs(dy)
    if silu:
        v = np.zeros_like(x) + (0 if bias is None else np.asarray(bias, np.float64)[:, None])
        size = np.abs(v)
        for k in range(W):
            v = v + w[:, k:k + 1] * e[..., k:k + L]
            size = size + np.abs(w[:, k:k + 1] * e[..., k:k + L])
        s = sigmoid(v)
        g = dy * (s + v * s * (1 - s))
        gsize = np.abs(dy) * (1 + size)
    de, desize = np.zeros_like(e), np.zeros_like(e)
    dw, dwsize = np.zeros((D, W)), np.zeros((D, W))
    lead = tuple(range(x.ndim - 2))
    for k in range(W):
        de[..., k:k + L] += w[:, k:k + 1] * g
        desize[..., k:k + L] += np.abs(w[:, k:k + 1]) * gsize
        dw[:, k] = (g * e[..., k:k + L]).sum(lead + (-1,))
        dwsize[:, k] = (gsize * np.abs(e[..., k:k + L])).sum(lead + (-1,))
    if dlast is not None:
        de[..., L:] += dlast
        desize[..., L:] += np.abs(dlast)
    return dict(dx=de[..., W - 1:], dh0=de[..., :W - 1], dweight=dw, dbias=g.sum(lead + (-1,)),
                dxsize=desize[..., W - 1:], dh0size=desize[..., :W - 1], dwsize=dwsize,
                dbsize=gsize.sum(lead + (-1,)))


def scan(u, delta, A, B, C, D=None, z=None, delta_bias=None, softplus=True, h0=None):
    """One sequence, token-major: u, delta, z (T, D), B, C (T, N)."""
    u, delta = np.asarray(u, np.float64), np.asarray(delta, np.float64)
    A, B, C = (np.asarray(a, np.float64) for a in (A, B, C))
    h = np.zeros(A.shape) if h0 is None else np.array(h0, np.float64)
    d = delta if delta_bias is None else delta + np.asarray(delta_bias, np.float64)
    if softplus:
        d = np.logaddexp(0.0, d)
    y = np.zeros_like(u)
    for t in range(u.shape[0]):
        h = np.exp(d[t][:, None] * A) * h + (d[t] * u[t])[:, None] * B[t][None]
        y[t] = h @ C[t]
    if D is not None:
        y = y + np.asarray(D, np.float64) * u
    if z is not None:
        z = np.asarray(z, np.float64)
        y = y * z * sigmoid(z)
    return y, h
