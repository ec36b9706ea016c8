"""Plain 64-bit forms of the router, the layer and the adapter projection, with
the bounds that fp32 accumulation and the stated roundings give them.

Rounding: a sum of n products in fp32, in any order, is off by at most
n 2^-24 times the sum of the magnitudes, to first order; the tests allow twice
that (EPS). A result in bf16 (8 significant bits) is off by 2^-8 of itself at
most, one in fp32 by 2^-24.
"""

import torch

EPS = 2.0 ** -23
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -23}


def f64(t):
    return t.detach().cpu().double()


def inputs(gen, *shape, dtype, std=1.0):
    return (torch.randn(*shape, generator=gen, dtype=torch.float32) * std).to(dtype)


def route(x, gate, K, bias=None, score="softmax", renorm=True, scale=1.0):
    """(idx, weights, bound of the weights, keys) in 64 bits."""
    x, gate = f64(x), f64(gate)
    logits = x @ gate.t()
    off = x.shape[1] * EPS * (x.abs() @ gate.abs().t()).max(1, keepdim=True)[0]
    p = torch.softmax(logits, 1) if score == "softmax" else torch.sigmoid(logits)
    keys = logits if bias is None else p + f64(bias)
    idx = torch.sort(keys, dim=1, descending=True, stable=True)[1][:, :K]
    w = p.gather(1, idx)
    if renorm:
        w = w / w.sum(1, keepdim=True)
    w = w * scale
    # a logit that is off by `off` changes a score by a factor within
    # exp(+-2 off), with renorm twice that; exp, sums and division add ulps
    return idx, w, w.abs() * (8 * off + 64 * EPS), keys


def layer(x, idx, w, w1, w2, begin, few=True):
    """(y, bound) of the experts' weighted sum for given routes, in 64 bits."""
    dt = x.dtype
    x, w1, w2 = f64(x), f64(w1), f64(w2)
    idx, w = idx.cpu(), f64(w)
    T, H = x.shape
    E, I = w1.shape[0], w1.shape[1] // 2
    y = torch.zeros(T, H, dtype=torch.float64)
    mag = torch.zeros(T, H, dtype=torch.float64)     # of the terms, for the sums' errors
    part = torch.zeros(T, H, dtype=torch.float64)    # of the experts' outputs, for roundings
    for e in range(E):
        t, k = (idx == begin + e).nonzero(as_tuple=True)
        if not t.numel():
            continue
        c = w[t, k][:, None]
        gu = x[t] @ w1[e].t()
        au = x[t].abs() @ w1[e].abs().t()
        g, u = gu[:, :I], gu[:, I:]
        h = g * torch.sigmoid(g) * u
        # |d silu| <= 1.1 |dg|
        hm = 1.1 * au[:, :I] * u.abs() + g.abs() * au[:, I:]
        y[t] += c * (h @ w2[e].t())
        mag[t] += c.abs() * (hm @ w2[e].abs().t())
        part[t] += c.abs() * (h.abs() @ w2[e].abs().t())
    bound = U[dt] * y.abs() + (H + I * idx.shape[1] + 64) * EPS * mag
    if dt == torch.bfloat16:
        # h as two bf16 numbers: 16 bits; more than 64 rows: h and the experts'
        # outputs are rounded to bf16
        bound = bound + (2.0 ** -15 if few else 2.0 ** -7) * part
    return y, bound


def adapter(x, w, a, b, ids, scales=None):
    """(y, bound) of the shared projection with adapters, in 64 bits."""
    dt = x.dtype
    x, w, a, b = f64(x), f64(w), f64(a), f64(b)
    ids = ids.cpu()
    T, H = x.shape
    y = x @ w.t()
    mag = x.abs() @ w.abs().t()
    low = torch.zeros_like(y)
    for i in range(a.shape[0]):
        t = (ids == i).nonzero()[:, 0]
        if not t.numel():
            continue
        s = 1.0 if scales is None else float(scales[i])
        v = x[t] @ a[i].t()
        y[t] += s * (v @ b[i].t())
        mag[t] += abs(s) * ((x[t].abs() @ a[i].abs().t()) @ b[i].abs().t())
        low[t] += abs(s) * (v.abs() @ b[i].abs().t())
    bound = U[dt] * y.abs() + (H + a.shape[1] + 64) * EPS * mag
    if T > 64:
        bound = bound + U[dt] * low    # the low-rank product in the storage type
    return y, bound


def check(got, want, bound, what):
    got = f64(got)
    assert got.shape == want.shape, what
    assert torch.isfinite(got).all(), what
    over = (got - want).abs() - bound
    worst = int(over.argmax())
    assert over.max() <= 0, (f"{what}: off by {float((got - want).abs().flatten()[worst]):.3e} where "
                             f"{float(bound.flatten()[worst]):.3e} is allowed")
