"""Plain 64-bit forms of the operators on blocks of 32 with scales, and the bounds of
their results.

A number in blocks is compared with its 64-bit value v: the kernel rounds a value that is
off v by a given err at most, to a scale s and an element of 4 (8 bits) or 2 (4 bits)
significant bits. s is one of the scales that magnitudes within err of the block's largest
have; the number is off by half a step of its binade and err.
"""

import torch

from tests._serving import EPS, U, f64

E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
MOST = {8: 448.0, 4: 6.0}
E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def value(q, s):
    """The numbers that (q, s) stands for, in 64 bits."""
    q, s = q.cpu(), s.cpu().view(torch.uint8).double()
    if q.dtype == torch.uint8:
        q = E2M1[torch.stack([q & 15, q >> 4], -1).long()].flatten(-2)
    power = torch.where(s == 255, float("nan"), torch.exp2(s - 127))
    return q.double() * power.repeat_interleave(32, -1)


def scale_byte(top, bits):
    """The scale of a block of that largest magnitude: 2^(byte - 127)."""
    m, e = torch.frexp(top.double() / MOST[bits])     # m in [1/2, 1), exact but at 448 and 6
    e = torch.where(m == 0.5, e - 1, e)
    return torch.where(top == 0, 0, (e + 127).clamp(0, 254))


def quantize(v, bits=8):
    """(q, s) of 64-bit (or exact) numbers v."""
    v = f64(v)
    b = v.unflatten(-1, (-1, 32))
    fine = b.isfinite()
    byte = scale_byte(torch.where(fine, b.abs(), 0.0).amax(-1), bits)
    b = b * torch.exp2(127.0 - byte)[..., None]
    if bits == 8:
        q = torch.where(fine, b, float("nan")).float().to(E4M3).flatten(-2)
        return q, byte.to(torch.uint8).view(E8M0)
    byte = torch.where(fine.all(-1), byte, 255)
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)
    a = torch.where(fine.all(-1, keepdim=True), b.abs(), 0.0)
    code = torch.bucketize(a, mid)     # ties: to the lower one
    odd = (code % 2 == 1) & (code < 7)
    tie = odd & (a == mid[code.clamp(max=6)])
    code = code + tie + 8 * (torch.signbit(b) & fine.all(-1, keepdim=True))
    code = code.to(torch.uint8).flatten(-2).unflatten(-1, (-1, 2))
    return code[..., 0] + 16 * code[..., 1], byte.to(torch.uint8).view(E8M0)


def check_blocks(got, want, err, what, bits=8):
    """(q, s) against 64-bit values `want` that the kernel had within err."""
    q, s = got
    v = value(q, s)
    assert v.shape == want.shape, what
    err = err.expand_as(want) if isinstance(err, torch.Tensor) else torch.full_like(want, err)
    byte = s.cpu().view(torch.uint8).long()
    b, d = want.abs().unflatten(-1, (-1, 32)), err.unflatten(-1, (-1, 32))
    low = scale_byte((b - d).clamp(min=0).amax(-1), bits)
    high = scale_byte((b + d).amax(-1), bits)
    assert ((byte >= low) & (byte <= high)).all(), f"{what}: scales"
    power = torch.exp2(byte.double() - 127).repeat_interleave(32, -1)
    least, digits = (2.0 ** -6, 3) if bits == 8 else (1.0, 1)
    binade = torch.floor(torch.log2(((want.abs() + err) / power).clamp(min=least)))
    bound = torch.exp2(binade - digits) * power / 2 + err
    over = (v - want).abs() - bound
    assert (over <= 0).all(), f"{what}: off by {float(over.max()):.3e} more than allowed"


def rms_norm(x, weight, eps, residual=None):
    """(y, z, bound of y before its rounding). A thread sums at most 33 numbers a row of
    32768 and less, then 6 and 16 sums: 55 2^-24 of the sum of squares and half that of its
    root; z, the root, the division and two products: 6 ulps."""
    z = f64(x) if residual is None else f64(x) + f64(residual)
    y = z / torch.sqrt(z.square().mean(1, keepdim=True) + eps) * f64(weight)
    terms = max(33, x.shape[1] // 1024 + 8)
    return y, z, ((terms + 22) / 2 + 6) * 2.0 ** -24 * y.abs()


def products(x, w, offsets, rows=None, swiglu=False, tiled=0.0):
    """(y, bound before rounding) in 64 bits of the rows in the segments; x [T, K] and
    w [E, N, K] in 64 bits. tiled: what a matrix instruction drops, relative to the sum of
    the products' magnitudes."""
    offsets = offsets.tolist()
    R = x.shape[0] if rows is None else rows.shape[0]
    K, N = x.shape[1], w.shape[1]
    x = x if rows is None else x[rows.long().clamp(0, x.shape[0] - 1).cpu()]
    outs = N // 2 if swiglu else N
    y = torch.zeros(R, outs, dtype=torch.float64)
    err = torch.zeros(R, outs, dtype=torch.float64)
    inside = torch.zeros(R, dtype=torch.bool)
    for e in range(w.shape[0]):
        a = min(max(offsets[e], 0), R)
        b = min(max(offsets[e + 1], a), R)
        if a == b:
            continue
        inside[a:b] = True
        p = x[a:b] @ w[e].t()
        d = ((K + 64) * EPS + tiled) * (x[a:b].abs() @ w[e].abs().t())
        if swiglu:
            g, u, dg, du = p[:, :outs], p[:, outs:], d[:, :outs], d[:, outs:]
            s = g * torch.sigmoid(g)
            p = s * u
            # |d silu| <= 1.1 |dg|; exp, reciprocal and products: 16 ulps
            d = 1.1 * dg * (u.abs() + du) + s.abs() * du + 16 * EPS * p.abs()
        y[a:b], err[a:b] = p, d
    return y, err, inside


def check_rows(got, want, err, inside, what):
    """bf16 results of the rows in the segments."""
    got, want, err = f64(got)[inside], want[inside], err[inside]
    assert torch.isfinite(got).all(), what
    bound = err + U[torch.bfloat16] * (want.abs() + err)
    over = (got - want).abs() - bound
    assert (over <= 0).all(), f"{what}: off by {float(over.max()):.3e} more than allowed"
