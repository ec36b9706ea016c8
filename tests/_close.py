"""Norm-wise checks of computed numbers against 64-bit values, beside the worst-case
bounds of tests/_serving.py: those hold for any order of a sum, these are what sums of
random terms come to, so that a part left out or an operand held in fewer bits shows.

An fp32 sum of n random terms, each partial sum rounded, is off by about sqrt(n) 2^-25
of its size; eps = (sqrt(n) + 16) 2^-23 is four times that, with room for the functions
between two sums.

A result in bf16 is compared with the 64-bit value rounded to bf16: the two are equal
unless that value lies within the error before the rounding of a midpoint, and then
they are an ulp apart. With an error of e |y| before the rounding the chance is
2 e |y| / ulp and the square of the difference ulp^2, ulp <= 2^-7 |y|: the sum of the
squares is at most 2^-6 e |y|^2. e is eps, and 2^-17 for a factor that is held in 16
significant bits (8 bits: 2^-9, sixteen times the difference). A few elements may by
chance all be at a midpoint: FLIPS of them.

The sizes are those of rows and blocks of a few dozen elements and more: a row of one
or two may come out near zero, far below what its sums went through.
"""

import torch

FLIPS = 4


def f64(t):
    return t.detach().cpu().double()


def groups(t):
    """Whole, by rows, and by blocks of 16 columns: [groups, elements]."""
    yield "all", t.reshape(1, -1)
    yield "row", t
    for c in range(0, t.shape[1], 16):
        yield f"columns {c}..", t[:, c:c + 16].reshape(1, -1)


def misses(got, want, n, dtype, bits16=True, wide=0.0):
    """The group that is off by more than it may be, or None. n: terms of a sum;
    bits16: a factor is held in 16 bits (bf16 only); wide: a relative error that
    the operator allows itself beside these."""
    got, want = f64(got), f64(want)
    assert got.shape == want.shape
    eps = (n ** 0.5 + 16) * 2.0 ** -23
    if dtype == torch.bfloat16:
        want = want.to(torch.bfloat16).double()
        e = eps + (2.0 ** -17 if bits16 else 0.0)
    for (name, d), (_, w) in zip(groups(got - want), groups(want)):
        size, top = w.square().sum(1), w.square().amax(1)
        if dtype == torch.bfloat16:
            allowed = (2.0 ** -6 * e + wide ** 2) * size + FLIPS * 2.0 ** -14 * top
        else:
            allowed = (eps + wide) ** 2 * size
        over = ~(d.square().sum(1) <= allowed)      # (NaN too)
        if over.any():
            at = int(over.nonzero()[0])
            return (f"{name} {at}: off by {float(d[at].norm() / w[at].norm()):.2e} of its norm, "
                    f"{float((allowed[at] / size[at]).sqrt()):.2e} allowed")
    return None


def check(got, want, n, dtype, what, **kw):
    miss = misses(got, want, n, dtype, **kw)
    assert miss is None, f"{what}: {miss}"
