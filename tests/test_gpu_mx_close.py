"""Norm-wise checks of expert_linear's results, beside the worst-case bounds of
tests/test_gpu_expert_linear.py, which for thousands of random products leave room for a few
hundredths of a result: a part of a sum left out, held in bf16 or read too early shows here.

The tiles' matrix instructions are documented to be off by 1.5e-5 of a sum's norm. As everywhere
in tests/_close.py four times that is allowed, E = 2^-14. Rounded to bf16 a result that is off by
E |y| differs from the rounded exact one in squares of at most 2^-6 E |y|^2 (tests/_close.py):
`wide` = sqrt(2^-6 2^-14) = 2^-10 beside an fp32 sum's.

In 8 bits an element of step d <= 2^-3 |y| that is off by e moves to a neighbour with a chance of
|e| / d, and the square of the difference is d^2: |e| d on the average, at most 2^-3 E |y|^2 summed.
With swiglu two sums enter a product and silu's slope is 1.1 at most: E sqrt(2) 1.1 < 2^-13. Its
root, sqrt(2^-3 2^-13) = 2^-8, is a sixth of the format's own rounding. Sums kept in bf16 (2^-9 of
each part, 1.1e-3 of the norm) would be off by 1.2e-2 of the norm, and in bf16 results by 4e-3.
"""

import pytest
import torch

import top_reduce_amd as tr
from tests import _close as C
from tests import _mx as M
from tests import _serving as S
from tests._gpu import say

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
KERNELS = ["rows", "tile32", "tile64", "tile256"]
SIZES = [([5, 11], 2880, 512), ([1, 15, 0, 33], 7168, 256), ([70, 200], 1024, 320), ([300, 64, 20], 4096, 256),
         ([130], 8480, 128), ([513, 40], 288, 192), ([256, 255], 2048, 512)]


def made(counts, K, N, bits):
    g = torch.Generator().manual_seed(K + N + bits)
    R, E = sum(counts), len(counts)
    x = M.quantize(torch.randn(R, K, generator=g, dtype=torch.float64))
    w = M.quantize(torch.randn(E, N, K, generator=g, dtype=torch.float64) * K ** -0.5, bits)
    offsets = torch.tensor([0] + counts).cumsum(0).int()
    xv, wv = M.value(*x), M.value(*w)
    want = torch.cat([xv[offsets[e]:offsets[e + 1]] @ wv[e].t() for e in range(E)])
    return tuple(t.cuda() for t in x), tuple(t.cuda() for t in w), offsets.cuda(), want


@pytest.mark.parametrize("counts,K,N", SIZES)
@pytest.mark.parametrize("bits", [8, 4])
def test_bf16(counts, K, N, bits):
    x, w, offsets, want = made(counts, K, N, bits)
    g, u = want[:, :N // 2], want[:, N // 2:]
    for kernel in KERNELS:
        say(f"experts {counts} K={K} N={N} bits={bits} {kernel}")
        wide = 0.0 if kernel == "rows" else 2.0 ** -10
        C.check(tr.expert_linear(x, w, offsets, kernel=kernel), want, K, BF, kernel, bits16=False, wide=wide)
        # (two factors: twice the square; silu's functions add 16 ulps of fp32, in eps)
        h = tr.expert_linear(x, w, offsets, swiglu=True, kernel=kernel)
        C.check(h, g * torch.sigmoid(g) * u, 4 * K, BF, kernel + " swiglu", bits16=False, wide=1.6 * wide)


@pytest.mark.parametrize("counts,K,N", SIZES)
@pytest.mark.parametrize("bits", [8, 4])
def test_8_bits(counts, K, N, bits):
    x, w, offsets, want = made(counts, K, N, bits)
    g, u = want[:, :N // 2], want[:, N // 2:]
    for kernel in KERNELS:
        say(f"experts {counts} K={K} N={N} bits={bits} {kernel}")
        for swiglu, v in ((False, want), (True, g * torch.sigmoid(g) * u)):
            got = M.value(*tr.expert_linear(x, w, offsets, swiglu=swiglu, out="mx8", kernel=kernel))
            exact = M.value(*M.quantize(v))
            off = float((got - exact).norm() / exact.norm())
            assert off <= 2.0 ** -8, f"{kernel} swiglu={swiglu}: off by {off:.2e} of the norm"
            assert float((got != exact).double().mean()) <= 2.0 ** -8      # of the elements


@pytest.mark.parametrize("T,K,N,bits", [(5, 2880, 512, 8), (64, 7168, 256, 4), (300, 1024, 320, 8)])
def test_these_checks_see_sums_kept_in_bf16(T, K, N, bits):
    """The same checks on results whose sums were rounded to bf16 once on the way: 2^-9 of a part of
    the size of a result, uniform."""
    _, _, _, want = made([T], K, N, bits)
    part = want + torch.randn_like(want) * want.abs().mean() * 2.0 ** -9 / 3 ** 0.5
    assert C.misses(part.to(BF), want, K, BF, bits16=False, wide=2.0 ** -10) is not None
    q = M.value(*M.quantize(part))
    exact = M.value(*M.quantize(want))
    assert float((q - exact).norm() / exact.norm()) > 2.0 ** -8
