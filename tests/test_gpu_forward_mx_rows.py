"""forward_mx where the plan has room for 256-row tiles: two kernels are launched, and the rows that
the segments hold say which of them works (64-row tiles below 56 rows an expert that has any).
Counts on both sides of that border and at it, against 64 bits, with every number of h and O
overwritten before, so that a tile that no kernel took shows.

The error, norm-wise: h in 8 bits is that of exact sums but for elements near a border, some
2^-8 of its norm at most (tests/test_gpu_mx_close.py); O is rounded to bf16 (2^-9 of each number),
and so is y; sums are off by less. In all below 2^-7 of y's norm. A row's norm may hang on one element
of h, silu(g) u with both large, say 0.3 of it; at a border this moves by a step, 2^-3 of itself at
most, so a row is allowed 2^-6 and the largest such step, 2^-3 |h_i| times the norm of w2's column i.
"""

import pytest
import torch

import top_reduce_amd as tr
from tests import _mx as M
from tests import _serving as S
from tests._gpu import say

pytestmark = pytest.mark.gpu
SHARE = 56

COUNTS = [[20, 30, 25, 10], [200, 3, 5, 6], [200, 3, 5, 0], [56, 56, 56, 56], [56, 56, 56, 55], [56, 57, 56, 56],
          [0, 55, 0, 0], [0, 56, 0, 0], [0, 0, 0, 57], [1, 0, 0, 0], [0, 0, 0, 0], [0, 111, 0, 0], [110, 0, 0, 1],
          [65, 1, 1, 150], [64, 64, 64, 31], [63, 65, 40, 55], [0, 300, 20, 700], [513, 2, 0, 1]]


def weights(g, E, N, K, bits):
    q, s = M.quantize(torch.randn(E, N, K, generator=g, dtype=torch.float64) * K ** -0.5, bits)
    return q.cuda(), s.cuda()


@pytest.fixture(scope="module")
def layers():
    return {}


def layer(layers, H, I, bits):
    """Weights of four experts, and their 64-bit values: made once for all counts."""
    if (H, I, bits) not in layers:
        g = torch.Generator().manual_seed(H + bits)
        w1, w2 = weights(g, 4, 2 * I, H, bits), weights(g, 4, H, I, bits)
        layers[H, I, bits] = (w1, w2, M.value(*w1).float().cuda(), M.value(*w2).float().cuda())
    return layers[H, I, bits]


@pytest.mark.parametrize("H,I", [(256, 2048), (4096, 256)])     # the rule's 256-row tiles: up; down
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("counts", COUNTS)
def test_the_rows_there(layers, H, I, bits, counts):
    T, K, E = 1024, 2, 4
    total, some = sum(counts), sum(c > 0 for c in counts)
    say(f"forward {counts} H={H} I={I} bits={bits}: {total} of {T * K} rows, "
        f"{'64' if total < SHARE * some else '256'}-row tiles")
    g = torch.Generator().manual_seed(total + bits)
    w1, w2, v1, v2 = layer(layers, H, I, bits)
    x = M.quantize(torch.randn(T, H, generator=g, dtype=torch.float64))
    idx = torch.full((T * K,), -1, dtype=torch.int64)
    at = torch.randperm(T * K, generator=g)[:total]
    idx[at] = torch.repeat_interleave(torch.arange(E), torch.tensor(counts))
    idx = idx.view(T, K)
    w = torch.rand(T, K, generator=g) + 0.5
    p = tr.plan(idx.cuda(), E=E, H=H, I=I)
    v = p.views()
    assert (v["offsets"][1:] - v["offsets"][:-1]).tolist() == counts
    v["h"].view(torch.uint8).fill_(0x7f)     # NaN as elements; a scale of 1 / 65536
    v["O"].fill_(float("nan"))
    y = tr.forward_mx(p, tuple(t.cuda() for t in x), w.cuda(), w1, w2)
    want = torch.zeros(T, H, dtype=torch.float64)
    step = torch.zeros(T, dtype=torch.float64)
    xv = M.value(*x)
    for e in range(E):
        t, k = (idx == e).nonzero(as_tuple=True)
        if not t.numel():
            continue
        # (products of 8-bit numbers are exact in 64 bits; the weights are held in fp32, exactly)
        gu = xv[t].cuda() @ v1[e].double().t()
        h = (gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]).cpu()
        o = (M.value(*M.quantize(h)).cuda() @ v2[e].double().t()).cpu()
        want.index_add_(0, t, w.double()[t, k][:, None] * o)
        step.index_add_(0, t, w.double()[t, k] * 2.0 ** -3 * (h.abs() * v2[e].double().norm(dim=0).cpu()).amax(1))
    got = S.f64(y)
    assert torch.isfinite(got).all()
    here = (idx >= 0).any(1)
    assert (got[~here] == 0).all()
    off, size = got - want, want.norm(dim=1)
    assert float(off.norm()) <= 2.0 ** -7 * float(want.norm()) and (off.norm(dim=1) <= 2.0 ** -6 * size + step).all()
    # bit for bit what the products of these rows alone give; the one that has no 256-row tiles here is
    # of 32-row ones, by the host's rule
    if total:
        up, down = ("tile64", "tile32") if I > H else ("tile32", "tile64")
        hh = tr.expert_linear(tuple(t.cuda() for t in x), w1, v["offsets"], rows=v["row_src"][:total].contiguous(),
                              swiglu=True, out="mx8", kernel=up)
        full = torch.zeros(T * K, H, dtype=torch.bfloat16, device="cuda")
        full[:total] = tr.expert_linear(hh, w2, v["offsets"], kernel=down)
        assert torch.equal(tr.combine_reduce(p, w.cuda(), expert_out=full), y)
