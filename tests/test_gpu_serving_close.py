"""The router, the layer and the projection against 64-bit values by the norm-wise
checks of tests/_close.py."""

import pytest
import torch

import top_reduce_amd as tr
from tests import _close as C
from tests import _serving as S
from tests._gpu import say

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("T,H,I,E,G,K,begin", [
    (1, 256, 128, 8, 8, 2, 0), (2, 264, 72, 6, 12, 3, 6), (7, 136, 70, 5, 5, 2, 0), (15, 512, 257, 8, 16, 4, 8),
    (16, 256, 128, 8, 8, 8, 0), (17, 1032, 33, 3, 9, 2, 3), (33, 2880, 40, 4, 4, 3, 0), (48, 64, 16, 300, 400, 6, 50),
    (64, 512, 128, 8, 64, 8, 56), (64, 72, 8, 70, 70, 32, 0), (29, 264, 130, 5, 10, 4, 5), (64, 128, 66, 66, 66, 5, 0),
    (20, 512, 160, 4, 4, 2, 0), (40, 256, 99, 6, 12, 4, 6), (64, 136, 257, 3, 3, 3, 0), (64, 256, 70, 5, 10, 8, 5),
    (33, 128, 64, 1, 1, 1, 0), (64, 256, 2048, 2, 2, 2, 0),    # many tokens an expert
    (8, 264, 2056, 16, 16, 4, 0), (8, 512, 2051, 16, 16, 4, 0), (9, 136, 1030, 40, 40, 5, 0),
    (64, 72, 1536, 24, 24, 6, 0), (1, 96, 1800, 32, 32, 32, 0), (64, 256, 2048, 8, 8, 4, 0),    # in parts
    (3, 4096, 24, 4, 4, 2, 0), (3, 4104, 24, 4, 4, 2, 0), (3, 7168, 24, 4, 4, 2, 0), (40, 2880, 800, 16, 16, 4, 0),
])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_layer(T, H, I, E, G, K, begin, dtype):
    say(f"layer close T={T} H={H} I={I} E={E} G={G} K={K} {dtype}")
    g = torch.Generator().manual_seed(T + H + I)
    x = S.inputs(g, T, H, dtype=dtype)
    gate = S.inputs(g, G, H, dtype=dtype, std=1.5 * H ** -0.5)
    w1 = S.inputs(g, E, 2 * I, H, dtype=dtype, std=H ** -0.5)
    w2 = S.inputs(g, E, H, I, dtype=dtype, std=I ** -0.5)
    y, idx, w = tr.layer(x.cuda(), gate.cuda(), w1.cuda(), w2.cuda(), K, expert_begin=begin, scale=1.5)
    want, _ = S.layer(x, idx, w, w1, w2, begin)
    C.check(y, want, H + I * K, dtype, "y")


@pytest.mark.parametrize("T", [65, 128, 300])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_layer_of_more_rows(T, dtype):
    """From 65 rows h and the experts' outputs are rounded to bf16: each is off by
    2^-9 of itself at most, and so is their sum."""
    H, I, E, G, K, begin = 512, 256, 8, 16, 4, 4
    g = torch.Generator().manual_seed(T)
    x = S.inputs(g, T, H, dtype=dtype)
    gate = S.inputs(g, G, H, dtype=dtype, std=1.5 * H ** -0.5)
    w1 = S.inputs(g, E, 2 * I, H, dtype=dtype, std=H ** -0.5)
    w2 = S.inputs(g, E, H, I, dtype=dtype, std=I ** -0.5)
    y, idx, w = tr.layer(x.cuda(), gate.cuda(), w1.cuda(), w2.cuda(), K, expert_begin=begin)
    want, _ = S.layer(x, idx, w, w1, w2, begin)
    C.check(y, want, H + I * K, dtype, "y", wide=2.0 ** -7 if dtype == BF else 0.0)


@pytest.mark.parametrize("T,H,N,R,A,run,dtype", [
    (1, 3584, 512, 16, 8, 1, BF), (8, 264, 1000, 8, 3, 1, BF), (16, 256, 256, 12, 16, 1, BF),
    (5, 7176, 6001, 20, 3, 1, BF), (16, 7168, 7160, 20, 3, 1, BF), (16, 4104, 8200, 20, 3, 1, F32),
    (1, 4104, 8200, 20, 3, 1, F32), (17, 1032, 33, 64, 40, 1, BF), (63, 512, 515, 100, 4, 5, BF),
    (64, 512, 256, 256, 64, 1, BF), (130, 264, 129, 12, 3, 7, BF), (300, 1032, 250, 64, 8, 1, BF),
    (513, 2880, 1001, 256, 4, 100, BF), (64, 72, 256, 64, 9, 3, F32), (200, 1448, 301, 12, 5, 40, F32),
    (256, 256, 256, 256, 3, 1, F32), (333, 1448, 1001, 12, 5, 40, F32),
    (1000, 512, 2050, 24, 4, 300, BF), (1000, 520, 4100, 16, 5, 1, BF), (2048, 264, 4100, 33, 3, 500, BF),
    (1000, 520, 4100, 16, 5, 50, F32), (2048, 264, 4100, 33, 3, 500, F32),
    (4096, 256, 8192, 16, 5, 700, BF), (4090, 384, 8192, 40, 9, 1, BF),
])
def test_projection(T, H, N, R, A, run, dtype):
    say(f"projection close T={T} H={H} N={N} R={R} A={A} run={run} {dtype}")
    g = torch.Generator().manual_seed(T + N)
    ids = torch.randint(-1, A + 1, (-(-T // run),), generator=g, dtype=torch.int32)
    ids = ids.repeat_interleave(run)[:T].contiguous()
    x, w = S.inputs(g, T, H, dtype=dtype), S.inputs(g, N, H, dtype=dtype, std=H ** -0.5)
    a = S.inputs(g, A, R, H, dtype=dtype, std=H ** -0.5)
    b = S.inputs(g, A, N, R, dtype=dtype, std=R ** -0.5)
    scales = torch.rand(A, generator=g) + 0.5
    y = tr.adapter_linear(x.cuda(), w.cuda(), a.cuda(), b.cuda(), ids.cuda(), scales=scales.cuda())
    want, _ = S.adapter(x, w, a, b, ids, scales)
    C.check(y, want, H + R, dtype, "y")


def exact_inputs(seed, T, H, G, dtype):
    """Small integers (times 1/8): every logit is exact in fp32 in any order of the
    sum, and many are equal."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(-2, 3, (T, H), generator=g).to(dtype)
    w = (torch.randint(-1, 2, (G, H), generator=g) / 8).to(dtype)
    return x, w


# exp, the sums' 64 + 6 and 6 roundings, division and scale: a few ulp and at most
# 76 half ulps; half as much again
WEIGHT = 64 * 2.0 ** -23


@pytest.mark.parametrize("T,H,G,K", [
    (1, 8, 1, 1), (1, 3584, 896, 16), (2, 264, 63, 3), (16, 256, 64, 8), (17, 40, 65, 32), (33, 2880, 257, 5),
    (64, 7168, 256, 8), (65, 136, 60, 4), (300, 1032, 130, 7), (1000, 512, 1025, 9), (5, 16, 4096, 32),
    (700, 1024, 512, 16), (16, 264, 32, 9), (100, 1000, 32, 32), (333, 2040, 16, 2), (4096, 40, 9, 3),
    (8192, 264, 256, 8),
])
@pytest.mark.parametrize("score,renorm,bias", [("softmax", True, False), ("sigmoid", False, False),
                                               ("softmax", False, True), ("sigmoid", True, True)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_router_weights_of_exact_logits(T, H, G, K, score, renorm, bias, dtype):
    """The logits are exact, so that the weights are off by what the scores' own
    functions are off by."""
    say(f"router close T={T} H={H} G={G} K={K} {score} {dtype}")
    x, gate = exact_inputs(T + G, T, H, G, dtype)
    # a bias that orders all experts alike for every row, far apart: no ties
    b = -torch.arange(G, dtype=torch.float32).flip(0) * 2 if bias else None
    idx, w = tr.route_topk(x.cuda(), gate.cuda(), K, bias=None if b is None else b.cuda(), score=score,
                           renorm=renorm, scale=1.5)
    logits = S.f64(x) @ S.f64(gate).t()
    p = torch.softmax(logits, 1) if score == "softmax" else torch.sigmoid(logits)
    keys = logits if b is None else p + S.f64(b)
    ref = torch.sort(keys, dim=1, descending=True, stable=True)[1][:, :K]
    assert torch.equal(idx.cpu(), ref)
    want = p.gather(1, ref)
    # (scores that are no normal floats count by their fp32 value)
    small = want < 2.0 ** -120
    total = want.sum(1, keepdim=True)
    ok = ~small & (total > 2.0 ** -110)
    if renorm:
        want = want / total
    want = want * 1.5
    assert ok.float().mean() > 0.5
    assert ((S.f64(w) - want).abs() <= WEIGHT * want)[ok].all()
    assert (S.f64(w) >= 0).all() and (S.f64(w) <= 1.5 * (1 + WEIGHT)).all()
