"""The router (route_topk) against its formula in 64 bits."""

import pytest
import torch

import top_reduce_amd as tr
from tests import _serving as S
from tests._gpu import say

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def exact_inputs(seed, T, H, G, dtype):
    """Small integers (times 1/8): every logit is exact in fp32 in any order of
    the sum, and many are equal."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(-2, 3, (T, H), generator=g).to(dtype)
    w = (torch.randint(-1, 2, (G, H), generator=g) / 8).to(dtype)
    return x, w


@pytest.mark.parametrize("T,H,G,K,dtype", [
    (1, 8, 1, 1, BF), (1, 3584, 896, 16, BF), (2, 264, 63, 3, BF), (16, 256, 64, 8, BF),
    (17, 40, 65, 32, BF), (33, 2880, 257, 5, BF), (64, 7168, 256, 8, BF), (65, 136, 60, 4, BF),
    (300, 1032, 130, 7, BF), (1000, 512, 1025, 9, BF), (5, 16, 4096, 32, BF),
    (1, 256, 8, 2, F32), (64, 100 * 8, 60, 4, F32), (129, 264, 129, 6, F32), (500, 1024, 16, 16, F32),
])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("sigmoid", False)])
def test_ties_go_to_the_lowest_id(T, H, G, K, dtype, score, renorm):
    say(f"route ties T={T} H={H} G={G} K={K} {dtype} {score}")
    x, w = exact_inputs(T + G, T, H, G, dtype)
    idx, wt = tr.route_topk(x.cuda(), w.cuda(), K, score=score, renorm=renorm, scale=1.5)
    ref, rw, tol, _ = S.route(x, w, K, score=score, renorm=renorm, scale=1.5)
    assert torch.equal(idx.cpu(), ref)
    S.check(wt, rw, tol, "weights")


@pytest.mark.parametrize("T,H,G,K,dtype", [(3, 512, 32, 4, BF), (64, 1024, 256, 8, BF),
                                           (700, 2048, 256, 8, BF), (90, 264, 96, 6, F32)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_bias_decides_the_choice_only(T, H, G, K, dtype, score):
    g = torch.Generator().manual_seed(T + H)
    x = S.inputs(g, T, H, dtype=dtype)
    w = S.inputs(g, G, H, dtype=dtype, std=1.5 * H ** -0.5)
    bias = torch.randn(G, generator=g) * 0.05
    ref, rw, tol, keys = S.route(x, w, K, bias=bias, score=score)
    idx, wt = tr.route_topk(x.cuda(), w.cuda(), K, bias=bias.cuda(), score=score,
                            idx_dtype=torch.int32)
    assert idx.dtype == torch.int32
    # rows whose choice does not hang on fp32 rounding (scores are below 1)
    top = torch.sort(keys, dim=1, descending=True)[0][:, :K + 1]
    clear = ((top[:, :-1] - top[:, 1:]) > 1e-4).all(1)
    assert clear.sum() > 0.5 * T
    assert torch.equal(idx.cpu().long()[clear], ref[clear])
    S.check(wt.cpu()[clear], rw[clear], tol[clear], "weights")


def test_rows_of_infinities_and_nan():
    T, H, G, K = 6, 64, 40, 8
    g = torch.Generator().manual_seed(1)
    x = S.inputs(g, T, H, dtype=F32)
    w = S.inputs(g, G, H, dtype=F32, std=H ** -0.5)
    clean_idx, clean_w = tr.route_topk(x.cuda(), w.cuda(), K)
    bad = x.clone()
    bad[1, 3] = float("nan")
    bad[2, 5] = float("inf")
    bad[4] = 3e38
    for score in ("softmax", "sigmoid"):
        idx, wt = tr.route_topk(bad.cuda(), w.cuda(), K, score=score)
        idx = idx.cpu()
        assert ((idx >= 0) & (idx < G)).all()
        assert all(len(set(row.tolist())) == K for row in idx)
        if score == "softmax":
            for t in (0, 3, 5):     # the other rows do not notice
                assert torch.equal(idx[t], clean_idx.cpu()[t])
                assert torch.equal(wt.cpu()[t], clean_w.cpu()[t])
            assert idx[1].tolist() == list(range(K))     # all NaN: the lowest ids
            assert torch.isnan(wt.cpu()[1]).all()
    # one expert's logit NaN: it is the last to be chosen
    wn = w.clone()
    wn[0] = float("nan")
    idx, _ = tr.route_topk(x.cuda(), wn.cuda(), G if G <= 32 else 32)
    assert not (idx.cpu() == 0).any()


@pytest.mark.parametrize("T,H,G,K", [(1, 8, 1, 1), (16, 264, 32, 9), (17, 520, 17, 4), (100, 1000, 32, 32),
                                     (333, 2040, 16, 2), (4096, 40, 9, 3), (4097, 40, 9, 3)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_small_routers(T, H, G, K, dtype):
    x, w = exact_inputs(T + H, T, H, G, dtype)
    idx, wt = tr.route_topk(x.cuda(), w.cuda(), K, renorm=False)
    ref, rw, tol, _ = S.route(x, w, K, renorm=False)
    assert torch.equal(idx.cpu(), ref)
    S.check(wt, rw, tol, "weights")
    # a row that is not a number stays by itself
    bad = x.clone()
    bad[T // 2, H - 1] = float("nan")
    i2, w2 = tr.route_topk(bad.cuda(), w.cuda(), K, renorm=False)
    rest = torch.arange(T) != T // 2
    assert torch.equal(i2.cpu()[rest], idx.cpu()[rest]) and torch.equal(w2.cpu()[rest], wt.cpu()[rest])
    assert sorted(i2[T // 2].tolist()) == i2[T // 2].unique().tolist()


def test_scores_that_vanish():
    """All sigmoids 0: weights 0 with renorm, not NaN."""
    x = torch.full((2, 8), 10.0, dtype=F32)
    w = torch.full((5, 8), -10.0, dtype=F32)
    idx, wt = tr.route_topk(x.cuda(), w.cuda(), 3, score="sigmoid")
    assert idx.tolist() == [[0, 1, 2]] * 2 and wt.tolist() == [[0.0] * 3] * 2


def test_same_bits_with_a_dirty_workspace_another_stream_and_given_outputs():
    for T in (7, 200):
        x, w = exact_inputs(3, T, 512, 48, BF)
        x, w = x.cuda(), w.cuda()
        idx, wt = tr.route_topk(x, w, 6)
        n = tr.route_workspace_size(T, 512, 48, 6)
        ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        out = torch.empty_like(idx), torch.empty_like(wt)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        got = tr.route_topk(x, w, 6, idx=out[0], weights=out[1], ws=ws, stream=s)
        s.synchronize()
        assert got[0] is out[0] and got[1] is out[1]
        assert torch.equal(out[0], idx) and torch.equal(out[1], wt)


def test_no_rows():
    idx, wt = tr.route_topk(torch.empty(0, 64, dtype=BF, device="cuda"),
                            torch.zeros(9, 64, dtype=BF, device="cuda"), 2)
    assert idx.shape == (0, 2) and wt.shape == (0, 2)


def test_refusals():
    x = torch.zeros(4, 64, dtype=BF, device="cuda")
    w = torch.zeros(16, 64, dtype=BF, device="cuda")
    with pytest.raises(tr.TopReduceError):
        tr.route_topk(x, w, 0)
    with pytest.raises(tr.TopReduceError):
        tr.route_topk(x, w, 17)
    with pytest.raises(tr.TopReduceError):
        tr.route_topk(x, w, 2, scale=float("nan"))
    with pytest.raises(tr.TopReduceError):
        tr.route_topk(x, w, 2, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        tr.route_topk(x, w, 2, score="tanh")
    with pytest.raises(ValueError):
        tr.route_topk(x, w[:, :32], 2)
    with pytest.raises(ValueError):
        tr.route_topk(x.cpu(), w, 2)
    with pytest.raises(TypeError):
        tr.route_topk(x, w.float(), 2)
    with pytest.raises(TypeError):
        tr.route_topk(x, w, 2, idx_dtype=torch.int16)
    with pytest.raises(TypeError):
        tr.route_topk(x.half(), w.half(), 2)
    with pytest.raises(TypeError):
        tr.route_topk(x, w, 2, bias=torch.zeros(16, dtype=BF, device="cuda"))
    with pytest.raises(ValueError):
        tr.route_topk(x.t().contiguous().t(), w, 2)
