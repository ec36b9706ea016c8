"""The whole layer (layer) against its formula in 64 bits, and against the
route_topk, plan and forward chain."""

import pytest
import torch

import top_reduce_amd as tr
from tests import _serving as S
from tests._gpu import say

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def make(seed, T, H, I, E, G, dtype):
    g = torch.Generator().manual_seed(seed)
    return (S.inputs(g, T, H, dtype=dtype), S.inputs(g, G, H, dtype=dtype, std=1.5 * H ** -0.5),
            S.inputs(g, E, 2 * I, H, dtype=dtype, std=H ** -0.5),
            S.inputs(g, E, H, I, dtype=dtype, std=I ** -0.5))


def run(x, gate, w1, w2, K, **kw):
    return tr.layer(x.cuda(), gate.cuda(), w1.cuda(), w2.cuda(), K, **kw)


@pytest.mark.parametrize("T,H,I,E,G,K,begin,dtype", [
    (1, 256, 128, 8, 8, 2, 0, BF), (1, 8, 1, 1, 1, 1, 0, BF), (1, 512, 96, 4, 4, 4, 0, BF),
    (2, 264, 72, 6, 12, 3, 6, BF), (7, 136, 70, 5, 5, 2, 0, BF), (15, 512, 257, 8, 16, 4, 8, BF),
    (16, 256, 128, 8, 8, 8, 0, BF), (17, 1032, 33, 3, 9, 2, 3, BF), (31, 256, 64, 2, 2, 1, 0, BF),
    (33, 2880, 40, 4, 4, 3, 0, BF), (48, 64, 16, 300, 400, 6, 50, BF), (64, 512, 128, 8, 64, 8, 56, BF),
    (64, 72, 8, 70, 70, 32, 0, BF), (64, 256, 2048, 2, 2, 2, 0, BF),
    (1, 256, 128, 8, 8, 2, 0, F32), (5, 40, 7, 3, 3, 2, 0, F32), (16, 256, 128, 8, 8, 2, 0, F32),
    (29, 264, 130, 5, 10, 4, 5, F32), (64, 128, 66, 66, 66, 5, 0, F32),
])
def test_against_the_formula(T, H, I, E, G, K, begin, dtype):
    say(f"layer T={T} H={H} I={I} E={E} G={G} K={K} {dtype}")
    x, gate, w1, w2 = make(T + H + I, T, H, I, E, G, dtype)
    y, idx, w = run(x, gate, w1, w2, K, expert_begin=begin, scale=1.5)
    ref_idx, ref_w, tol, keys = S.route(x, gate, K, scale=1.5)
    top = torch.sort(keys, dim=1, descending=True)[0][:, :K + 1]
    clear = ((top[:, :-1] - top[:, 1:]) > 1e-4).all(1)
    assert torch.equal(idx.cpu()[clear], ref_idx[clear])
    S.check(w.cpu()[clear], ref_w[clear], tol[clear], "weights")
    ref, bound = S.layer(x, idx, w, w1, w2, begin)
    S.check(y, ref, bound, "y")
    none = ~((idx.cpu() >= begin) & (idx.cpu() < begin + E)).any(1)
    view = torch.int16 if dtype == BF else torch.int32
    assert not y.cpu()[none].view(view).any()        # +0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,H,I,E,G,K", [
    (20, 512, 160, 4, 4, 2), (40, 256, 99, 6, 12, 4), (40, 264, 99, 6, 6, 4), (64, 136, 257, 3, 3, 3),
    (64, 256, 70, 5, 10, 8), (33, 128, 64, 1, 1, 1),    # many tokens an expert
    (8, 264, 2056, 16, 16, 4), (8, 512, 2051, 16, 16, 4), (9, 136, 1030, 40, 40, 5),
    (64, 72, 1536, 24, 24, 6), (1, 96, 1800, 32, 32, 32),    # the reduction in parts
    (3, 4096, 24, 4, 4, 2), (3, 4104, 24, 4, 4, 2), (3, 7168, 24, 4, 4, 2),
])
def test_shapes_that_divide_the_work_differently(T, H, I, E, G, K, dtype):
    say(f"layer T={T} H={H} I={I} E={E} G={G} K={K} {dtype}")
    x, gate, w1, w2 = make(T + H + I, T, H, I, E, G, dtype)
    y, idx, w = run(x, gate, w1, w2, K, expert_begin=G - E)
    ref, bound = S.layer(x, idx, w, w1, w2, G - E)
    S.check(y, ref, bound, "y")


@pytest.mark.parametrize("T", [65, 200])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_more_rows_are_the_router_plan_and_forward(T, dtype):
    H, I, E, G, K, begin = 256, 128, 8, 16, 4, 4
    x, gate, w1, w2 = (t.cuda() for t in make(T, T, H, I, E, G, dtype))
    y, idx, w = tr.layer(x, gate, w1, w2, K, expert_begin=begin, score="sigmoid", scale=2.0)
    i2, w2_ = tr.route_topk(x, gate, K, score="sigmoid", scale=2.0)
    p = tr.plan(i2, E=E, H=H, I=I, dtype=dtype, expert_begin=begin)
    y2 = tr.forward(p, x, w2_, w1, w2)
    assert torch.equal(idx, i2) and torch.equal(w, w2_) and torch.equal(y, y2)
    ref, bound = S.layer(x, idx, w, w1, w2, begin, few=False)
    S.check(y, ref, bound, "y")


def test_few_rows_agree_with_the_chain():
    T, H, I, E, G, K = 24, 256, 128, 8, 8, 2
    x, gate, w1, w2 = (t.cuda() for t in make(5, T, H, I, E, G, BF))
    y, idx, w = tr.layer(x, gate, w1, w2, K)
    p = tr.plan(idx, E=E, H=H, I=I)
    y2 = tr.forward(p, x, w, w1, w2)
    ref, bound = S.layer(x, idx, w, w1, w2, 0, few=False)
    S.check(y2, ref, bound, "chain")
    S.check(y, ref, bound, "layer")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_experts_that_no_row_chose_are_not_read(dtype):
    T, H, I, E, G, K = 3, 256, 128, 12, 24, 2
    x, gate, w1, w2 = make(9, T, H, I, E, G, dtype)
    y, idx, w = run(x, gate, w1, w2, K, expert_begin=6)
    used = set((idx.cpu() - 6).flatten().tolist())
    for e in range(E):
        if e not in used:
            w1[e], w2[e] = float("nan"), float("nan")
    y2, _, _ = run(x, gate, w1, w2, K, expert_begin=6)
    assert torch.equal(y, y2)


@pytest.mark.parametrize("T", [3, 30, 64])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_an_expert_of_nan_and_infinity_reaches_its_own_rows_only(T, dtype):
    H, I, E, K = 256, 96, 6, 2
    x, gate, w1, w2 = make(10 + T, T, H, I, E, E, dtype)
    y, idx, _ = run(x, gate, w1, w2, K)
    w1[1], w2[4] = float("nan"), float("inf")
    y2, _, _ = run(x, gate, w1, w2, K)
    for e in (1, 4):
        assert not torch.isfinite(y2[(idx == e).any(1)]).any()
    rest = ~((idx == 1) | (idx == 4)).any(1)
    assert torch.equal(y[rest], y2[rest])


@pytest.mark.parametrize("dtype,I", [(BF, 128), (BF, 70), (F32, 66)])
def test_rows_with_nan_and_infinity_stay_apart(dtype, I):
    T, H, E, K = 40, 256, 4, 2
    x, gate, w1, w2 = make(11, T, H, I, E, E, dtype)
    y, _, _ = run(x, gate, w1, w2, K)
    bad = x.clone()
    bad[3, 7], bad[20, 1] = float("nan"), float("inf")
    y2, idx, _ = run(bad, gate, w1, w2, K)
    rest = [t for t in range(T) if t not in (3, 20)]
    assert torch.equal(y[rest], y2[rest])
    assert torch.isnan(y2[3]).all()
    assert ((idx >= 0) & (idx < E)).all()


def test_h_past_bf16_range_is_infinite_not_nan():
    """An expert whose h overflows gives infinities, as the formula in fp32 does."""
    H, I, E = 256, 128, 1
    x = torch.full((2, H), 1.0, dtype=BF)
    gate = torch.zeros(1, H, dtype=BF)
    w1 = torch.full((E, 2 * I, H), 1e18, dtype=BF)
    w2 = torch.ones(E, H, I, dtype=BF)
    y, _, _ = run(x, gate, w1, w2, 1)
    assert torch.isinf(y).all()


@pytest.mark.parametrize("T", [4, 64])
def test_same_bits_in_place_in_a_dirty_workspace_and_on_another_stream(T):
    H, I, E, G, K = 512, 160, 16, 16, 4
    x, gate, w1, w2 = (t.cuda() for t in make(T, T, H, I, E, G, BF))
    y, idx, w = tr.layer(x, gate, w1, w2, K)
    n = tr.layer_workspace_size(T, H, I, E, G, K)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    x2 = x.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        out = tr.layer(x2, gate, w1, w2, K, ws=ws, stream=s)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, (y, idx, w)))
    tr.layer(x2, gate, w1, w2, K, y=x2, ws=ws, stream=s)
    s.synchronize()
    assert torch.equal(x2, y)


@pytest.mark.parametrize("T,I,E,dtype", [(3, 96, 8, BF), (40, 96, 8, BF), (64, 1030, 2, BF), (29, 200, 5, F32)])
def test_rows_do_not_depend_on_their_order(T, I, E, dtype):
    x, gate, w1, w2 = (t.cuda() for t in make(T, T, 256, I, E, E, dtype))
    y, idx, w = tr.layer(x, gate, w1, w2, 2)
    at = torch.randperm(T, generator=torch.Generator().manual_seed(T)).cuda()
    y2, i2, w2_ = tr.layer(x[at].contiguous(), gate, w1, w2, 2)
    assert torch.equal(idx[at], i2) and torch.equal(w[at], w2_) and torch.equal(y[at], y2)


def test_graph_replays_follow_their_inputs():
    T, H, I, E, G, K = 8, 512, 128, 16, 32, 4
    x, gate, w1, w2 = (t.cuda() for t in make(2, T, H, I, E, G, BF))
    n = tr.layer_workspace_size(T, H, I, E, G, K)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    y = torch.empty_like(x)
    idx = torch.empty(T, K, dtype=torch.int64, device="cuda")
    w = torch.empty(T, K, device="cuda")
    call = lambda: tr.layer(x, gate, w1, w2, K, expert_begin=8, y=y, idx=idx, weights=w, ws=ws)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k in range(4):
        x.copy_(torch.randn(T, H, device="cuda").to(BF))
        want = tr.layer(x, gate, w1, w2, K, expert_begin=8)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (y, idx, w))), k


def test_weights_past_four_gigabytes():
    """The last expert's weights lie past 2^32 bytes."""
    H, I, E, K = 4096, 2048, 140, 1
    w1 = torch.zeros(E, 2 * I, H, dtype=BF, device="cuda")     # 4.7 GB
    w2 = torch.zeros(E, H, I, dtype=BF, device="cuda")         # 2.3 GB
    g = torch.Generator().manual_seed(3)
    a = S.inputs(g, 2 * I, H, dtype=BF, std=H ** -0.5)
    b = S.inputs(g, H, I, dtype=BF, std=I ** -0.5)
    w1[E - 1], w2[E - 1] = a.cuda(), b.cuda()
    x = S.inputs(g, 2, H, dtype=BF)
    gate = torch.zeros(E, H, dtype=BF)
    gate[E - 1] = x[0] / 8
    x[1] = x[0]
    y, idx, w = tr.layer(x.cuda(), gate.cuda(), w1, w2, K)
    assert idx.flatten().tolist() == [E - 1] * 2
    ref, bound = S.layer(x, idx - (E - 1), w, a[None], b[None], 0)
    S.check(y, ref, bound, "y")


def test_no_rows():
    x, gate, w1, w2 = make(1, 0, 64, 32, 2, 2, BF)
    y, idx, w = run(x, gate, w1, w2, 1)
    assert y.shape == (0, 64) and idx.shape == (0, 1) and w.shape == (0, 1)


def test_refusals():
    x, gate, w1, w2 = (t.cuda() for t in make(1, 4, 64, 32, 4, 8, BF))
    for kw in (dict(expert_begin=5), dict(expert_begin=-1),
               dict(ws=torch.empty(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(tr.TopReduceError):
            tr.layer(x, gate, w1, w2, 2, **kw)
    with pytest.raises(tr.TopReduceError):
        tr.layer(x, gate, w1, w2, 9)
    with pytest.raises(ValueError):
        tr.layer(x, gate, w1, w2[:, :, :16].contiguous(), 2)
    with pytest.raises(ValueError):
        tr.layer(x, gate, w1[:, :63].contiguous(), w2, 2)
    with pytest.raises(ValueError):
        tr.layer(x, gate, w1.transpose(1, 2), w2, 2)
    with pytest.raises(TypeError):
        tr.layer(x, gate, w1.float(), w2, 2)
    with pytest.raises(ValueError):
        tr.layer(x, gate, w1, w2, 2, y=torch.empty(4, 32, dtype=BF, device="cuda"))
