"""The layer in 8 and 4 bits: norm, router, plan and experts together, as a served block
runs them; captured, on another stream, and against 64 bits."""

import pytest
import torch

import top_reduce_amd as tr
from tests import _mx as M
from tests import _serving as S
from tests._gpu import say

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
TILED = 2.0 ** -10


def weights(g, E, N, K, bits):
    q, s = M.quantize(torch.randn(E, N, K, generator=g, dtype=torch.float64) * K ** -0.5, bits)
    return q.cuda(), s.cuda()


def block(T, H, I, E, G, K, bits, seed=0):
    g = torch.Generator().manual_seed(seed + T + H)
    return {"x": S.inputs(g, T, H, dtype=BF).cuda(), "r": S.inputs(g, T, H, dtype=BF, std=3.0).cuda(),
            "norm": (1 + 0.2 * torch.randn(H, generator=g)).to(BF).cuda(),
            "gate": S.inputs(g, G, H, dtype=BF, std=1.5 * H ** -0.5).cuda(),
            "w1": weights(g, E, 2 * I, H, bits), "w2": weights(g, E, H, I, bits), "E": E, "I": I, "K": K}


def run(b, x=None, r=None, begin=0, **kw):
    n = tr.rms_norm(b["x"] if x is None else x, b["norm"], residual=b["r"] if r is None else r, out="both", **kw)
    idx, w = tr.route_topk(n.y, b["gate"], b["K"], **kw)
    p = tr.plan(idx, E=b["E"], H=n.y.shape[1], I=b["I"], expert_begin=begin, **kw)
    return tr.forward_mx(p, (n.q, n.s), w, b["w1"], b["w2"], **kw), n, idx, w


@pytest.mark.parametrize("T,H,I,E,G,K,begin", [(1, 64, 32, 4, 4, 2, 0), (7, 256, 96, 6, 12, 3, 6), (64, 512, 128, 8, 8, 4, 0),
                                               (300, 384, 160, 4, 8, 2, 2), (900, 256, 64, 3, 3, 2, 0)])
@pytest.mark.parametrize("bits", [8, 4])
def test_block(T, H, I, E, G, K, begin, bits):
    say(f"block T={T} H={H} I={I} E={E} G={G} K={K} bits={bits}")
    b = block(T, H, I, E, G, K, bits)
    y, n, idx, w = run(b, begin=begin)
    x, w1, w2 = M.value(n.q, n.s), M.value(*b["w1"]), M.value(*b["w2"])
    idx, w = idx.cpu(), S.f64(w)
    want = torch.zeros(T, H, dtype=torch.float64)
    bound = torch.zeros_like(want)
    for e in range(E):
        t, k = (idx == begin + e).nonzero(as_tuple=True)
        if not t.numel():
            continue
        h, err, _ = M.products(x[t], w1[e:e + 1], torch.tensor([0, t.numel()]), swiglu=True, tiled=TILED)
        # h in 8 bits: half a step, 2^-4 of a number's binade, 2^-10 448/256 of the block's largest
        top = (h.abs() + err).unflatten(-1, (-1, 32)).amax(-1).repeat_interleave(32, -1)
        err = err + 2.0 ** -4 * (h.abs() + err) + 2.0 ** -16 * top
        o = h @ w2[e].t()
        d = err @ w2[e].abs().t() + ((I + 64) * S.EPS + TILED) * (h.abs() @ w2[e].abs().t()) + 2.0 ** -8 * o.abs()
        c = w[t, k][:, None]
        want[t] += c * o
        bound[t] += c.abs() * d
    bound = 1.01 * bound + 2.0 ** -8 * (want.abs() + bound)
    S.check(y, want, bound, "y")
    assert float((S.f64(y) - want).norm()) <= 0.06 * float(want.norm())     # 2^-4 of every h at most
    none = ~((idx >= begin) & (idx < begin + E)).any(1)
    assert (S.f64(y)[none] == 0).all()


@pytest.mark.parametrize("T", [3, 200])
def test_it_is_its_parts(T):
    b = block(T, 256, 64, 4, 4, 2, 8)
    y, n, idx, w = run(b)
    p = tr.plan(idx, E=4, H=256, I=64)
    v = p.views()
    h = tr.expert_linear((n.q, n.s), b["w1"], v["offsets"], rows=v["row_src"], swiglu=True, out="mx8")
    o = tr.expert_linear(h, b["w2"], v["offsets"])
    assert torch.equal(tr.combine_reduce(p, w, expert_out=o), y)
    # without weights: weight 1
    assert torch.equal(tr.forward_mx(p, (n.q, n.s), None, b["w1"], b["w2"]),
                       tr.combine_reduce(p, None, expert_out=o))


@pytest.mark.parametrize("G,kernel", [(128, "tile64"), (16, "tile256"), (4, "tile256")])
@pytest.mark.parametrize("bits", [8, 4])
def test_the_rows_there_choose_the_kernel(G, kernel, bits):
    """4 of G experts here: 32, 256 and 1024 rows each of the 1024 that the plan has room for."""
    say(f"forward {G} {bits}")
    T, H, I, E, K = 512, 256, 2048, 4, 8 if G > 8 else 4
    g = torch.Generator().manual_seed(G + bits)
    w1, w2 = weights(g, E, 2 * I, H, bits), weights(g, E, H, I, bits)
    x = tuple(t.cuda() for t in M.quantize(torch.randn(2 * T, H, generator=g, dtype=torch.float64)))
    idx = torch.stack([torch.randperm(G, generator=g)[:K] for _ in range(2 * T)]).cuda()
    w = torch.rand(2 * T, K, generator=g).cuda()
    p = tr.plan(idx, E=E, H=H, I=I)
    y = tr.forward_mx(p, x, w, w1, w2)
    v = p.views()
    h = tr.expert_linear(x, w1, v["offsets"], rows=v["row_src"], swiglu=True, out="mx8", kernel=kernel)
    o = tr.expert_linear(h, w2, v["offsets"])
    assert torch.equal(tr.combine_reduce(p, w, expert_out=o), y)


@pytest.mark.parametrize("T", [1, 40, 300])
def test_captured_and_replayed(T):
    b = block(T, 256, 64, 4, 8, 2, 4)
    x, r = b["x"].clone(), b["r"].clone()
    run(b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(b, x, r)
    for k in range(4):
        g = torch.Generator().manual_seed(100 + k)
        x.copy_(S.inputs(g, T, 256, dtype=BF))
        r.copy_(S.inputs(g, T, 256, dtype=BF))
        graph.replay()
        want = run(b, x, r)     # eager, between the replays
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1].residual, want[1].residual)


@pytest.mark.parametrize("T", [2, 150])
def test_on_another_stream(T):
    b = block(T, 256, 64, 4, 8, 2, 8)
    q4 = tr.quantize_mx(b["gate"], 4)
    q8 = tr.quantize_mx(b["x"])
    off = torch.tensor([0, T // 2, T, T, T], dtype=torch.int32, device="cuda")
    calls = [lambda **kw: tr.rms_norm(b["x"], b["norm"], residual=b["r"], out="both", **kw),
             lambda **kw: tr.quantize_mx(b["x"], **kw), lambda **kw: (tr.linear_mx4(b["x"], q4, **kw),),
             lambda **kw: tr.expert_linear(q8, b["w1"], off, swiglu=True, out="mx8", **kw),
             lambda **kw: (tr.expert_linear(q8, b["w1"], off, **kw),)]
    p = tr.plan(torch.zeros(T, 1, dtype=torch.int64, device="cuda"), E=4, H=256, I=64)
    calls.append(lambda **kw: (tr.forward_mx(p, q8, None, b["w1"], b["w2"], **kw),))
    for call in calls:
        want = [t.clone() for t in call()]
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        big = torch.randn(2048, 2048, device="cuda")
        torch.cuda.synchronize()
        with torch.cuda.stream(s):      # keeps the stream busy, so that the calls wait in it
            for _ in range(8):
                big = big @ big * 1e-3
        got = []
        for _ in range(3):
            got.append(call(stream=s))
            for t in want:              # the current stream's next allocations, written
                torch.empty(t.numel() * t.element_size(), dtype=torch.uint8, device="cuda").fill_(255)
        s.synchronize()
        for out in got:
            assert all(torch.equal(u.view(torch.uint8), v.view(torch.uint8)) for u, v in zip(out, want))


def test_refusals_of_the_binding():
    b = block(4, 64, 32, 2, 2, 1, 8)
    n = tr.rms_norm(b["x"], b["norm"], out="mx8")
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    x = (n.q, n.s)
    bad = [lambda: tr.rms_norm(b["x"], b["norm"].float()), lambda: tr.rms_norm(b["x"], b["norm"][:32]),
           lambda: tr.rms_norm(b["x"].t(), b["norm"]), lambda: tr.rms_norm(b["x"], b["norm"], out="q"),
           lambda: tr.rms_norm(b["x"], b["norm"], out="mx8", y=b["x"]),
           lambda: tr.rms_norm(b["x"], b["norm"], q=n.q), lambda: tr.rms_norm(b["x"], b["norm"], residual_out=b["r"]),
           lambda: tr.rms_norm(b["x"], b["norm"], residual=b["r"].float()),
           lambda: tr.rms_norm(b["x"].half(), b["norm"].half()),
           lambda: tr.rms_norm(b["x"][:, :40].contiguous(), b["norm"][:40].contiguous(), out="both"),
           lambda: tr.quantize_mx(b["x"][:, :40].contiguous()), lambda: tr.quantize_mx(b["x"].double()),
           lambda: tr.expert_linear(x, b["w1"], off.long()), lambda: tr.expert_linear(x, b["w1"], off[:2]),
           lambda: tr.expert_linear(x, b["w1"], off, rows=off.long()),
           lambda: tr.expert_linear(x, b["w1"], off, out="f32"),
           lambda: tr.expert_linear((n.q, n.s.view(torch.uint8)), b["w1"], off),
           lambda: tr.expert_linear(x, (b["w1"][0].float(), b["w1"][1]), off),
           lambda: tr.expert_linear(x, (b["w1"][0][:, :, :32].contiguous(), b["w1"][1]), off),
           lambda: tr.linear_mx4(b["x"], tr.quantize_mx(b["gate"], 8)),
           lambda: tr.linear_mx4(b["x"], tr.quantize_mx(b["gate"], 4), y=b["r"].float())]
    for k, call in enumerate(bad):
        with pytest.raises((TypeError, ValueError, tr.TopReduceError)):
            call()
            say(f"refusal {k} did not come")
    p = tr.plan(torch.zeros(4, 1, dtype=torch.int64, device="cuda"), E=2, H=64, I=32, dtype=torch.float32)
    with pytest.raises(tr.TopReduceError):
        tr.forward_mx(p, x, None, b["w1"], b["w2"])
