"""Norm, experts' products and projections in 8 and 4 bits past 32 bits of offset, with many
experts, and two at once. What is large is compared with the same rows in a small call, whose
results have the same bits (a row's do not hang on the others)."""

import pytest
import torch

import top_reduce_amd as tr
from tests import _mx as M
from tests._gpu import say

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def blocks(g, *shape):
    """Numbers in 8 bits, made on the GPU."""
    q = torch.randint(0, 100, shape, generator=g, device="cuda", dtype=torch.uint8)
    q += 128 * torch.randint(0, 2, shape, generator=g, device="cuda", dtype=torch.uint8)
    s = torch.randint(118, 124, (*shape[:-1], shape[-1] // 32), generator=g, device="cuda", dtype=torch.uint8)
    return q.view(M.E4M3), s.view(M.E8M0)


def part(pair, a, b):
    return pair[0][a:b].contiguous(), pair[1][a:b].contiguous()


def same(got, want):
    for u, v in zip(got if isinstance(got, tuple) else (got,), want if isinstance(want, tuple) else (want,)):
        assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.fixture
def g():
    yield torch.Generator(device="cuda").manual_seed(3)
    torch.cuda.empty_cache()


@pytest.mark.parametrize("out", ["bf16", "mx8"])
@pytest.mark.parametrize("kernel", ["tile64", "tile256"])
def test_results_past_32_bits(g, kernel, out):
    R, K, N = 70000, 256, 32768
    say(f"experts {R} x {K} x {N} {kernel} {out}")
    x, w = blocks(g, R, K), blocks(g, 2, N, K)
    y = tr.expert_linear(x, w, ints(0, 40000, R), out=out, kernel=kernel)
    for a, off in ((R - 40, ints(0, 0, 40)), (39970, ints(0, 30, 40))):
        want = tr.expert_linear(part(x, a, a + 40), w, off, out=out, kernel=kernel)
        same(part(y, a, a + 40) if out == "mx8" else y[a:a + 40], want)


def test_rows_past_32_bits(g):
    T, K, N = 70000, 32768, 64
    x, w = blocks(g, T, K), blocks(g, 2, N, K)
    for kernel in ("tile32", "tile256"):
        say(f"experts {T} x {K} x {N} {kernel}")
        y = tr.expert_linear(x, w, ints(0, 40000, T), kernel=kernel)
        same(y[T - 40:], tr.expert_linear(part(x, T - 40, T), w, ints(0, 0, 40), kernel=kernel))
    # gathered ones are addressed with 31 bits in the tiles, and not in the other kernel
    rows = torch.tensor([T - 1, 3, T - 1, 65537], dtype=torch.int32, device="cuda")
    with pytest.raises(tr.TopReduceError):
        tr.expert_linear(x, w, ints(0, 2, 4), rows=rows, kernel="tile32")
    few = tuple(t.view(torch.uint8)[rows.long()].view(t.dtype) for t in x)
    same(tr.expert_linear(x, w, ints(0, 2, 4), rows=rows),
         tr.expert_linear(few, w, ints(0, 2, 4), kernel="rows"))


@pytest.mark.parametrize("bits", [8, 4])
def test_norm_and_quantize_past_32_bits(g, bits):
    T, H = 300000, 7168
    x = torch.empty(T, H, dtype=BF, device="cuda").normal_(generator=g)
    n = 37
    if bits == 8:
        weight = torch.rand(H, generator=g, device="cuda").to(BF)
        got = tr.rms_norm(x, weight, out="both")
        want = tr.rms_norm(x[T - n:].contiguous(), weight, out="both")
        same((got.y[T - n:], got.q[T - n:], got.s[T - n:]), (want.y, want.q, want.s))
        del got
    q = tr.quantize_mx(x, bits)
    same(part(q, T - n, T), tr.quantize_mx(x[T - n:].contiguous(), bits))


@pytest.mark.parametrize("T,K,N", [(70000, 256, 32768), (1100000, 2048, 64)])
def test_linear_past_32_bits(g, T, K, N):
    say(f"linear {T} x {K} x {N}")
    x = torch.empty(T, K, dtype=BF, device="cuda").normal_(generator=g)
    w = tr.quantize_mx(torch.randn(N, K, generator=g, device="cuda"), 4)
    y = tr.linear_mx4(x, w)
    same(y[T - 50:], tr.linear_mx4(x[T - 50:].contiguous(), w))


@pytest.mark.parametrize("E,most", [(65, 3), (700, 2), (1024, 1), (1024, 90)])
@pytest.mark.parametrize("kernel", ["auto", "rows", "tile32", "tile64", "tile256"])
def test_many_experts(g, E, most, kernel):
    say(f"{E} experts of up to {most} rows, {kernel}")
    K, N = 256, 64
    counts = torch.randint(0, most + 1, (E,), generator=g, device="cuda")
    off = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
    R = int(off[-1])
    x, w = blocks(g, R, K), blocks(g, E, N, K)
    y = tr.expert_linear(x, w, off, kernel=kernel)
    owner = torch.repeat_interleave(torch.arange(E, device="cuda"), counts)
    xv, wv = M.value(*x).cuda(), M.value(*w).cuda()
    # of the sum of magnitudes: 2^-10 (the tiles), 256 2^-24, and the rounding's 2^-8
    bound = 2.0 ** -8 + 2.0 ** -9
    for a in range(0, R, 8192):
        o = wv[owner[a:a + 8192]]
        want = torch.matmul(o, xv[a:a + 8192, :, None])[..., 0]
        size = torch.matmul(o.abs(), xv[a:a + 8192, :, None].abs())[..., 0]
        assert ((y[a:a + 8192].double() - want).abs() <= bound * size).all()


def test_two_at_once(g):
    """Two streams, each with its own plan, workspace and results."""
    H, I, E, T = 512, 128, 8, 90
    w1, w2, w4 = blocks(g, E, 2 * I, H), blocks(g, E, H, I), tr.quantize_mx(torch.randn(256, 4096, device="cuda"), 4)
    x = [blocks(g, T, H) for _ in range(2)]
    wide = [torch.randn(40, 4096, device="cuda").to(BF) for _ in range(2)]
    idx = [torch.randint(0, E, (T, 2), generator=g, device="cuda") for _ in range(2)]
    plans = [tr.plan(i, E=E, H=H, I=I) for i in idx]
    want = [(tr.forward_mx(plans[k], x[k], None, w1, w2), tr.linear_mx4(wide[k], w4)) for k in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for k in range(2):
            got[k].append((tr.forward_mx(plans[k], x[k], None, w1, w2, stream=streams[k]),
                           tr.linear_mx4(wide[k], w4, stream=streams[k])))
    torch.cuda.synchronize()
    for k in range(2):
        for v in got[k]:
            same(v, want[k])


def test_graphs_that_share_a_workspace(g):
    w = tr.quantize_mx(torch.randn(256, 4096, generator=g, device="cuda"), 4)
    x = [torch.randn(T, 4096, generator=g, device="cuda").to(BF) for T in (40, 20)]
    n = max(tr.linear_mx4_workspace_size(v.shape[0], 4096, 256) for v in x)
    assert n > 256
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    y = [tr.linear_mx4(v, w, ws=ws) for v in x]
    torch.cuda.synchronize()
    graphs = []
    for v, out in zip(x, y):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            tr.linear_mx4(v, w, y=out, ws=ws)
    for _ in range(4):
        for k in (0, 1, 0):
            x[k].normal_(generator=g)
            ws.fill_(255)
            graphs[k].replay()
            same(y[k], tr.linear_mx4(x[k], w))
            torch.cuda.synchronize()


@pytest.mark.parametrize("flags", [0, tr.FLAG_NO_XE])
@pytest.mark.parametrize("counts", [(8, 3, 0), (0, 8, 8), (0, 0, 0)])
def test_padded_rows(g, counts, flags):
    """A buffer whose blocks of 8 rows hold fewer tokens: as with ids of none."""
    H, I, E, T = 256, 64, 4, 24
    w1, w2, x = blocks(g, E, 2 * I, H), blocks(g, E, H, I), blocks(g, T, H)
    idx = torch.randint(0, E, (T, 2), generator=g, device="cuda")
    weights = torch.rand(T, 2, generator=g, device="cuda")
    p = tr.plan(idx, E=E, H=H, I=I, flags=flags, block_rows=8, block_counts=ints(*counts))
    y = tr.forward_mx(p, x, weights, w1, w2)
    pad = torch.tensor([r % 8 >= counts[r // 8] for r in range(T)], device="cuda")
    q = tr.plan(idx.masked_fill(pad[:, None], -1), E=E, H=H, I=I)
    want = tr.forward_mx(q, x, weights, w1, w2)
    assert torch.equal(y[~pad], want[~pad]) and (want[pad] == 0).all()
    assert (y[pad] == 0).all()
