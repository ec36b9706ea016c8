"""rms_norm and quantize_mx against their formulas in 64 bits."""

import pytest
import torch

import top_reduce_amd as tr
from tests import _mx as M
from tests import _serving as S
from tests._gpu import say

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
SIZES = [(1, 32), (3, 64), (5, 512), (7, 544), (64, 2048), (2, 2080), (1, 7168), (33, 7168), (4, 8192), (3, 8224),
         (2, 32768), (2, 32800), (300, 2880)]


def inputs(T, H, dtype, residual):
    g = torch.Generator().manual_seed(T + H)
    x = S.inputs(g, T, H, dtype=dtype)
    r = S.inputs(g, T, H, dtype=dtype, std=5.0) if residual else None
    w = (1 + 0.3 * torch.randn(H, generator=g)).to(dtype)
    return x, r, w


def cuda(t):
    return None if t is None else t.cuda()


@pytest.mark.parametrize("T,H", SIZES + [(9, 8), (6, 1000), (2, 40000)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("residual", [False, True])
def test_norm(T, H, dtype, residual):
    say(f"norm T={T} H={H} {dtype} residual={residual}")
    x, r, w = inputs(T, H, dtype, residual)
    out = "both" if H % 32 == 0 else "same"
    got = tr.rms_norm(x.cuda(), w.cuda(), 1e-5, residual=cuda(r), out=out)
    y, z, err = M.rms_norm(x, w, 1e-5, r)
    half = torch.finfo(dtype).eps / 2
    S.check(got.y, y, err + half * (y.abs() + err) + 1e-30, "y")
    if residual:
        S.check(got.residual, z, half * z.abs() * (1 + 2.0 ** -20) + 2.0 ** -24 * z.abs(), "residual")
    else:
        assert got.residual is None
    if out == "both":
        M.check_blocks((got.q, got.s), y, err, "8 bits")
        only = tr.rms_norm(x.cuda(), w.cuda(), 1e-5, residual=cuda(r), out="mx8")
        assert only.y is None
        assert torch.equal(only.q.view(torch.uint8), got.q.view(torch.uint8))
        assert torch.equal(only.s.view(torch.uint8), got.s.view(torch.uint8))


@pytest.mark.parametrize("T,H", [(3, 64), (5, 7168), (2, 40000)])
def test_outputs_over_the_inputs(T, H):
    x, r, w = inputs(T, H, BF, True)
    want = tr.rms_norm(x.cuda(), w.cuda(), residual=r.cuda())
    a, b = x.cuda(), r.cuda()
    got = tr.rms_norm(a, w.cuda(), residual=b, y=a, residual_out=b)
    assert got.y is a and got.residual is b
    assert torch.equal(a, want.y) and torch.equal(b, want.residual)


@pytest.mark.parametrize("T,H,dtype,residual", [(1100, 8192, BF, True), (12000, 8192, BF, True), (9000, 8192, F32, False)])
def test_large_batches_are_their_rows(T, H, dtype, residual):
    """Outputs, and inputs, that the caches do not hold."""
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, H, generator=g, device="cuda").to(dtype)
    r = torch.randn(T, H, generator=g, device="cuda").to(dtype) if residual else None
    w = torch.randn(H, generator=g, device="cuda").to(dtype)
    got = tr.rms_norm(x, w, residual=r, out="both")
    for a in (0, T // 2, T - 64):
        some = tr.rms_norm(x[a:a + 64], w, residual=None if r is None else r[a:a + 64], out="both")
        for u, v in zip(got, some):
            assert (u is None and v is None) or torch.equal(u[a:a + 64].view(torch.uint8), v.view(torch.uint8))
    assert torch.isfinite(got.y).all()


def test_rows_stand_alone():
    x, r, w = inputs(6, 96, BF, True)
    clean = tr.rms_norm(x.cuda(), w.cuda(), residual=r.cuda(), out="both")
    bad = x.clone()
    bad[1, 5], bad[3, 7], bad[4] = float("nan"), float("inf"), 0.0
    r2 = r.clone()
    r2[4] = 0.0
    got = tr.rms_norm(bad.cuda(), w.cuda(), residual=r2.cuda(), out="both")
    for t in (0, 2, 5):
        for u, v in zip(got, clean):
            assert torch.equal(u[t].view(torch.uint8), v[t].view(torch.uint8))
    assert torch.isnan(got.y[1]).all() and torch.isnan(got.q[1].float()).all()
    assert torch.isnan(got.y[3, 7]) and torch.isnan(got.q.float()[3, 7])
    assert (got.y[4] == 0).all() and (got.q[4].float() == 0).all()
    assert (got.s[4].view(torch.uint8) == 0).all()       # nothing in the block: 2^-127


def test_no_rows():
    got = tr.rms_norm(torch.empty(0, 64, dtype=BF, device="cuda"), torch.ones(64, dtype=BF, device="cuda"),
                      out="both")
    assert got.y.shape == (0, 64) and got.s.shape == (0, 2)
    q, s = tr.quantize_mx(torch.empty(0, 64, dtype=BF, device="cuda"))
    assert q.shape == (0, 64) and s.shape == (0, 2)


@pytest.mark.parametrize("shape", [(1, 32), (3, 96), (2, 5, 64), (257, 7168), (64,)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("bits", [8, 4])
def test_quantize_is_exact(shape, dtype, bits):
    """Bit for bit: one rounding of numbers that are known."""
    g = torch.Generator().manual_seed(sum(shape))
    x = S.inputs(g, *shape, dtype=dtype) * torch.exp2(torch.randint(-20, 20, (*shape[:-1], 1), generator=g)).to(dtype)
    q, s = tr.quantize_mx(x.cuda(), bits)
    wq, ws = M.quantize(x, bits)
    assert torch.equal(s.cpu().view(torch.uint8), ws.view(torch.uint8))
    assert torch.equal(q.cpu().view(torch.uint8), wq.view(torch.uint8))


@pytest.mark.parametrize("bits", [8, 4])
def test_quantize_at_the_edges(bits):
    top = M.MOST[bits]
    x = torch.zeros(12, 32)
    x[0, 3] = top                                   # the largest: scale 1
    x[1, 3] = torch.nextafter(torch.tensor(top), torch.tensor(1e9))    # past it: scale 2
    x[2] = torch.arange(32) * top / 62              # ties among them
    x[3] = -x[2]
    x[4, 0], x[4, 1] = 3.4e38, 1e30
    x[5, 0] = 1e-45                                 # subnormal
    x[6] = 2.0 ** -130
    x[7, 31] = 2.0 ** -118
    x[8] = 1.0
    x[8, 4] = float("nan")
    x[9] = 2.0
    x[9, 30] = float("inf")
    x[10, 2], x[10, 3] = -float("inf"), 5.0
    q, s = tr.quantize_mx(x.cuda(), bits)
    wq, ws = M.quantize(x, bits)
    assert torch.equal(s.cpu().view(torch.uint8), ws.view(torch.uint8))
    got, want = M.value(q, s), M.value(wq, ws)
    assert torch.equal(torch.nan_to_num(got, nan=-1.0), torch.nan_to_num(want, nan=-1.0))
