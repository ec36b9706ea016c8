"""linear_mx4 against its formula in 64 bits."""

import pytest
import torch

import top_reduce_amd as tr
from tests import _close as C
from tests import _mx as M
from tests import _serving as S
from tests._gpu import say

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def case(T, K, N, dtype):
    g = torch.Generator().manual_seed(T + K + N)
    x = S.inputs(g, T, K, dtype=dtype)
    w = M.quantize(torch.randn(N, K, generator=g, dtype=torch.float64) * K ** -0.5, 4)
    return x, w


@pytest.mark.parametrize("T,K,N", [
    (1, 32, 1), (1, 7168, 256), (2, 96, 33), (3, 1440, 1001), (15, 160, 64), (16, 512, 500), (17, 2880, 66),
    (33, 1056, 129), (64, 1024, 256), (65, 256, 48), (130, 4096, 40), (1, 4128, 300), (7, 128, 4), (5, 640, 2),
    (500, 352, 70), (17, 256, 128), (20, 7168, 300), (32, 768, 129), (33, 512, 1000), (64, 7168, 130),
    (100, 1600, 384), (64, 2880, 2050), (200, 288, 520), (70, 8192, 17), (600, 1024, 4100), (8, 8480, 40),
    (16, 16416, 33), (4, 16384, 50),
])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_linear(T, K, N, dtype):
    say(f"linear4 T={T} K={K} N={N} {dtype}")
    x, w = case(T, K, N, dtype)
    y = tr.linear_mx4(x.cuda(), (w[0].cuda(), w[1].cuda()))
    xv, wv = S.f64(x), M.value(*w)
    want = xv @ wv.t()
    S.check(y, want, S.U[dtype] * want.abs() + (K + 64) * S.EPS * (xv.abs() @ wv.abs().t()), "y")
    if N >= 32:
        C.check(y, want, K, dtype, "y", bits16=False)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,K", [(1, 256), (9, 256), (30, 544), (70, 256), (70, 800), (2, 224)])
def test_rows_stand_alone(T, K, dtype):
    x, w = case(T, K, 96, dtype)
    w = (w[0].cuda(), w[1].cuda())
    clean = tr.linear_mx4(x.cuda(), w)
    bad = x.clone()
    bad[T // 2, 200] = float("nan")
    got = tr.linear_mx4(bad.cuda(), w)
    keep = torch.arange(T) != T // 2
    assert torch.isnan(got[T // 2]).all() and torch.equal(got[keep.cuda()], clean[keep.cuda()])
    s = w[1].view(torch.uint8).clone()
    s[50, 2] = 255
    got = tr.linear_mx4(x.cuda(), (w[0], s.view(M.E8M0)))
    keep = torch.arange(96, device="cuda") != 50
    assert torch.isnan(got[:, 50]).all() and torch.equal(got[:, keep], clean[:, keep])


def test_no_rows():
    _, w = case(1, 64, 32, BF)
    assert tr.linear_mx4(torch.empty(0, 64, dtype=BF, device="cuda"), (w[0].cuda(), w[1].cuda())).shape == (0, 32)


def test_a_workspace_of_the_callers():
    x, w = case(40, 4096, 256, BF)
    x, w = x.cuda(), (w[0].cuda(), w[1].cuda())
    want = tr.linear_mx4(x, w)
    n = tr.linear_mx4_workspace_size(40, 4096, 256)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    y = torch.empty_like(want)
    assert tr.linear_mx4(x, w, y=y, ws=ws) is y and torch.equal(y, want)
    with pytest.raises(tr.TopReduceError):
        tr.linear_mx4(x, w, ws=ws[:256])
    # one that is not needed may be there all the same
    assert torch.equal(tr.linear_mx4(x[:3].contiguous(), w, ws=ws), tr.linear_mx4(x[:3].contiguous(), w))


@pytest.mark.parametrize("T,K", [(3, 512), (3, 4096), (20, 512), (20, 4096), (9, 64)])
def test_fp32_rows_of_any_size(T, K):
    """Numbers near both ends of fp32, infinities and signalling NaN: what fp32 products give."""
    g = torch.Generator().manual_seed(T + K)
    w = M.quantize(torch.randint(1, 7, (48, K), generator=g).double() * 0.5, 4)      # no zeros
    x = torch.randn(T, K, generator=g) * torch.tensor([2.0 ** 60, 2.0 ** -60, 1.0])[torch.arange(T) % 3, None]
    x[1] = torch.randn(K, generator=g) * 2.0 ** -100
    y = tr.linear_mx4(x.cuda(), (w[0].cuda(), w[1].cuda()))
    xv, wv = S.f64(x), M.value(*w)
    # (products below 2^-126 may be lost)
    S.check(y, xv @ wv.t(), S.U[F32] * (xv @ wv.t()).abs() + (K + 64) * (S.EPS * (xv.abs() @ wv.abs().t()) + 2.0 ** -126), "y")
    top = torch.zeros(T, K)
    top[0, 5] = torch.finfo(F32).max / 8
    y = tr.linear_mx4(top.cuda(), (w[0].cuda(), w[1].cuda()))
    want = S.f64(top) @ wv.t()
    assert ((S.f64(y) - want).abs() <= 2.0 ** -23 * want.abs()).all() and torch.isfinite(y).all()
    odd = x.clone()
    odd[0, 7] = float("inf")
    odd[2, K - 1] = float("-inf")
    odd.view(torch.int32)[1, 3] = 0x7f800001
    y = tr.linear_mx4(odd.cuda(), (w[0].cuda(), w[1].cuda()))
    assert (y[0] == float("inf")).all() and (y[2] == float("-inf")).all() and torch.isnan(y[1]).all()
    odd[0, 8] = float("-inf")
    assert torch.isnan(tr.linear_mx4(odd.cuda(), (w[0].cuda(), w[1].cuda()))[0]).all()
