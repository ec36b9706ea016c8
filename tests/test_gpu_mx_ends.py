"""linear_mx4 and expert_linear at the ends of their sizes and numbers."""

import ctypes

import pytest
import torch

import top_reduce_amd as tr
from tests import _close as C
from tests import _mx as M
from tests import _serving as S
from tests._gpu import say
from top_reduce_amd import _binding as B

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def pair(p):
    return tuple(t.cuda() for t in p)


@pytest.mark.parametrize("T,K,N", [(1, 4096, 16), (2, 4096, 8), (16, 4096, 1), (1, 8192, 8), (4, 16384, 1), (1, 4096, 1),
                                   (1, 16384, 33)])
def test_the_smallest_shared_sums(T, K, N):
    """Parts of K whose sums are 256 bytes and less: with a workspace of the call's and of the caller's."""
    say(f"linear4 T={T} K={K} N={N}")
    g = torch.Generator().manual_seed(T + N)
    x = S.inputs(g, T, K, dtype=F32)
    w = M.quantize(torch.randn(N, K, generator=g, dtype=torch.float64), 4)
    n = tr.linear_mx4_workspace_size(T, K, N, F32)
    assert n > 256
    y = tr.linear_mx4(x.cuda(), pair(w))
    assert torch.equal(y, tr.linear_mx4(x.cuda(), pair(w), ws=torch.full((n,), 255, dtype=torch.uint8, device="cuda")))
    xv, wv = S.f64(x), M.value(*w)
    want = xv @ wv.t()
    S.check(y, want, S.U[F32] * want.abs() + (K + 64) * S.EPS * (xv.abs() @ wv.abs().t()), "y")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K,N", [(4096, 16), (7168, 7168), (256, 16384)])
def test_no_rows(K, N, dtype):
    w = (torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda"),
         torch.zeros(N, K // 32, dtype=torch.uint8, device="cuda").view(M.E8M0))
    assert tr.linear_mx4(torch.empty(0, K, dtype=dtype, device="cuda"), w).shape == (0, N)


@pytest.mark.parametrize("kernel", ["rows", "tile256", "auto"])
def test_as_many_rows_as_there_may_be(kernel):
    """2^31 - 1 gathered rows: segments that begin off a tile and end at the last row, whose strips and
    counts of tiles pass 2^31 on the way."""
    T, K, R = 64, 256, (1 << 31) - 1
    say(f"experts {R} rows {kernel}")
    g = torch.Generator().manual_seed(5)
    x = pair(M.quantize(torch.randn(T, K, generator=g, dtype=torch.float64)))
    w = pair(M.quantize(torch.randn(2, 1, K, generator=g, dtype=torch.float64)))
    rows = torch.randint(0, T, (R,), dtype=torch.int32, device="cuda")
    each = torch.arange(T, dtype=torch.int32, device="cuda").repeat(2)
    table = tr.expert_linear(x, w, torch.tensor([0, T, 2 * T], dtype=torch.int32, device="cuda"), rows=each,
                             kernel="tile256" if kernel == "auto" else kernel).reshape(2, T)
    assert len(table.unique()) > T
    y = torch.full((R, 1), 7.0, dtype=BF, device="cuda")
    tr.expert_linear(x, w, torch.tensor([5, 70, R], dtype=torch.int32, device="cuda"), rows=rows, y=y, kernel=kernel)
    assert (y[:5] == 7).all() and torch.equal(y[5:70, 0], table[0][rows[5:70].long()])
    step = 1 << 27
    for a in range(70, R, step):
        assert torch.equal(y[a:a + step, 0], table[1][rows[a:a + step].long()]), a
    del y, rows
    torch.cuda.empty_cache()


def test_a_plan_with_tiles_past_a_launch():
    """Sizes whose 64-row tiles are more than a launch has blocks for, 254 GB in earnest: here the plan
    holds no rows, so that neither weights nor rows of h are read or written."""
    T, K, E, H, I = 14336, 2, 1024, 256, 563200
    say(f"forward T={T} E={E} H={H} I={I}")
    lib = tr.load_library()
    p = tr.plan(torch.full((T, K), -1, dtype=torch.int64, device="cuda"), E=E, H=H, I=I, flags=tr.FLAG_NO_XE)
    assert int(p.views()["offsets"].max()) == 0
    x = torch.zeros(T, H, dtype=torch.uint8, device="cuda")
    y = torch.full((T, H), 7.0, dtype=BF, device="cuda")
    a = x.data_ptr()
    for bits in (4, 8):
        status = lib.moe_forward_mx(ctypes.byref(p.struct), a, a, None, bits, a, a, a, a, y.data_ptr(), B._raw_stream(y.device))
        assert status == 0, lib.moe_last_error()
        torch.cuda.synchronize()
        assert (y == 0).all()
        y.fill_(7)
    del p
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,K", [(3, 64), (3, 512), (1, 4096), (4, 4096), (20, 512), (20, 4096), (16, 256), (40, 1056)])
@pytest.mark.parametrize("low", [100, 112, 120, 126, 134, 140])
def test_small_numbers_count_in_full(T, K, low):
    """Rows in fp32 down to the smallest, beside weights that bring the products back: fp32's own 24
    bits (fewer below 2^-126, exact there), whatever the kernel. Rows of large ones among them."""
    say(f"linear4 T={T} K={K} x near 2^-{low}")
    g = torch.Generator().manual_seed(T + K + low)
    q, s = M.quantize(torch.randn(48, K, generator=g, dtype=torch.float64), 4)
    s = (s.view(torch.uint8) + 100).view(M.E8M0)
    x = torch.ldexp(torch.randn(T, K, generator=g, dtype=torch.float64),
                    torch.randint(-low - 4, -low + 1, (T, K), generator=g).double()).float()
    x[T // 2, ::3] = 0.0
    if T > 1:
        x[0] *= 2.0 ** 90
    y = tr.linear_mx4(x.cuda(), pair((q, s)))
    xv, wv = S.f64(x), M.value(q, s)
    want = xv @ wv.t()
    S.check(y, want, S.U[F32] * want.abs() + (K + 64) * S.EPS * (xv.abs() @ wv.abs().t()), "y")
    C.check(y, want, K, F32, "y")
    # and of single numbers: no sum to hide in, each product rounded once
    one = torch.zeros(T, K)
    at = torch.arange(T) * 7 % K
    one[torch.arange(T), at] = x[torch.arange(T), at]
    want = S.f64(one) @ wv.t()
    y = S.f64(tr.linear_mx4(one.cuda(), pair((q, s))))
    assert ((y - want).abs() <= 2.0 ** -23 * want.abs()).all() and ((want != 0).any() or T == 1)
    # what is not finite among them stays in its row
    bad = x.clone()
    bad[T - 1, 5], bad[T // 2, 6] = float("inf"), float("nan")
    z = tr.linear_mx4(bad.cuda(), pair((q, s))).cpu()
    hit = torch.zeros(T, dtype=torch.bool)
    hit[T - 1] = hit[T // 2] = True
    assert not z[hit].isfinite().any() and torch.equal(z[~hit], tr.linear_mx4(x.cuda(), pair((q, s))).cpu()[~hit])


def ends(bits, E, N, K, scale, code):
    """[E, N, K] numbers, all of one element and one scale."""
    q = torch.full((E, N, K * bits // 8), code, dtype=torch.uint8)
    return (q.view(M.E4M3) if bits == 8 else q), torch.full((E, N, K // 32), scale, dtype=torch.uint8).view(M.E8M0)


@pytest.mark.parametrize("bits,code,scale", [(8, 0x7e, 254), (8, 0x7e, 247), (4, 0x77, 254), (8, 0x38, 254), (4, 0x22, 254)])
@pytest.mark.parametrize("kernel", ["rows", "tile32", "tile64", "tile256"])
@pytest.mark.parametrize("n", [3, 40])
def test_weights_past_fp32(bits, code, scale, kernel, n):
    """Weights of 2^128 and more, which the format has and fp32 has not: the tiles multiply blocks as
    they are, the kernel of rows takes such a number as infinite."""
    K = 256
    w = ends(bits, 1, 32, K, scale, code)
    x = torch.zeros(n, K, dtype=torch.uint8)
    x[:, 9] = 0x38                                       # 1, scaled
    x = (x.view(M.E4M3), torch.full((n, K // 32), 127 - 60, dtype=torch.uint8).view(M.E8M0))
    off = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    y = S.f64(tr.expert_linear(pair(x), pair(w), off, kernel=kernel))
    v = M.value(*w)[0, 0, 0]
    if kernel == "rows" and v >= 2.0 ** 128:
        assert not y.isfinite().any()
    else:
        want = v * 2.0 ** -60
        assert ((y - want).abs() <= 2.0 ** -8 * want).all()


@pytest.mark.parametrize("scale", [0, 1, 3, 8, 20])
@pytest.mark.parametrize("kernel", ["rows", "tile32", "tile64", "tile256"])
@pytest.mark.parametrize("n", [3, 40])
def test_weights_below_bf16(scale, kernel, n):
    """Weights of 8 bits down to 2^-136: in the kernel of rows those below 2^-133 go by bf16's steps."""
    K = 256
    g = torch.Generator().manual_seed(scale)
    q = torch.randint(1, 0x78, (1, 32, K), generator=g, dtype=torch.uint8).view(M.E4M3)
    w = (q, torch.full((1, 32, K // 32), scale, dtype=torch.uint8).view(M.E8M0))
    x = M.quantize(torch.rand(n, K, generator=g, dtype=torch.float64) + 0.5)
    x = (x[0], (x[1].view(torch.uint8) + 110).view(M.E8M0))
    off = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    y = S.f64(tr.expert_linear(pair(x), pair(w), off, kernel=kernel))
    xv, wv = M.value(*x), M.value(*w)[0]
    want, size = xv @ wv.t(), xv.abs() @ wv.abs().t()
    step = 2.0 ** -134 * xv.abs().sum(1, keepdim=True) if kernel == "rows" else 0.0      # half of bf16's smallest
    assert ((y - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -10 * size + step).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,K", [(2, 64), (2, 512), (20, 512), (2, 4096), (20, 4096)])
def test_projection_weights_past_fp32(T, K, dtype):
    """Infinite, as in a weight matrix of fp32; the largest below it is not."""
    x = torch.zeros(T, K, dtype=dtype, device="cuda")
    x[:, 9] = 2.0 ** -60
    for code, scale in ((0x77, 254), (0x66, 254), (0x55, 254), (0x77, 252), (0x22, 254)):
        q, s = ends(4, 1, 16, K, scale, code)
        v = M.value(q, s)[0, 0, 0]
        y = S.f64(tr.linear_mx4(x, pair((q[0], s[0]))))
        if v >= 2.0 ** 128:
            assert not y.isfinite().any(), (code, scale)
        else:
            assert (y == v * 2.0 ** -60).all(), (code, scale)
