"""Values at the edges of the types in the layer and the projection: products
past fp32's range, infinite weights."""

import pytest
import torch

import top_reduce_amd as tr
from tests import _serving as S
from tests._gpu import say

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("T", [2, 30, 64])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_gate_far_below_zero_beside_a_huge_up_value(T, dtype):
    """silu(g) u where g u alone is past fp32: silu comes first. g = -64:
    -64 e^-64 2.5e38; g = -512: 0 in fp32."""
    say(f"huge up values T={T} {dtype}")
    H, I = 256, 64
    x = torch.ones(T, H, dtype=dtype)
    gate = torch.zeros(2, H, dtype=dtype)
    w1 = torch.empty(2, 2 * I, H, dtype=dtype)
    w1[0, :I], w1[1, :I] = -0.25, -2.0
    w1[:, I:] = 1e36
    w2 = torch.full((2, H, I), 1e-14, dtype=dtype)
    y, idx, w = tr.layer(x.cuda(), gate.cuda(), w1.cuda(), w2.cuda(), 2)
    assert idx.tolist() == [[0, 1]] * T and w.tolist() == [[0.5, 0.5]] * T
    g, u = -64.0, H * float(w1[0, I, 0].double())
    want = 0.5 * I * g / (1 + torch.tensor(-g).double().exp()) * u * w2[0, 0, 0].double()
    # e^64 in fp32: its argument's last bit is 64 2^-24 of the result; then one rounding
    assert ((S.f64(y) - want).abs() <= (2.0 ** -16 + S.U[dtype]) * want.abs()).all()


def alike(got, want, what):
    """Infinities of the same signs, NaN in the same places, the rest finite."""
    got = S.f64(got)
    assert torch.equal(got.isposinf(), want.isposinf()), what
    assert torch.equal(got.isneginf(), want.isneginf()), what
    assert torch.equal(got.isnan(), want.isnan()), what


@pytest.mark.parametrize("T,I,dtype", [(1, 96, BF), (9, 70, BF), (33, 257, BF), (64, 2048, BF), (9, 70, F32)])
def test_infinite_down_weights_give_infinities_of_the_right_sign(T, I, dtype):
    """h is two numbers in bf16: the second one times an infinite weight is NaN
    where it is 0, and of either sign where it is not."""
    say(f"infinite w2 T={T} I={I} {dtype}")
    H, E = 264, 2
    g = torch.Generator().manual_seed(T + I)
    x = S.inputs(g, T, H, dtype=dtype)
    gate = torch.zeros(E, H, dtype=dtype)
    w1 = S.inputs(g, E, 2 * I, H, dtype=dtype, std=H ** -0.5)
    # one row of each expert whose h are bf16 numbers (0 as the second one): u is a
    # power of two times x's column of ones, g is large
    x[:, 0] = 1.0
    w1[:, 3], w1[:, I + 3] = 0.0, 0.0
    w1[:, 3, 0], w1[:, I + 3, 0] = 32.0, -4.0
    w2 = S.inputs(g, E, H, I, dtype=dtype, std=I ** -0.5)
    inf = float("inf")
    w2[0, 5, 7], w2[1, 40, 2], w2[0, 41, 3], w2[1, 100, 3] = inf, -inf, inf, -inf
    w2[0, 200, 8], w2[0, 200, 9], w2[1, 201, 4] = inf, -inf, float("nan")
    y, idx, w = tr.layer(x.cuda(), gate.cuda(), w1.cuda(), w2.cuda(), 2)
    assert idx.tolist() == [[0, 1]] * T
    x6 = S.f64(x)
    want = 0.0
    for e in range(E):
        gu = x6 @ S.f64(w1[e]).t()
        h = 0.5 * gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
        assert (h.abs() > 1e-30).all()
        want = want + h @ S.f64(w2[e]).t()
    alike(y, want, "y")
    assert (~torch.isfinite(want)).sum() >= 6 * T


@pytest.mark.parametrize("T,H,N,R,A,dtype", [
    (1, 256, 130, 12, 2, BF), (40, 264, 257, 33, 3, BF), (90, 256, 300, 64, 2, BF), (9, 256, 130, 12, 2, F32),
])
def test_infinite_adapter_weights_give_infinities_of_the_right_sign(T, H, N, R, A, dtype):
    check_infinite_adapters(T, H, N, R, A, 1, dtype)


def check_infinite_adapters(T, H, N, R, A, run, dtype):
    say(f"infinite b T={T} H={H} N={N} R={R} {dtype}")
    g = torch.Generator().manual_seed(T + N)
    x = S.inputs(g, T, H, dtype=dtype)
    w = S.inputs(g, N, H, dtype=dtype, std=H ** -0.5)
    a = S.inputs(g, A, R, H, dtype=dtype, std=H ** -0.5)
    b = S.inputs(g, A, N, R, dtype=dtype, std=R ** -0.5)
    ids = (torch.arange(-(-T // run)) % (A + 1)).to(torch.int32).repeat_interleave(run)[:T].contiguous()
    # a low-rank product that is a bf16 number: its second number is 0
    x[:, 0] = 1.0
    a[:, 3] = 0.0
    a[:, 3, 0] = -4.0
    inf = float("inf")
    b[:, 5, 7], b[:, 40, 2], b[:, 41, 3], b[:, 100, 3] = inf, -inf, inf, -inf
    b[:, 120, 8], b[:, 120, 9], b[:, 121, 4] = inf, -inf, float("nan")
    y = tr.adapter_linear(x.cuda(), w.cuda(), a.cuda(), b.cuda(), ids.cuda())
    want = S.f64(x) @ S.f64(w).t()
    for i in range(A):
        mine = ids == i
        v = S.f64(x[mine]) @ S.f64(a[i]).t()
        assert (v.abs() > 1e-30).all()
        want[mine] += v @ S.f64(b[i]).t()
    alike(y, want, "y")
    assert (~torch.isfinite(want)).sum() >= 6 * int((ids < A).sum())


@pytest.mark.parametrize("T,H,N,R,A,run,dtype", [
    (700, 264, 4096, 20, 3, 9, BF), (2048, 256, 4100, 16, 2, 300, BF),       # 64 x 64, 128 x 256
    (4100, 128, 8192, 24, 4, 1, BF), (4100, 256, 8192, 16, 4, 300, BF),      # 256 x 256
    (700, 264, 4096, 20, 3, 9, F32),
])
def test_infinite_adapter_weights_on_tiles(T, H, N, R, A, run, dtype):
    check_infinite_adapters(T, H, N, R, A, run, dtype)


# 2^128 - 2^118: a number of fp32 (the largest is 2^128 - 2^104), but 2^128, infinity,
# once it is rounded to bf16 (the largest is 2^128 - 2^120)
TOP = 2.0 ** 128 - 2.0 ** 118


@pytest.mark.parametrize("T,dtype", [(1, BF), (20, BF), (64, BF), (20, F32)])
def test_h_between_the_ranges_of_bf16_and_fp32(T, dtype):
    say(f"h past bf16 T={T} {dtype}")
    H, I = 64, 40
    x = torch.ones(T, H, dtype=dtype)
    w1 = torch.zeros(1, 2 * I, H, dtype=dtype)
    w1[0, :I, 0], w1[0, :I, 1], w1[0, I:, 2] = 2.0 ** 60, -2.0 ** 50, 2.0 ** 68     # h = TOP
    w1[0, I // 2:I] *= -1.0       # silu is 0 there
    w2 = torch.zeros(1, H, I, dtype=dtype)
    w2[0, :, 3], w2[0, 1::2, 3] = 2.0 ** -120, -2.0 ** -121
    y, _, w = tr.layer(x.cuda(), torch.zeros(1, H, dtype=dtype).cuda(), w1.cuda(), w2.cuda(), 1)
    assert w.tolist() == [[1.0]] * T
    want = (TOP * w2[0, :, 3].double()).to(dtype).expand(T, H)
    assert torch.equal(y.cpu(), want)


@pytest.mark.parametrize("T,N,dtype", [(1, 64, BF), (40, 130, BF), (700, 4096, BF), (4100, 8192, BF), (40, 130, F32)])
def test_low_rank_products_between_the_ranges_of_bf16_and_fp32(T, N, dtype):
    say(f"low-rank product past bf16 T={T} N={N} {dtype}")
    H, R = 128, 8
    x = torch.zeros(T, H, dtype=dtype)
    x[:, :3] = 1.0
    a, b = torch.zeros(1, R, H, dtype=dtype), torch.zeros(1, N, R, dtype=dtype)
    a[0, 5, 0], a[0, 5, 1], a[0, 5, 2] = 2.0 ** 127, 2.0 ** 126, 2.0 ** 126 - 2.0 ** 118     # their sum: TOP
    b[0, :, 5], b[0, 1::2, 5] = 2.0 ** -120, -2.0 ** -121
    y = tr.adapter_linear(x.cuda(), torch.zeros(N, H, dtype=dtype).cuda(), a.cuda(), b.cuda(),
                          torch.zeros(T, dtype=torch.int32).cuda())
    want = (TOP * b[0, :, 5].double()).to(dtype).expand(T, N)
    assert torch.equal(y.cpu(), want)
