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
