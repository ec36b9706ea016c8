"""The projection with adapters on integers, whose sums are exact in fp32 in any
order: y is the formula's value, rounded once. The low-rank products have up to 16
significant bits, so a product held in fewer gives other values, and so does any
operand, part of a sum or adapter that is left out."""

import pytest
import torch

import top_reduce_amd as tr
from tests._gpu import say

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def integers(gen, lo, hi, *shape):
    return torch.randint(lo, hi + 1, shape, generator=gen, device="cuda", dtype=torch.float64)


def run_exact(T, H, N, R, A, run, dtype, most_x=2, most_w=1, most_a=60, most_b=1):
    g = torch.Generator(device="cuda").manual_seed(T + N + R)
    x, w = integers(g, -most_x, most_x, T, H), integers(g, -most_w, most_w, N, H)
    a, b = integers(g, -most_a, most_a, A, R, H), integers(g, -most_b, most_b, A, N, R)
    ids = torch.randint(-1, A + 1, (-(-T // run),), generator=g, device="cuda", dtype=torch.int32)
    ids = ids.repeat_interleave(run)[:T].contiguous()
    scales = 2.0 ** torch.randint(-1, 2, (A,), generator=g, device="cuda").float()
    want = x @ w.t()
    for i in range(A):
        t = (ids == i).nonzero()[:, 0]
        v = float(scales[i]) * (x[t] @ a[i].t())
        # integers before their scale: 16 significant bits
        assert dtype == F32 or v.numel() == 0 or v.abs().max() < 2 ** 16 * float(scales[i])
        want[t] += v @ b[i].t()
        most = v.abs() @ b[i].abs().t() + x[t].abs() @ w.abs().t()
        assert most.numel() == 0 or most.max() < 2 ** 23    # every sum, in halves: below 2^24
    y = tr.adapter_linear(x.to(dtype), w.to(dtype), a.to(dtype), b.to(dtype), ids, scales=scales)
    assert torch.equal(y, want.float().to(dtype))


@pytest.mark.parametrize("T,H,N,R,A,run", [
    (1, 256, 130, 12, 2, 1), (9, 1032, 300, 33, 4, 1), (16, 7168, 7160, 16, 3, 1),    # streamed
    (40, 264, 257, 64, 9, 1), (64, 512, 1024, 256, 5, 3), (200, 1448, 301, 12, 5, 40),    # in parts
    (513, 280, 2048, 20, 4, 100), (700, 512, 4096, 256, 3, 9), (1000, 256, 2050, 8, 6, 1),    # 64 x 64
    (1000, 512, 4100, 40, 5, 300), (2048, 264, 4096, 17, 9, 1),    # 128 x 128, 128 x 256
    (4100, 128, 8192, 8, 4, 1), (4100, 256, 8192, 24, 4, 50), (8000, 384, 4352, 256, 2, 700),    # 256 x 256
])
def test_bf16(T, H, N, R, A, run):
    say(f"adapter exact T={T} H={H} N={N} R={R} A={A} run={run}")
    run_exact(T, H, N, R, A, run, BF)


@pytest.mark.parametrize("most", [dict(most_w=999, most_a=999), dict(most_x=999, most_a=1),
                                  dict(most_a=1, most_b=999)], ids=["weights", "x", "b"])
@pytest.mark.parametrize("T,H,N,R,A,run", [
    (1, 256, 130, 12, 2, 1), (16, 4104, 8200, 20, 3, 1), (40, 264, 257, 64, 9, 1), (200, 1448, 301, 12, 5, 40),
    (513, 280, 2048, 20, 4, 100), (1000, 512, 4100, 40, 5, 300), (2048, 264, 4096, 17, 9, 1),
])
def test_f32(T, H, N, R, A, run, most):
    """Operands of ten bits, one after another: rounded to eight they give other sums."""
    say(f"adapter exact fp32 T={T} H={H} N={N} R={R} A={A} run={run} {most}")
    run_exact(T, H, N, R, A, run, F32, **most)
