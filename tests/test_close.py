"""What the norm-wise checks of tests/_close.py let through and what they reject:
operators computed on the CPU, soundly and with a fault."""

import pytest
import torch

from tests import _close as C
from tests import _serving as S

BF, F32 = torch.bfloat16, torch.float32


def split16(v):
    hi = v.to(BF).float()
    return hi + (v - hi).to(BF).float()


def layer_inputs(T, H, I, E, K, dtype):
    g = torch.Generator().manual_seed(T + H + I)
    x = S.inputs(g, T, H, dtype=dtype)
    w1 = S.inputs(g, E, 2 * I, H, dtype=dtype, std=H ** -0.5)
    w2 = S.inputs(g, E, H, I, dtype=dtype, std=I ** -0.5)
    idx = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)])
    w = torch.rand(T, K, generator=g) + 0.2
    return x, idx, w / w.sum(1, keepdim=True), w1, w2


def layer_f32(x, idx, w, w1, w2, fault=None):
    """The layer as the kernels round it, in fp32."""
    dt, I = x.dtype, w2.shape[2]
    if fault == "bf16 operands":
        x, w1, w2 = (t.to(BF).float() for t in (x, w1, w2))
    x, w1, w2 = x.float(), w1.float(), w2.float()
    y = torch.zeros(x.shape)
    for e in range(w1.shape[0]):
        t, k = (idx == e).nonzero(as_tuple=True)
        if fault == "an expert" and e == int(idx[0, 0]):
            continue
        gu = x[t] @ w1[e].t()
        h = w[t, k][:, None].float() * (gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:])
        if dt == BF:
            h = h.to(BF).float() if fault == "h in 8 bits" else split16(h)
        if fault == "a part":
            h[:, :-(-I // 4)] = 0.0
        y[t] += h @ w2[e].t()
    return (torch.zeros_like(y) if fault == "zero" else y).to(dt)


SHAPES = [(1, 96, 1800, 32, 32), (8, 512, 2051, 16, 4), (64, 72, 1536, 24, 6), (9, 136, 1030, 40, 5),
          (16, 256, 128, 8, 2), (29, 264, 130, 5, 4), (3, 7168, 24, 4, 2), (64, 256, 2048, 2, 2)]


@pytest.mark.parametrize("T,H,I,E,K", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_layers(T, H, I, E, K, dtype):
    args = layer_inputs(T, H, I, E, K, dtype)
    want, _ = S.layer(*args, 0)
    n = H + I * K
    assert C.misses(layer_f32(*args), want, n, dtype) is None
    faults = ["zero", "an expert", "a part"]
    if dtype == F32:
        faults.append("bf16 operands")
    elif T * H >= 2000:        # enough elements to tell
        faults.append("h in 8 bits")
    for fault in faults:
        assert C.misses(layer_f32(*args, fault), want, n, dtype), fault


def adapter_f32(x, w, a, b, ids, scales, fault=None):
    dt = x.dtype
    if fault == "bf16 operands":
        x, w, a, b = (t.to(BF).float() for t in (x, w, a, b))
    x, w, a, b = x.float(), w.float(), a.float(), b.float()
    if fault == "a part":
        x = x.clone()
        x[:, :x.shape[1] // 4] = 0.0
    y = x @ w.t()
    for i in range(a.shape[0]):
        t = (ids == i).nonzero()[:, 0]
        if fault == "an adapter" and i == int(ids.max()):
            continue
        v = float(scales[i]) * (x[t] @ a[i].t())
        if dt == BF:
            v = v.to(BF).float() if fault == "v in 8 bits" else split16(v)
        y[t] += v @ b[i].t()
    return (torch.zeros_like(y) if fault == "zero" else y).to(dt)


@pytest.mark.parametrize("T,H,N,R,A", [(1, 3584, 512, 16, 8), (16, 256, 256, 12, 4), (64, 512, 256, 256, 9),
                                       (130, 264, 129, 12, 3), (513, 2880, 250, 256, 4), (16, 4104, 2000, 20, 3)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_projections(T, H, N, R, A, dtype):
    g = torch.Generator().manual_seed(T + N)
    args = (S.inputs(g, T, H, dtype=dtype), S.inputs(g, N, H, dtype=dtype, std=H ** -0.5),
            S.inputs(g, A, R, H, dtype=dtype, std=H ** -0.5), S.inputs(g, A, N, R, dtype=dtype, std=R ** -0.5),
            torch.arange(T, dtype=torch.int32) % A, torch.rand(A, generator=g) + 0.5)
    want, _ = S.adapter(*args)
    assert C.misses(adapter_f32(*args), want, H + R, dtype) is None
    faults = ["zero", "an adapter", "a part"]
    if dtype == F32:
        faults.append("bf16 operands")
    elif T * N >= 2000:
        faults.append("v in 8 bits")
    for fault in faults:
        assert C.misses(adapter_f32(*args, fault), want, H + R, dtype), fault
