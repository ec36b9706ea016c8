"""The projection with adapters, the router and the layer together, as
examples/serving_block.py runs them."""

import pytest
import torch

from examples import serving_block as B
from tests import _serving as S
from tests._gpu import say

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def check(block, x, ids, out, idx, weights, few):
    h = block.project(x, ids)      # the same bits again
    ref, bound = S.adapter(x, block.w, block.a, block.b, ids, block.scales)
    S.check(h, ref, bound, "projection")
    ref_idx, ref_w, tol, keys = S.route(h, block.gate, block.K)
    top = torch.sort(keys, dim=1, descending=True)[0][:, :block.K + 1]
    clear = ((top[:, :-1] - top[:, 1:]) > 1e-4).all(1)
    assert torch.equal(idx.cpu()[clear], ref_idx[clear])
    S.check(weights.cpu()[clear], ref_w[clear], tol[clear], "weights")
    y, bound = S.layer(h, idx, weights, block.w1, block.w2, block.begin, few=few)
    # the layer's output and the sum are rounded
    ref = S.f64(h) + y
    S.check(out, ref, bound + S.U[h.dtype] * (ref.abs() + bound), "output")


@pytest.mark.parametrize("T,dtype", [(1, BF), (7, BF), (48, BF), (64, F32)])
def test_decode_calls_and_graph(T, dtype):
    say(f"block decode T={T} {dtype}")
    block = B.Block(H=256, I=128, G=16, E=8, K=4, A=5, R=12, begin=4, dtype=dtype)
    graph = B.DecodeGraph(block, T)
    for seed in range(3):
        x, ids = B.tokens(T, 256, 5, 1, dtype, seed)
        out, idx, weights = block.decode(x, ids)
        check(block, x, ids, out, idx, weights, few=True)
        assert torch.equal(graph.step(x, ids), out)
        assert torch.equal(graph.idx, idx) and torch.equal(graph.weights, weights)


@pytest.mark.parametrize("T,dtype", [(65, BF), (700, BF), (200, F32)])
def test_prompt(T, dtype):
    say(f"block prompt T={T} {dtype}")
    block = B.Block(H=512, I=192, G=16, E=8, K=4, A=5, R=16, begin=8, dtype=dtype)
    x, ids = B.tokens(T, 512, 5, 40, dtype, T)
    check(block, x, ids, *block.prompt(x, ids), few=False)
