"""The block in 8 and 4 bits as examples/serving_block_mx.py runs it: the graph's replays
against the calls, and a batch's rows against a smaller one's."""

import pytest
import torch

from examples import serving_block_mx as B
from tests._gpu import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 5, 70])
@pytest.mark.parametrize("bits", [8, 4])
def test_graph_and_calls(T, bits):
    say(f"block T={T} bits={bits}")
    block = B.Block(512, 128, 16, 8, 4, bits)
    graph = B.DecodeGraph(block, T)
    for seed in range(3):
        x, r = B.tokens(T, 512, seed)
        want = block(x, r)
        got = graph.step(x, r)
        torch.cuda.synchronize()
        for u, v in zip(got, want):
            assert torch.equal(u, v)
        assert torch.isfinite(got[0].float()).all() and (got[0] != 0).any()


def test_experts_of_two_gpus_share_the_routes():
    """Two halves of the experts: the same routes, and each its own rows' share."""
    x, r = B.tokens(40, 512, 9)
    low = B.Block(512, 128, 16, 8, 4)
    high = B.Block(512, 128, 16, 8, 4, begin=8)
    a, b = low(x, r), high(x, r)
    assert torch.equal(a[2], b[2]) and torch.equal(a[3], b[3]) and torch.equal(a[1], b[1])
    mine = (a[2] < 8).any(1)
    assert (a[0][~mine] == 0).all() and (b[0][(a[2] >= 8).sum(1) == 0] == 0).all()
