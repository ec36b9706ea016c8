"""Prompts of the block in 8 and 4 bits as examples/serving_block_mx.py runs it."""

import pytest
import torch

import top_reduce_amd as tr
from examples import serving_block_mx as B
from tests._gpu import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [256, 257, 700])
@pytest.mark.parametrize("bits", [8, 4])
def test_prompt(T, bits):
    say(f"block T={T} bits={bits}")
    block = B.Block(512, 128, 16, 8, 4, bits)
    x, r = B.tokens(T, 512, T)
    got = block(x, r)
    assert torch.isfinite(got[0].float()).all() and (got[0] != 0).any()
    # the projection with x in 8 bits: half a step of a number's binade, 2^-4 of itself at most
    few = tr.linear_mx4(x, block.w).double()
    many = block.project(x).double()
    assert many.shape == few.shape and float((many - few).norm()) <= 2.0 ** -4 * float(few.norm())
    assert torch.equal(many, few) == (T <= B.FEW)
    # and its rows are a larger prompt's
    more = block.project(torch.cat([x, x[:300]]))
    assert torch.equal(more[T:], more[:300][:more.shape[0] - T])
