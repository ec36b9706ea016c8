"""Calls on a stream that is not the current one, without a workspace or outputs
of the caller's: the current stream's next allocations must not meet the call's."""

import pytest
import torch

import top_reduce_amd as tr
from tests import _serving as S
from tests._gpu import say

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def cases(T, dtype):
    g = torch.Generator().manual_seed(T)
    H, I, E, G, K, R, A = 512, 160, 16, 16, 4, 24, 5
    x, gate, w1, w2, w, a, b = (S.inputs(g, *shape, dtype=dtype, std=std).cuda() for shape, std in (
        ((T, H), 1.0), ((G, H), 1.5 * H ** -0.5), ((E, 2 * I, H), H ** -0.5), ((E, H, I), I ** -0.5),
        ((H, H), H ** -0.5), ((A, R, H), H ** -0.5), ((A, H, R), R ** -0.5)))
    ids = (torch.arange(T) % (A + 1) - 1).to(torch.int32).cuda()
    return {"route_topk": (lambda **kw: tr.route_topk(x, gate, K, **kw),
                           tr.route_workspace_size(T, H, G, K, dtype)),
            "layer": (lambda **kw: tr.layer(x, gate, w1, w2, K, **kw),
                      tr.layer_workspace_size(T, H, I, E, G, K, dtype)),
            "adapter_linear": (lambda **kw: (tr.adapter_linear(x, w, a, b, ids, **kw),),
                               tr.adapter_workspace_size(T, H, H, R, A, dtype))}


@pytest.mark.parametrize("name", ["route_topk", "layer", "adapter_linear"])
@pytest.mark.parametrize("T,dtype", [(3, BF), (40, BF), (700, BF), (200, F32)])
def test_calls_on_another_stream_keep_their_memory(name, T, dtype):
    say(f"other stream {name} T={T} {dtype}")
    call, need = cases(T, dtype)[name]
    want = [t.clone() for t in call()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    big = torch.randn(2048, 2048, device="cuda")
    torch.cuda.synchronize()
    got = []
    with torch.cuda.stream(s):      # keeps the stream busy, so that the calls wait in it
        for _ in range(8):
            big = big @ big * 1e-3
    for _ in range(3):
        got.append(call(stream=s))
        # the current stream takes memory of the workspace's and the outputs' sizes, and writes it
        for n in (need, *(t.numel() * t.element_size() for t in want)):
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)
    s.synchronize()
    for out in got:
        assert all(torch.equal(u, v) for u, v in zip(out, want))


@pytest.mark.parametrize("name", ["route_topk", "layer", "adapter_linear"])
def test_outputs_stay_while_the_current_stream_uses_them(name):
    call, _ = cases(40, BF)[name]
    want = [t.clone() for t in call()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    big = torch.randn(2048, 2048, device="cuda")
    out = call(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for _ in range(8):              # the copies below wait behind these
        big = big @ big * 1e-3
    copies = [t.clone() for t in out]
    del out
    for _ in range(4):              # the other stream's next calls write their own outputs
        for t in call(stream=s):
            with torch.cuda.stream(s):
                t.zero_()
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(copies, want))
