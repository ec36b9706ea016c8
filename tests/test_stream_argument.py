"""stream= of the serving entry points, without a GPU: what the call allocates
by itself belongs to the stream that its kernels run on, and outputs stay the
caller's for as long as its own stream works on them."""

import contextlib

import pytest
import torch

from top_reduce_amd import _binding as B

DEV = torch.device("cuda", 0)
T, H, N, G, K, E, I, R, A = 3, 64, 48, 16, 2, 4, 32, 8, 5


class Stream:
    def __init__(self, handle, device=DEV):
        self.cuda_stream, self.device = handle, device


class Fake(torch.Tensor):
    """A host tensor that says it is on the GPU and notes what is done with it."""

    @property
    def device(self):
        return DEV

    @property
    def is_cuda(self):
        return True

    def record_stream(self, stream):
        self.recorded = stream


def fake(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Fake)


@pytest.fixture
def world(monkeypatch):
    """The binding with streams, allocations and kernel launches recorded."""
    w = type("World", (), {})()
    w.current, w.allocations, w.launched = Stream(0), [], []
    lib = B.load_library()

    @contextlib.contextmanager
    def on(stream):
        before, w.current = w.current, stream
        yield
        w.current = before

    def empty(*shape, dtype=None, device=None):
        t = fake(*shape, dtype=dtype)
        w.allocations.append((t, w.current.cuda_stream))
        return t

    class Lib:
        def __getattr__(self, name):
            real = getattr(lib, name)
            if name not in ("moe_route_topk", "moe_layer", "moe_adapter_linear"):
                return real

            def launch(*args):
                w.launched.append(args[-1])
                return 0
            return launch

    monkeypatch.setattr(B, "_lib", Lib())
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch, "empty_like", lambda t: empty(*t.shape, dtype=t.dtype))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: w.current)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: w.current.cuda_stream,
                        raising=False)
    return w


def calls():
    gate, w1, w2 = fake(G, H), fake(E, 2 * I, H), fake(E, H, I)
    w, a, b = fake(N, H), fake(A, R, H), fake(A, N, R)
    ids = fake(T, dtype=torch.int32)
    return {
        "route_topk": (lambda x, **kw: B.route_topk(x, gate, K, **kw),
                       lambda: dict(idx=fake(T, K, dtype=torch.int64), weights=fake(T, K, dtype=torch.float32))),
        "layer": (lambda x, **kw: B.layer(x, gate, w1, w2, K, **kw),
                  lambda: dict(y=fake(T, H), idx=fake(T, K, dtype=torch.int64),
                               weights=fake(T, K, dtype=torch.float32))),
        "adapter_linear": (lambda x, **kw: (B.adapter_linear(x, w, a, b, ids, **kw),),
                           lambda: dict(y=fake(T, N))),
    }


@pytest.mark.parametrize("name", ["route_topk", "layer", "adapter_linear"])
def test_what_a_call_allocates_belongs_to_its_stream(world, name):
    call, _ = calls()[name]
    out = call(fake(T, H), stream=Stream(7))
    assert world.launched == [7] and world.current.cuda_stream == 0
    assert len(world.allocations) == len(out) + 1            # the outputs and the workspace
    assert all(s == 7 for _, s in world.allocations)
    # the outputs go back to a caller whose own stream works on them
    assert all(t.recorded.cuda_stream == 0 for t in out)


@pytest.mark.parametrize("name", ["route_topk", "layer", "adapter_linear"])
def test_given_outputs_are_left_alone(world, name):
    call, outputs = calls()[name]
    given = outputs()
    out = call(fake(T, H), stream=Stream(7), **given)
    assert world.launched == [7]
    assert [id(t) for t in out] == [id(t) for t in given.values()]
    assert not any(hasattr(t, "recorded") for t in out)
    assert [s for _, s in world.allocations] == [7]          # the workspace


@pytest.mark.parametrize("name", ["route_topk", "layer", "adapter_linear"])
@pytest.mark.parametrize("stream", [None, Stream(0)])
def test_the_current_stream_takes_no_detour(world, name, stream):
    call, _ = calls()[name]
    out = call(fake(T, H), stream=stream)
    assert world.launched == [0]
    assert not any(hasattr(t, "recorded") for t in out)


@pytest.mark.parametrize("name", ["route_topk", "layer", "adapter_linear"])
def test_a_stream_of_another_device_is_refused(world, name):
    call, _ = calls()[name]
    with pytest.raises(ValueError, match="stream"):
        call(fake(T, H), stream=Stream(7, torch.device("cuda", 1)))
    assert not world.launched
