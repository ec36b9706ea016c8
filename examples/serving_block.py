"""One block of a served mixture-of-experts model with an adapter per request:
a projection that all requests share with each request's low-rank adapter beside
it, the router, this GPU's experts.

A decode batch is two calls (adapter_linear, layer), captured once into a HIP
graph and replayed with the next tokens. A prompt goes through the router and the
plan, so that the routes are at hand for what exchanges rows between GPUs
(adapter_linear, route_topk, plan, forward).

    python examples/serving_block.py                 # decode of 64 and a prompt of 4096
    python examples/serving_block.py --T 8 --prompt 0 --steps 100
"""

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import top_reduce_amd as tr  # noqa: E402


class Block:
    """Weights of a block on the current device. The experts held here are
    [begin, begin + E) of G."""

    def __init__(self, H, I, G, E, K, A, R, begin=0, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

        self.K, self.E, self.begin = K, E, begin
        self.w = normal(H, H, std=H ** -0.5)
        self.a = normal(A, R, H, std=H ** -0.5)
        self.b = normal(A, H, R, std=R ** -0.5)
        self.scales = torch.rand(A, generator=g, device="cuda") + 0.5
        self.gate = normal(G, H, std=1.5 * H ** -0.5)
        self.w1 = torch.stack([normal(2 * I, H, std=H ** -0.5) for _ in range(E)])
        self.w2 = torch.stack([normal(H, I, std=I ** -0.5) for _ in range(E)])

    def project(self, x, ids, ws=None):
        """x w^T with the adapters that ids (int32 [T], -1: none) names."""
        return tr.adapter_linear(x, self.w, self.a, self.b, ids, scales=self.scales, ws=ws)

    def decode(self, x, ids, ws=None):
        """(output, idx, weights) of a batch of single tokens. ws: the
        workspaces of `workspaces`, or None to allocate."""
        h = self.project(x, ids, ws and ws[0])
        y, idx, weights = tr.layer(h, self.gate, self.w1, self.w2, self.K, expert_begin=self.begin,
                                   ws=ws and ws[1])
        return h + y, idx, weights

    def prompt(self, x, ids):
        """(output, idx, weights) of many tokens, by way of the plan."""
        h = self.project(x, ids)
        idx, weights = tr.route_topk(h, self.gate, self.K)
        p = tr.plan(idx, E=self.E, H=h.shape[1], I=self.w2.shape[2], dtype=h.dtype,
                    expert_begin=self.begin)
        return h + tr.forward(p, h, weights, self.w1, self.w2), idx, weights

    def workspaces(self, T):
        N, H = self.w.shape
        A, R = self.a.shape[:2]
        sizes = (tr.adapter_workspace_size(T, H, N, R, A, self.w.dtype),
                 tr.layer_workspace_size(T, N, self.w2.shape[2], self.E, self.gate.shape[0], self.K,
                                         self.w.dtype))
        return tuple(torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes)


class DecodeGraph:
    """A decode step of T tokens as one graph: fill x and ids, replay, read out."""

    def __init__(self, block, T):
        H = block.w.shape[1]
        self.x = torch.zeros(T, H, dtype=block.w.dtype, device="cuda")
        self.ids = torch.full((T,), -1, dtype=torch.int32, device="cuda")
        ws = block.workspaces(T)
        block.decode(self.x, self.ids, ws)      # loads the kernels before the capture
        torch.cuda.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.out, self.idx, self.weights = block.decode(self.x, self.ids, ws)
        self.ws = ws

    def step(self, x, ids):
        self.x.copy_(x)
        self.ids.copy_(ids)
        self.graph.replay()
        return self.out


def tokens(T, H, A, run, dtype, seed):
    """Inputs of T tokens whose requests have `run` tokens each; one request in
    ten has no adapter."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, H, generator=g, device="cuda").to(dtype)
    n = -(-T // run)
    ids = torch.randint(0, A, (n,), generator=g, device="cuda", dtype=torch.int32)
    ids[torch.rand(n, generator=g, device="cuda") < 0.1] = -1
    return x, ids.repeat_interleave(run)[:T].contiguous()


def timed(what, step, steps):
    for _ in range(3):
        step()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(steps):
        step()
    torch.cuda.synchronize()
    print(f"{what}: {(time.perf_counter() - t) * 1e6 / steps:.1f} us", flush=True)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("T", 64), ("prompt", 4096), ("H", 7168), ("I", 2048), ("G", 256), ("E", 32),
                        ("K", 8), ("A", 16), ("R", 32), ("run", 512), ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    block = Block(a.H, a.I, a.G, a.E, a.K, a.A, a.R)
    if a.T:
        x, ids = tokens(a.T, a.H, a.A, 1, block.w.dtype, 1)
        timed(f"decode of {a.T}, calls", lambda: block.decode(x, ids), a.steps)
        graph = DecodeGraph(block, a.T)
        timed(f"decode of {a.T}, graph", lambda: graph.step(x, ids), a.steps)
        local = int(((graph.idx >= 0) & (graph.idx < a.E)).sum())
        print(f"  {local} of {a.T * a.K} routes are local", flush=True)
    if a.prompt:
        x, ids = tokens(a.prompt, a.H, a.A, a.run, block.w.dtype, 2)
        timed(f"prompt of {a.prompt}", lambda: block.prompt(x, ids), a.steps)


if __name__ == "__main__":
    main()
