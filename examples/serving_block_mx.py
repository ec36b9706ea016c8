"""One block of a served mixture-of-experts model in 8 and 4 bits: a projection with
weights in 4 bits, the residual's addition and the norm, the router, this GPU's experts.

    h = x w^T;  r' = h + r;  n = norm(r'), in bf16 for the router and in 8 bits for the experts
    y = this GPU's share of the experts' outputs for n

The same calls (linear_mx4, rms_norm, route_topk, plan, forward_mx) take a decode batch,
captured once into a HIP graph and replayed with the next tokens, and a prompt, whose
projection is a product in 8 bits (quantize_mx, expert_linear with one expert): linear_mx4
is for few rows.

    python examples/serving_block_mx.py                        # decode of 64 and a prompt of 4096
    python examples/serving_block_mx.py --T 1 --prompt 0 --bits 4 --steps 100
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import top_reduce_amd as tr  # noqa: E402
from examples.serving_block import timed  # noqa: E402


# Rows of x up to which linear_mx4 is the faster one. 256 / 512 / 4096 rows, 7168 x 7168: 33 / 67 /
# 470 us, against 33 / 41 / 185 with x in 8 bits.
FEW = 256


class Block:
    """Weights of a block on the current device: the projection's in 4 bits, the experts' in
    `bits`. The experts held here are [begin, begin + E) of G."""

    def __init__(self, H, I, G, E, K, bits=8, begin=0, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)

        def experts(N, K):
            pairs = [tr.quantize_mx(normal(N, K, std=K ** -0.5), bits) for _ in range(E)]
            return tuple(torch.stack([p[i].view(torch.uint8) for p in pairs]).view(pairs[0][i].dtype) for i in (0, 1))

        self.H, self.I, self.K, self.E, self.begin = H, I, K, E, begin
        self.w = tr.quantize_mx(normal(H, H, std=H ** -0.5), 4)
        self.all = torch.tensor([0, 2 ** 31 - 1], dtype=torch.int32, device="cuda")     # one expert's: every row
        self.norm = normal(H, std=0.2) + 1
        self.gate = normal(G, H, std=1.5 * H ** -0.5)
        self.w1, self.w2 = experts(2 * I, H), experts(H, I)

    def project(self, x):
        if x.shape[0] <= FEW:
            return tr.linear_mx4(x, self.w)
        return tr.expert_linear(tr.quantize_mx(x), tuple(t[None] for t in self.w), self.all)

    def __call__(self, x, residual):
        """(y, next residual, idx, weights) of rows x [T, H] and their residuals."""
        n = tr.rms_norm(self.project(x), self.norm, residual=residual, out="both")
        idx, weights = tr.route_topk(n.y, self.gate, self.K)
        p = tr.plan(idx, E=self.E, H=self.H, I=self.I, expert_begin=self.begin, flags=tr.FLAG_NO_XE)
        return tr.forward_mx(p, (n.q, n.s), weights, self.w1, self.w2), n.residual, idx, weights


class DecodeGraph:
    """A step of T tokens as one graph: fill x and residual, replay, read out."""

    def __init__(self, block, T):
        self.x = torch.zeros(T, block.H, dtype=torch.bfloat16, device="cuda")
        self.residual = torch.zeros_like(self.x)
        block(self.x, self.residual)            # loads the kernels before the capture
        torch.cuda.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.out = block(self.x, self.residual)

    def step(self, x, residual):
        self.x.copy_(x)
        self.residual.copy_(residual)
        self.graph.replay()
        return self.out


def tokens(T, H, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, r = (torch.randn(T, H, generator=g, device="cuda") for _ in range(2))
    return x.to(torch.bfloat16), (3 * r).to(torch.bfloat16)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("T", 64), ("prompt", 4096), ("H", 7168), ("I", 2048), ("G", 256), ("E", 32), ("K", 8),
                        ("bits", 8), ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    block = Block(a.H, a.I, a.G, a.E, a.K, a.bits)
    if a.T:
        x, r = tokens(a.T, a.H, 1)
        timed(f"decode of {a.T}, calls", lambda: block(x, r), a.steps)
        graph = DecodeGraph(block, a.T)
        timed(f"decode of {a.T}, graph", lambda: graph.step(x, r), a.steps)
        local = int(((graph.out[2] >= 0) & (graph.out[2] < a.E)).sum())
        print(f"  {local} of {a.T * a.K} routes are local", flush=True)
    if a.prompt:
        x, r = tokens(a.prompt, a.H, 2)
        timed(f"prompt of {a.prompt}", lambda: block(x, r), a.steps)


if __name__ == "__main__":
    main()
