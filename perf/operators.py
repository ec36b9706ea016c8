"""Cases that measure the serving operators around the expert MLP.

Three operators, all for inference:

* ``route``: the router. Logits of every token against the gate's rows, a
  softmax or sigmoid score, the K best experts (ties to the lowest id) and
  their gate weights.
* ``layer``: a whole mixture-of-experts layer for a few tokens: the router,
  the local experts' SwiGLU MLPs and their weighted sum.
* ``adapter``: a projection that all requests share, with a low-rank adapter
  of its own for each token's request beside it.

``own`` false: the operators' formulas in elementary torch operations, in 32
bits, rounded once at the end. ``own`` true: the package's entry points.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

# Two scores that decide the order of a token's experts differ by at least
# this much: where they are closer, sums in another order give another order.
MARGIN = 5e-5


def listed():
    return [
        # The layer. One token of a chat against a model whose experts all
        # live here (the hidden and intermediate sizes of workload c5).
        {"name": "layer one token", "op": "layer", "T": 1, "H": 7168, "I": 2048, "E": 32, "G": 32,
         "K": 8, "begin": 0, "dtype": "bf16", "score": "softmax", "renorm": True, "bias": False,
         "scale": 1.0},
        # A decode batch on one of 32 ranks (workload c3's sizes): few routes
        # are local, and most tokens have none.
        {"name": "layer decode share", "op": "layer", "T": 8, "H": 3584, "I": 2048, "E": 28,
         "G": 896, "K": 16, "begin": 140, "dtype": "bf16", "score": "softmax", "renorm": True,
         "bias": False, "scale": 1.0},
        # A larger decode batch on one of 8 ranks: most local experts get one
        # to four tokens; the sigmoid score with a balancing bias.
        {"name": "layer decode 64", "op": "layer", "T": 64, "H": 7168, "I": 2048, "E": 32, "G": 256,
         "K": 8, "begin": 96, "dtype": "bf16", "score": "sigmoid", "renorm": True, "bias": True,
         "scale": 2.5},
        # Sizes that fill no tile (the package's own 2880 x 1440 test shape).
        {"name": "layer odd", "op": "layer", "T": 7, "H": 2880, "I": 1440, "E": 32, "G": 32, "K": 4,
         "begin": 0, "dtype": "bf16", "score": "softmax", "renorm": False, "bias": False,
         "scale": 1.0},
        # The smallest model in full precision (workload c1's sizes): latency.
        {"name": "layer tiny f32", "op": "layer", "T": 16, "H": 256, "I": 128, "E": 8, "G": 8, "K": 2,
         "begin": 0, "dtype": "f32", "score": "softmax", "renorm": True, "bias": False,
         "scale": 1.0},
        # The router alone. One decoded token against 896 experts.
        {"name": "route one token", "op": "route", "T": 1, "H": 3584, "G": 896, "K": 16,
         "dtype": "bf16", "score": "softmax", "renorm": True, "bias": False, "scale": 1.0},
        # A prefill of 16384 tokens (workload c5's sizes).
        {"name": "route prefill", "op": "route", "T": 16384, "H": 7168, "G": 256, "K": 8,
         "dtype": "bf16", "score": "sigmoid", "renorm": True, "bias": True, "scale": 2.5},
        # A mixed batch in full precision, with an odd number of experts.
        {"name": "route mixed f32", "op": "route", "T": 961, "H": 2880, "G": 60, "K": 4,
         "dtype": "f32", "score": "softmax", "renorm": False, "bias": False, "scale": 1.0},
        # Adapters. One decode step of eight requests with eight adapters.
        {"name": "adapter decode 8", "op": "adapter", "T": 8, "H": 3584, "N": 3584, "R": 16, "A": 8,
         "run": 1, "dtype": "bf16"},
        # A larger decode step, wide ranks.
        {"name": "adapter decode 64", "op": "adapter", "T": 64, "H": 7168, "N": 7168, "R": 64,
         "A": 24, "run": 1, "dtype": "bf16"},
        # Prompts of several hundred tokens each, sixteen adapters.
        {"name": "adapter prefill", "op": "adapter", "T": 8192, "H": 7168, "N": 7168, "R": 32,
         "A": 16, "run": 700, "dtype": "bf16"},
        # Short prompts in full precision, odd sizes.
        {"name": "adapter odd f32", "op": "adapter", "T": 333, "H": 1448, "N": 1001, "R": 12, "A": 5,
         "run": 40, "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    """An integer, uniform over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["layer", "route", "adapter"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    H = 8 * _log(rng, 32, 896)
    if rng.random() < 0.3:
        H = max(256, H // 256 * 256)
    if op == "adapter":
        N = _log(rng, 250, 7168)
        if rng.random() < 0.5:
            N = max(256, N // 256 * 256)
        T = _log(rng, 1, 8192 if dtype == "bf16" else 1024)
        return {"op": op, "T": T, "H": H, "N": N, "R": _log(rng, 4, 64), "A": _log(rng, 1, 32),
                "run": _log(rng, 1, 512), "dtype": dtype}
    score = rng.choice(["softmax", "sigmoid"])
    case = {"op": op, "H": H, "dtype": dtype, "score": score, "renorm": rng.random() < 0.7,
            "bias": score == "sigmoid" and rng.random() < 0.6,
            "scale": rng.choice([1.0, 2.5])}
    if op == "route":
        G = _log(rng, 8, 896)
        return dict(case, T=_log(rng, 1, 16384 if dtype == "bf16" and G <= 256 else 2048), G=G,
                    K=min(G, _log(rng, 1, 16)))
    E = _log(rng, 2, 32)
    G = min(896, E * rng.choice([1, 1, 2, 8, 32]))
    inner = _log(rng, 64, 2048 if dtype == "bf16" else 512)
    if rng.random() < 0.4:
        inner = max(128, inner // 128 * 128)
    return dict(case, T=_log(rng, 1, 64), I=inner, E=E, G=G, K=min(G, _log(rng, 1, 16)),
                begin=E * rng.randrange(G // E))


def _keys(logits, bias, score):
    """What the experts are ordered by: the logits themselves (a softmax or
    sigmoid keeps their order), or the scores with the balancing bias."""
    if bias is None:
        return logits
    s = torch.exp(logits - logits.max(1, keepdim=True)[0])
    s = s / s.sum(1, keepdim=True) if score == "softmax" else 1 / (1 + torch.exp(-logits))
    return s + bias.to(logits.dtype)


def prepare(case, seed):
    dev, dt = "cuda", DTYPES[case["dtype"]]
    gen = torch.Generator(device=dev).manual_seed(seed)
    T, H = case["T"], case["H"]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device=dev, dtype=dt) * std

    x = normal(T, H)
    if case["op"] == "adapter":
        N, R, A = case["N"], case["R"], case["A"]
        # runs of tokens of one request; about one request in ten has no adapter
        n = -(-T // case["run"])
        ids = torch.randint(0, A, (n,), generator=gen, device=dev, dtype=torch.int32)
        ids[torch.rand(n, generator=gen, device=dev) < 0.1] = -1
        ids = ids.repeat_interleave(case["run"])[:T].contiguous()
        return {"case": case, "x": x, "w": normal(N, H, std=H ** -0.5),
                "a": normal(A, R, H, std=H ** -0.5), "b": normal(A, N, R, std=R ** -0.5), "ids": ids,
                "scales": torch.rand(A, generator=gen, device=dev) + 0.5}
    G, K = case["G"], case["K"]
    gate = normal(G, H, std=1.5 * H ** -0.5)
    bias = torch.randn(G, generator=gen, device=dev) * 0.02 if case["bias"] else None
    # A token whose order of experts hangs on rounding has no one answer: draw
    # such tokens again.
    for _ in range(20):
        keys = _keys(x.double() @ gate.double().t(), bias, case["score"])
        top = torch.topk(keys, min(K + 1, G), dim=1)[0]
        near = (top[:, :-1] - top[:, 1:] < MARGIN).any(1)
        if not bool(near.any()):
            break
        x[near] = normal(int(near.sum()), H)
    state = {"case": case, "x": x, "gate": gate, "bias": bias}
    if case["op"] == "layer":
        E, inner = case["E"], case["I"]
        state["w1"] = normal(E, 2 * inner, H, std=H ** -0.5)
        state["w2"] = normal(E, H, inner, std=inner ** -0.5)
    return state


def _route(x, gate, bias, case):
    logits = x.float() @ gate.float().t()
    order = torch.sort(_keys(logits, bias, case["score"]), dim=1, descending=True, stable=True)[1]
    idx = order[:, :case["K"]].contiguous()
    if case["score"] == "softmax":
        s = torch.exp(logits - logits.max(1, keepdim=True)[0])
        s = s / s.sum(1, keepdim=True)
    else:
        s = 1 / (1 + torch.exp(-logits))
    w = s.gather(1, idx)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return idx, w * case["scale"]


def _layer(s, case):
    idx, w = _route(s["x"], s["gate"], s["bias"], case)
    T, H, E, inner = case["T"], case["H"], case["E"], case["I"]
    # gates of the local experts as a dense [T, E] matrix
    all_gates = torch.zeros(T, case["G"], device=w.device).scatter_(1, idx, w)
    gates = all_gates[:, case["begin"]:case["begin"] + E]
    gu = (s["x"].float() @ s["w1"].float().view(E * 2 * inner, H).t()).view(T, E, 2, inner)
    g, u = gu[:, :, 0], gu[:, :, 1]
    h = g / (1 + torch.exp(-g)) * u * gates[:, :, None]
    y = h.reshape(T, E * inner) @ s["w2"].float().transpose(1, 2).reshape(E * inner, H)
    return {"y": y.to(s["x"].dtype), "idx": idx, "weights": w}


def _adapter(s, case):
    A, R, H, N = case["A"], case["R"], case["H"], case["N"]
    x, ids = s["x"].float(), s["ids"].long()
    mine = ids[:, None] == torch.arange(A, device=x.device)[None, :]
    v = (x @ s["a"].float().view(A * R, H).t()).view(-1, A, R)
    v = v * (mine * s["scales"][None, :])[:, :, None]
    y = x @ s["w"].float().t()
    y = y + v.view(-1, A * R) @ s["b"].float().transpose(1, 2).reshape(A * R, N)
    return y.to(s["x"].dtype)


def run(state):
    case = state["case"]
    if own:
        import top_reduce_amd as tr
        if case["op"] == "adapter":
            return tr.adapter_linear(state["x"], state["w"], state["a"], state["b"], state["ids"],
                                     scales=state["scales"])
        how = {"bias": state["bias"], "score": case["score"], "renorm": case["renorm"],
               "scale": case["scale"]}
        if case["op"] == "route":
            idx, w = tr.route_topk(state["x"], state["gate"], case["K"], **how)
            return {"idx": idx, "weights": w}
        y, idx, w = tr.layer(state["x"], state["gate"], state["w1"], state["w2"], case["K"],
                             expert_begin=case["begin"], **how)
        return {"y": y, "idx": idx, "weights": w}
    if case["op"] == "adapter":
        return _adapter(state, case)
    if case["op"] == "route":
        idx, w = _route(state["x"], state["gate"], state["bias"], case)
        return {"idx": idx, "weights": w}
    return _layer(state, case)


def work(case):
    b = 2 if case["dtype"] == "bf16" else 4
    T, H = case["T"], case["H"]
    if case["op"] == "adapter":
        N, R = case["N"], case["R"]
        # adapters that some token uses, were the requests' adapters uniform
        used = case["A"] * (1 - (1 - 0.9 / case["A"]) ** -(-T // case["run"]))
        return {"bytes": b * (T * H + N * H + T * N + used * R * (H + N)) + 4 * T,
                "flops": 2 * T * N * H + 0.9 * 2 * T * R * (H + N)}
    G, K = case["G"], case["K"]
    bytes_, flops = b * (T * H + G * H) + 12 * T * K, 2 * T * G * H
    if case["op"] == "layer":
        # local experts with a token and local routes, were the routes uniform
        active = case["E"] * (1 - (1 - K / G) ** T)
        routes = T * K * case["E"] / G
        bytes_ += b * (active * 3 * H * case["I"] + T * H)
        flops += routes * 6 * H * case["I"]
    return {"bytes": bytes_, "flops": flops}


def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"].double()
    T, H = case["T"], case["H"]
    if case["op"] == "adapter":
        y = x.matmul(s["w"].double().t())
        for k in range(case["A"]):
            rows = (s["ids"] == k).nonzero()[:, 0]
            low = x[rows].matmul(s["a"][k].double().t())
            y[rows] += s["scales"][k].double() * low.matmul(s["b"][k].double().t())
        return y
    K = case["K"]
    logits = torch.stack([x.matmul(g.double()) for g in s["gate"]], 1)
    p = torch.softmax(logits, 1) if case["score"] == "softmax" else torch.sigmoid(logits)
    idx = torch.topk(logits if s["bias"] is None else p + s["bias"].double(), K, dim=1)[1]
    w = torch.take_along_dim(p, idx, 1)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = w * case["scale"]
    if case["op"] == "route":
        return {"idx": idx, "weights": w}
    y = torch.zeros(T, H, dtype=torch.float64, device=x.device)
    for e in range(case["E"]):
        t, slot = (idx == case["begin"] + e).nonzero(as_tuple=True)
        if t.numel():
            gu = x[t].matmul(s["w1"][e].double().t())
            h = torch.nn.functional.silu(gu[:, :case["I"]]) * gu[:, case["I"]:]
            y[t] += w[t, slot][:, None] * h.matmul(s["w2"][e].double().t())
    return {"y": y, "idx": idx, "weights": w}
