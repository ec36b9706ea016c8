"""Cases that measure the operators of a layer served in 8 and 4 bits.

Rows and weights are held in blocks of 32 numbers along the reduction dimension:
elements of 8 bits (e4m3) or 4 (e2m1, two in a byte, the even one in the low half)
and one scale a block, a power of two in a byte of its own (e8m0). The scale is the
smallest power of two that brings the block's largest magnitude to 448 or below (6
for 4 bits), elements are rounded to the nearest, ties to the even one.

Three operators, all for inference:

* ``norm``: y = z / sqrt(mean(z^2) + eps) * weight with z = x + residual; y in the
  rows' type, in 8 bits with scales, or both; z is the next residual.
* ``experts``: the rows of each expert's segment, in 8 bits, times its weights, in 8
  or 4: plain, or as silu(gate) * up; in bfloat16, or in 8 bits with scales again.
  Segments are ragged, many may be empty; the rows may be read through a table.
* ``linear4``: a few rows in full types times weights in 4 bits.

``own`` false: the operators' formulas in elementary torch operations, in 32 bits,
rounded once at the end. ``own`` true: the package's entry points.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-6


def listed():
    return [
        # The norm before a block's router and experts (hidden size of workloads c2 and
        # c5): one decoded token, y for the router, 8 bits for the experts.
        {"name": "norm one token", "op": "norm", "T": 1, "H": 7168, "dtype": "bf16",
         "residual": True, "out": "both"},
        # The same for a prefill of 16384 tokens.
        {"name": "norm prefill", "op": "norm", "T": 16384, "H": 7168, "dtype": "bf16",
         "residual": True, "out": "both"},
        # A final norm in full precision, no residual, an odd batch.
        {"name": "norm odd f32", "op": "norm", "T": 961, "H": 2880, "dtype": "f32",
         "residual": False, "out": "same"},
        # One token's eight experts, up projection: eight experts with a row each.
        {"name": "experts one token up", "op": "experts", "T": 1, "R": 8, "K": 7168, "N": 4096,
         "E": 32, "bits": 8, "skew": -1.0, "swiglu": True, "out": "mx8", "gather": True},
        # A decode batch of 64 tokens on one of 8 ranks: 64 routes over 32 experts.
        {"name": "experts decode up w4", "op": "experts", "T": 64, "R": 64, "K": 7168, "N": 4096,
         "E": 32, "bits": 4, "skew": 0.0, "swiglu": True, "out": "mx8", "gather": True},
        {"name": "experts decode down", "op": "experts", "T": 64, "R": 64, "K": 2048, "N": 7168,
         "E": 32, "bits": 8, "skew": 0.0, "swiglu": False, "out": "bf16", "gather": False},
        # A prefill with uneven experts (workload c5's sizes and Zipf routing).
        {"name": "experts prefill up", "op": "experts", "T": 16384, "R": 16384, "K": 7168, "N": 4096,
         "E": 32, "bits": 8, "skew": 1.0, "swiglu": True, "out": "mx8", "gather": True},
        {"name": "experts prefill down", "op": "experts", "T": 16384, "R": 16384, "K": 2048,
         "N": 7168, "E": 32, "bits": 8, "skew": 1.0, "swiglu": False, "out": "bf16", "gather": False},
        # A mixed batch at sizes that fill no tile (the package's 2880 x 1440 test shape).
        {"name": "experts odd w4", "op": "experts", "T": 333, "R": 961, "K": 2880, "N": 1440, "E": 12,
         "bits": 4, "skew": 0.5, "swiglu": False, "out": "bf16", "gather": True},
        # Projections in 4 bits: one decoded token.
        {"name": "linear4 one token", "op": "linear4", "T": 1, "K": 7168, "N": 7168, "dtype": "bf16"},
        # A decode batch.
        {"name": "linear4 decode 64", "op": "linear4", "T": 64, "K": 7168, "N": 7168,
         "dtype": "bf16"},
        # A small projection in full precision, odd sizes.
        {"name": "linear4 odd f32", "op": "linear4", "T": 5, "K": 1440, "N": 1001, "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    """An integer, uniform over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "experts", "experts", "linear4"])
    if op == "norm":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        out = rng.choice(["same", "mx8", "both"])
        T = _log(rng, 1, 16384 if dtype == "bf16" else 4096)
        H = 8 * _log(rng, 8, 896) if out == "same" else 32 * _log(rng, 2, 224)
        return {"op": op, "T": T, "H": H, "dtype": dtype, "residual": rng.random() < 0.7, "out": out}
    K = 32 * _log(rng, 4, 224)
    if rng.random() < 0.5:
        K = max(128, K // 128 * 128)
    if op == "linear4":
        return {"op": op, "T": _log(rng, 1, 64), "K": K, "N": _log(rng, 32, 7168),
                "dtype": rng.choice(["bf16", "bf16", "f32"])}
    swiglu = rng.random() < 0.5
    out = rng.choice(["bf16", "mx8"])
    N = 64 * _log(rng, 1, 64) if out == "mx8" else 2 * _log(rng, 40, 3584)
    R = _log(rng, 1, 8192)
    gather = rng.random() < 0.6
    return {"op": op, "T": max(1, R // rng.choice([1, 2, 4])) if gather else R, "R": R, "K": K, "N": N,
            "E": _log(rng, 1, 32), "bits": rng.choice([8, 4]), "skew": rng.choice([0.0, 0.5, 1.0]),
            "swiglu": swiglu, "out": out, "gather": gather}


def _to_mx(v, bits):
    """(q, s) of 32-bit numbers along the last dimension."""
    v = v.float()
    b = v.reshape(*v.shape[:-1], -1, 32)
    top = b.abs().amax(-1, keepdim=True).double() / (448.0 if bits == 8 else 6.0)
    m, e = torch.frexp(top)
    e = torch.where(m == 0.5, e - 1, e)
    e = torch.where(m == 0, -127, e).clamp(-127, 127)
    b = torch.ldexp(b, -e).float()
    s = (e + 127).to(torch.uint8).squeeze(-1).view(torch.float8_e8m0fnu)
    if bits == 8:
        return b.reshape(v.shape).to(torch.float8_e4m3fn), s
    a = b.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5)
            + (a > 5.0) + 8 * torch.signbit(b))
    code = code.to(torch.uint8).reshape(*v.shape[:-1], -1, 2)
    return code[..., 0] + 16 * code[..., 1], s


def _from_mx(q, s, dtype=torch.float32):
    """The numbers that (q, s) stands for."""
    if q.dtype == torch.uint8:
        table = torch.tensor(E2M1 + tuple(-t for t in E2M1), dtype=dtype, device=q.device)
        v = torch.stack([table[(q & 15).int()], table[(q >> 4).int()]], -1)
    else:
        v = q.to(dtype)
    v = v.reshape(*s.shape, 32) * s.to(dtype)[..., None]
    return v.reshape(*s.shape[:-1], -1)


def _odds(case):
    p = [(e + 1) ** -case["skew"] for e in range(case["E"])]
    return [v / sum(p) for v in p]


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device=dev, dtype=dtype) * std

    state = {"case": case}
    if case["op"] == "norm":
        T, H, dt = case["T"], case["H"], DTYPES[case["dtype"]]
        state["x"] = normal(T, H, dtype=dt)
        # a residual stream is larger than what a block adds, and a few of its columns
        # far larger
        if case["residual"]:
            wide = torch.where(torch.rand(H, generator=gen, device=dev) < 0.01, 30.0, 3.0)
            state["residual"] = (normal(T, H) * wide).to(dt)
        state["weight"] = (normal(H, std=0.2) + 1.0).to(dt)
        return state
    K, N = case["K"], case["N"]
    if case["op"] == "linear4":
        state["x"] = normal(case["T"], K, dtype=DTYPES[case["dtype"]])
        state["w"] = _to_mx(normal(N, K, std=K ** -0.5), 4)
        return state
    T, R, E = case["T"], case["R"], case["E"]
    state["x"] = _to_mx(normal(T, K), 8)
    if case["skew"] < 0:    # a row each for R of the experts
        ids = torch.randperm(E, generator=gen, device=dev)[:R]
    else:
        p = torch.tensor(_odds(case), device=dev)[torch.randperm(E, generator=gen, device=dev)]
        ids = torch.multinomial(p, R, replacement=True, generator=gen)
    counts = (ids[None, :] == torch.arange(E, device=dev)[:, None]).sum(1)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=dev)
    offsets[1:] = counts.cumsum(0)
    state["offsets"], state["longest"] = offsets, int(counts.max())
    state["rows"] = None
    if case["gather"]:      # by expert, then by row
        rows = torch.randint(0, T, (R,), generator=gen, device=dev)
        order = torch.sort(torch.sort(ids)[0] * T + rows)[0]
        state["rows"] = (order % T).to(torch.int32)
    w = [_to_mx(normal(N, K, std=K ** -0.5), case["bits"]) for _ in range(E)]
    state["w"] = (torch.stack([q for q, _ in w]),
                  torch.stack([s.view(torch.uint8) for _, s in w]).view(torch.float8_e8m0fnu))
    return state


def _norm(s, case):
    z = s["x"].float()
    if case["residual"]:
        z = z + s["residual"].float()
    y = z / torch.sqrt((z * z).mean(1, keepdim=True) + EPS) * s["weight"].float()
    q, e = _to_mx(y, 8) if case["out"] != "same" else (None, None)
    dt = s["x"].dtype
    return {"y": None if case["out"] == "mx8" else y.to(dt), "q": q, "s": e,
            "residual": z.to(dt) if case["residual"] else None}


def _experts(s, case):
    E, R = case["E"], case["R"]
    x, offsets = _from_mx(*s["x"]), s["offsets"].long()
    at = torch.arange(s["longest"], device=x.device)[None, :] + offsets[:-1, None]     # [E, longest]
    mine = at < offsets[1:, None]
    at = at.clamp(max=R - 1)
    rows = at if s["rows"] is None else s["rows"].long()[at]
    y = torch.bmm(x[rows], _from_mx(*s["w"]).transpose(1, 2))
    y = y[mine]     # expert by expert: the rows in order
    if case["swiglu"]:
        g, u = y[:, :case["N"] // 2], y[:, case["N"] // 2:]
        y = g / (1 + torch.exp(-g)) * u
    if case["out"] == "bf16":
        return {"y": y.to(torch.bfloat16)}
    q, e = _to_mx(y, 8)
    return {"q": q, "s": e}


def run(state):
    case = state["case"]
    if own:
        import top_reduce_amd as tr
        if case["op"] == "norm":
            r = tr.rms_norm(state["x"], state["weight"], EPS, residual=state.get("residual"),
                            out=case["out"])
            return {"y": r.y, "q": r.q, "s": r.s, "residual": r.residual}
        if case["op"] == "linear4":
            return {"y": tr.linear_mx4(state["x"], state["w"])}
        r = tr.expert_linear(state["x"], state["w"], state["offsets"], rows=state["rows"],
                             swiglu=case["swiglu"], out=case["out"])
        return {"y": r} if case["out"] == "bf16" else {"q": r[0], "s": r[1]}
    if case["op"] == "norm":
        return _norm(state, case)
    if case["op"] == "linear4":
        x = state["x"]
        return {"y": (x.float() @ _from_mx(*state["w"]).t()).to(x.dtype)}
    return _experts(state, case)


def work(case):
    if case["op"] == "norm":
        T, H, b = case["T"], case["H"], 2 if case["dtype"] == "bf16" else 4
        full = (2 if case["residual"] else 0) + 1 + (case["out"] != "mx8")
        return {"bytes": T * H * b * full + H * b + (case["out"] != "same") * T * H * 33 / 32,
                "flops": 5 * T * H}
    K, N = case["K"], case["N"]
    if case["op"] == "linear4":
        T, b = case["T"], 2 if case["dtype"] == "bf16" else 4
        return {"bytes": N * K * 17 / 32 + b * T * (K + N), "flops": 2 * T * N * K}
    T, R, E = case["T"], case["R"], case["E"]
    # experts that have a row, as many as these odds give
    used = R if case["skew"] < 0 else sum(1 - (1 - p) ** R for p in _odds(case))
    x_rows = T * (1 - (1 - 1 / T) ** R) if case["gather"] else R
    outs = N // 2 if case["swiglu"] else N
    return {"bytes": used * N * K * (case["bits"] / 8 + 1 / 32) + x_rows * K * 33 / 32
            + R * outs * (2 if case["out"] == "bf16" else 33 / 32) + 4 * (E + 1) + 4 * R * case["gather"],
            "flops": 2 * R * N * K}


def _exact_mx8(v):
    """(q, s) as the numbers they are, in 64 bits, by steps of each number's binade."""
    b = v.unflatten(-1, (-1, 32))
    top = b.abs().max(-1, keepdim=True)[0]
    e = torch.ceil(torch.log2(top.clamp(min=1e-300) / 448)).clamp(-127, 127)
    e = torch.where(top > 448 * torch.exp2(e), e + 1, e)
    e = torch.where(top <= 448 * torch.exp2(e - 1), e - 1, e).clamp(-127, 127)
    b = b / torch.exp2(e)
    binade = torch.floor(torch.log2(b.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(binade - 3)
    return (torch.round(b / step) * step).flatten(-2), torch.exp2(e).squeeze(-1)


def _exact_value(q, s):
    """What (q, s) stands for, in 64 bits."""
    if q.dtype == torch.uint8:
        code = torch.cat([(q & 15)[..., None], (q >> 4)[..., None]], -1).flatten(-2).long()
        mag, sign = code & 7, 1.0 - 2.0 * (code >> 3)
        # 2^(c/2 - 1) (1 + half of the last bit), and 0 and 1/2 below
        v = torch.where(mag < 2, 0.5 * mag, torch.exp2((mag // 2).double() - 1) * (1 + 0.5 * (mag % 2))) * sign
    else:
        v = q.double()
    power = torch.exp2(s.view(torch.uint8).double() - 127)
    return v * power.repeat_interleave(32, -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        z = s["x"].double()
        if case["residual"]:
            z += s["residual"].double()
        inv = torch.rsqrt(z.square().sum(1) / case["H"] + EPS)
        y = torch.einsum("th,t,h->th", z, inv, s["weight"].double())
        q, e = _exact_mx8(y) if case["out"] != "same" else (None, None)
        return {"y": None if case["out"] == "mx8" else y, "q": q, "s": e,
                "residual": z if case["residual"] else None}
    if case["op"] == "linear4":
        return {"y": torch.nn.functional.linear(s["x"].double(), _exact_value(*s["w"]))}
    x = _exact_value(*s["x"])
    if s["rows"] is not None:
        x = x[s["rows"].long()]
    offsets = s["offsets"].tolist()
    parts = []
    for e in range(case["E"]):
        w = _exact_value(s["w"][0][e], s["w"][1][e])
        y = torch.nn.functional.linear(x[offsets[e]:offsets[e + 1]], w)
        if case["swiglu"]:
            g, u = y.chunk(2, 1)
            y = torch.nn.functional.silu(g) * u
        parts.append(y)
    y = torch.cat(parts)
    if case["out"] == "bf16":
        return {"y": y}
    q, e = _exact_mx8(y)
    return {"q": q, "s": e}
