"""Rows and weights in 8 and 4 bits: norm, experts' products, projections.

Numbers in blocks of 32 along the last dimension are a pair (q, s) of contiguous
tensors: q float8_e4m3fn [..., K], or uint8 [..., K/2] for 4 bits (e2m1, the number at
an even k in the low half of its byte), and s float8_e8m0fnu [..., K/32], one power of
two for each block. As in _binding.py: checks and marshalling only; tensors that a
caller gives must be ready on `stream`, and what a call allocates belongs to it.
"""

from __future__ import annotations

import ctypes as C
import functools
from typing import NamedTuple, Optional, Tuple, Union

import torch

from . import _binding as B
from ._binding import (_arg, _check, _dev_tensor, _dtype_code, _elsewhere, _need, _raw_stream, _run_on,
                       _ws_arg, _x_arg)

E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
BLOCK = 32
NO_WS = 256     # the size of a workspace that is not needed
KERNELS = {"auto": 0, "rows": 1, "tile32": 2, "tile64": 3, "tile256": 4}

Mx = Tuple[torch.Tensor, torch.Tensor]


class Normed(NamedTuple):
    """What rms_norm returns; None for what was not asked for."""
    y: Optional[torch.Tensor]
    q: Optional[torch.Tensor]
    s: Optional[torch.Tensor]
    residual: Optional[torch.Tensor]


def _launch(dev, call, *args) -> None:
    """call(*args, stream) with the tensors' device as the current one."""
    lib = B.load_library()
    if torch._C._cuda_getDevice() == dev.index:
        status = getattr(lib, call)(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            status = getattr(lib, call)(*args, _raw_stream(dev))
    if status:
        _check(status)


def _out(t: Optional[torch.Tensor], name: str, dtype, shape, dev) -> Tuple[torch.Tensor, int]:
    """An output that the caller gives, checked, or a new one; and its address."""
    if t is None:
        t = torch.empty(*shape, dtype=dtype, device=dev)
        return t, t.data_ptr()
    return t, _arg(t, name, dtype, shape, dev)


def _pair(t, name: str) -> Mx:
    if not isinstance(t, (tuple, list)) or len(t) != 2 or not all(isinstance(v, torch.Tensor) for v in t):
        raise TypeError(f"{name} must be a pair (q, s) of tensors")
    return t[0], t[1]


def _bits(q: torch.Tensor, name: str) -> int:
    if q.dtype == E4M3:
        return 8
    if q.dtype == torch.uint8:
        return 4
    raise TypeError(f"{name} must be float8_e4m3fn (8 bits) or uint8 (4 bits) (got {q.dtype})")


def quantize_mx(x: torch.Tensor, bits: int = 8, q: Optional[torch.Tensor] = None,
                s: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> Mx:
    """moe_quantize_mx: (q, s) of x [..., K] (bfloat16 or float32, K a multiple of 32) in
    8 or 4 bits. A block's scale is the smallest power of two that brings its largest
    magnitude to 448 (4 bits: 6) or below; elements are rounded to nearest, ties to even."""
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise ValueError("x must be a [..., K] tensor")
    if bits not in (8, 4):
        raise ValueError(f"bits must be 8 or 4 (got {bits!r})")
    if not x.is_cuda or not x.is_contiguous():
        _dev_tensor(x, "x")
    dev = x.device
    if _elsewhere(stream, dev):
        return _run_on(stream, (q, s), quantize_mx, x, bits, q, s)
    code = _dtype_code(x.dtype)
    *lead, K = x.shape
    if K % BLOCK:
        raise ValueError(f"rows of {K} have no whole blocks of {BLOCK}")
    qt, qs = (E4M3, (*lead, K)) if bits == 8 else (torch.uint8, (*lead, K // 2))
    q, qp = _out(q, "q", qt, qs, dev)
    s, sp = _out(s, "s", E8M0, (*lead, K // BLOCK), dev)
    rows = x.numel() // K if K else 0
    if rows:
        _launch(dev, "moe_quantize_mx", rows, K, code, bits, x.data_ptr(), qp, sp)
    return q, s


@functools.lru_cache(maxsize=512)
def _norm_desc(T, H, dtype, eps):
    return C.byref(B.NormDesc(T=T, H=H, dtype=_dtype_code(dtype), eps=eps))


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
             residual: Optional[torch.Tensor] = None, out: str = "same",
             y: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
             s: Optional[torch.Tensor] = None, residual_out: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None) -> Normed:
    """moe_rms_norm: y = z / sqrt(mean(z^2) + eps) * weight over the rows of
    z = x + residual. x [T, H], residual [T, H] or None, weight [H].

    out: "same" for y in x's type, "mx8" for (q, s) in 8 bits, "both". The field
    `residual` is z in x's type (None without a residual); residual_out may be the
    residual itself, and y may be x. y, (q, s) and the next residual are each rounded
    once from fp32."""
    dev = _x_arg(x)
    if _elsewhere(stream, dev):
        return Normed(*_run_on(stream, (y, q, s, residual_out), rms_norm, x, weight, eps, residual, out,
                               y, q, s, residual_out))
    if out not in ("same", "mx8", "both"):
        raise ValueError(f"out must be 'same', 'mx8' or 'both' (got {out!r})")
    T, H = x.shape
    dt = x.dtype
    desc = _norm_desc(T, H, dt, eps)
    wp = _arg(weight, "weight", dt, (H,), dev)
    yp = qp = sp = rp = op = None
    if out != "mx8":
        y, yp = _out(y, "y", dt, (T, H), dev)
    elif y is not None:
        raise ValueError("y is given, and out is 'mx8'")
    if out != "same":
        if H % BLOCK:
            raise ValueError(f"rows of {H} have no whole blocks of {BLOCK}")
        q, qp = _out(q, "q", E4M3, (T, H), dev)
        s, sp = _out(s, "s", E8M0, (T, H // BLOCK), dev)
    elif q is not None or s is not None:
        raise ValueError("q or s is given, and out is 'same'")
    if residual is not None:
        rp = _arg(residual, "residual", dt, (T, H), dev)
        residual_out, op = _out(residual_out, "residual_out", dt, (T, H), dev)
    elif residual_out is not None:
        raise ValueError("residual_out is given without a residual")
    if T:
        _launch(dev, "moe_rms_norm", desc, x.data_ptr(), rp, wp, yp, op, qp, sp)
    return Normed(y, q, s, residual_out)


@functools.lru_cache(maxsize=512)
def _expert_desc(T, R, K, N, E, bits, swiglu, out, kernel):
    if kernel not in KERNELS:
        raise ValueError(f"kernel must be one of {', '.join(KERNELS)} (got {kernel!r})")
    return C.byref(B.ExpertDesc(T=T, R=R, K=K, N=N, E=E, bits=bits, swiglu=swiglu, out=out,
                                kernel=KERNELS[kernel], reserved=0))


def expert_linear(x: Mx, w: Mx, offsets: torch.Tensor, rows: Optional[torch.Tensor] = None,
                  swiglu: bool = False, out: str = "bf16", y: Optional[torch.Tensor] = None,
                  ys: Optional[torch.Tensor] = None, kernel: str = "auto",
                  stream: Optional[torch.cuda.Stream] = None) -> Union[torch.Tensor, Mx]:
    """moe_expert_linear: y[r] = w[e] x[rows[r]] for the rows r of each expert's segment,
    offsets[e] <= r < offsets[e + 1].

    x: (q, s) in 8 bits, q [T, K]; w: (q, s) in 8 or 4 bits, q [E, N, K] or [E, N, K/2];
    offsets: int32 [E + 1] on the GPU, ascending (the plan's); rows: int32 [R] (the plan's
    row_src), or None where row r of the result is row r of x. swiglu: rows [0, N/2) of an
    expert's weights are gate, the others up, and the result is silu(gate) * up [R, N/2].
    out: "bf16", or "mx8" for a pair (q, s). Rows outside every segment are left as they
    are in y and ys (undefined where the call allocates them)."""
    xq, xs = _pair(x, "x")
    wq, ws = _pair(w, "w")
    dev = _x_arg(xq)
    if _elsewhere(stream, dev):
        return _run_on(stream, (y, ys), expert_linear, x, w, offsets, rows, swiglu, out, y, ys,
                       kernel)
    if out not in ("bf16", "mx8"):
        raise ValueError(f"out must be 'bf16' or 'mx8' (got {out!r})")
    if wq.dim() != 3:
        raise ValueError("w must hold an [E, N, K] tensor")
    bits = _bits(wq, "w")
    T, K = xq.shape
    E, N = wq.shape[:2]
    if K % BLOCK:
        raise ValueError(f"rows of {K} have no whole blocks of {BLOCK}")
    xp = _arg(xq, "x", E4M3, (T, K), dev)
    xsp = _arg(xs, "x's scales", E8M0, (T, K // BLOCK), dev)
    wp = _arg(wq, "w", wq.dtype, (E, N, K * bits // 8), dev)
    wsp = _arg(ws, "w's scales", E8M0, (E, N, K // BLOCK), dev)
    op = _arg(offsets, "offsets", torch.int32, (E + 1,), dev)
    R, rp = T, None
    if rows is not None:
        R = rows.shape[0] if isinstance(rows, torch.Tensor) and rows.dim() == 1 else -1
        rp = _arg(rows, "rows", torch.int32, (R,), dev)
    desc = _expert_desc(T, R, K, N, E, bits, 1 if swiglu else 0, 1 if out == "mx8" else 0, kernel)
    outs = N // 2 if swiglu else N
    ysp = None
    if out == "bf16":
        if ys is not None:
            raise ValueError("ys is given, and out is 'bf16'")
        y, yp = _out(y, "y", torch.bfloat16, (R, outs), dev)
    else:
        if outs % BLOCK:
            raise ValueError(f"rows of {outs} outputs have no whole blocks of {BLOCK}")
        y, yp = _out(y, "y", E4M3, (R, outs), dev)
        ys, ysp = _out(ys, "ys", E8M0, (R, outs // BLOCK), dev)
    _launch(dev, "moe_expert_linear", desc, xp, xsp, wp, wsp, op, rp, yp, ysp)
    return y if out == "bf16" else (y, ys)


@functools.lru_cache(maxsize=512)
def _linear4_plan(T, K, N, dtype):
    d = B.Linear4Desc(T=T, K=K, N=N, dtype=_dtype_code(dtype), reserved=0)
    return C.byref(d), _need(B.load_library().moe_linear_mx4_workspace, d)


def linear_mx4_workspace_size(T: int, K: int, N: int, dtype=torch.bfloat16) -> int:
    """Bytes of ws for linear_mx4 of these sizes."""
    return _linear4_plan(T, K, N, dtype)[1]


def linear_mx4(x: torch.Tensor, w: Mx, y: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """moe_linear_mx4: y [T, N] = x w^T for a few rows x [T, K] (bfloat16 or float32) and
    weights in 4 bits, w = (q [N, K/2] uint8, s [N, K/32])."""
    dev = _x_arg(x)
    wq, wscale = _pair(w, "w")
    if _elsewhere(stream, dev):
        return _run_on(stream, (y,), linear_mx4, x, w, y, ws)
    if wq.dim() != 2:
        raise ValueError("w must hold an [N, K/2] tensor")
    T, K = x.shape
    N, dt = wq.shape[0], x.dtype
    if K % BLOCK:
        raise ValueError(f"rows of {K} have no whole blocks of {BLOCK}")
    desc, need = _linear4_plan(T, K, N, dt)
    wp = _arg(wq, "w", torch.uint8, (N, K // 2), dev)
    sp = _arg(wscale, "w's scales", E8M0, (N, K // BLOCK), dev)
    y, yp = _out(y, "y", dt, (T, N), dev)
    if not T:
        return y
    if ws is None and need == NO_WS:
        _launch(dev, "moe_linear_mx4", desc, x.data_ptr(), wp, sp, yp, None, 0)
    else:
        ws = _ws_arg(ws, need, dev)
        _launch(dev, "moe_linear_mx4", desc, x.data_ptr(), wp, sp, yp, ws.data_ptr(), ws.numel())
    return y


def forward_mx(p: B.MoePlan, x: Mx, topk_weights: Optional[torch.Tensor], w1: Mx, w2: Mx,
               y: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """moe_forward_mx: y [T, H] bfloat16, as forward, with rows x in 8 bits and weights w1
    [E, 2I, H] (gate | up) and w2 [E, H, I] in 8 bits or both in 4. The plan is one of
    bfloat16."""
    d = p.desc
    dev = p.ws.device
    if _elsewhere(stream, dev):
        return _run_on(stream, (y,), forward_mx, p, x, topk_weights, w1, w2, y)
    xq, xs = _pair(x, "x")
    (q1, s1), (q2, s2) = _pair(w1, "w1"), _pair(w2, "w2")
    bits = _bits(q1, "w1")
    if d.H % BLOCK or d.I % BLOCK:
        raise ValueError(f"H and I must be multiples of {BLOCK} (got {d.H} and {d.I})")
    xp = _arg(xq, "x", E4M3, (d.T, d.H), dev)
    xsp = _arg(xs, "x's scales", E8M0, (d.T, d.H // BLOCK), dev)
    w1p = _arg(q1, "w1", q1.dtype, (d.E, 2 * d.I, d.H * bits // 8), dev)
    s1p = _arg(s1, "w1's scales", E8M0, (d.E, 2 * d.I, d.H // BLOCK), dev)
    w2p = _arg(q2, "w2", q1.dtype, (d.E, d.H, d.I * bits // 8), dev)
    s2p = _arg(s2, "w2's scales", E8M0, (d.E, d.H, d.I // BLOCK), dev)
    wp = None if topk_weights is None else _arg(topk_weights, "topk_weights", torch.float32,
                                                (d.T, d.K), dev)
    y, yp = _out(y, "y", torch.bfloat16, (d.T, d.H), dev)
    _launch(dev, "moe_forward_mx", C.byref(p.struct), xp, xsp, wp, bits, w1p, s1p, w2p, s2p, yp)
    return y
