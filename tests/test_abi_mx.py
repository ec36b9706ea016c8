"""Checks of the entry points for rows and weights in 8 and 4 bits that need no GPU:
struct layouts, and refusals on the host before anything is launched."""

import ctypes as C
import os
import subprocess

import pytest
import torch

import top_reduce_amd as tr
from tests import _mx as M
from top_reduce_amd import _binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 40      # never dereferenced: the checks fail first
FAR = 1 << 44


def test_struct_layouts_match_the_binding(tmp_path):
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "topreduce.h"', "int main(void){"]
    want = []
    for name, cls in (("tr_norm_desc", B.NormDesc), ("tr_expert_desc", B.ExpertDesc),
                      ("tr_linear4_desc", B.Linear4Desc)):
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        want.append(C.sizeof(cls))
        for f, _ in cls._fields_:
            lines.append(f'printf("%zu\\n", offsetof({name}, {f}));')
            want.append(getattr(cls, f).offset)
    lines.append("return 0;}")
    prog = tmp_path / "layout.c"
    prog.write_text("\n".join(lines))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I",
                    "/opt/rocm/include", str(prog), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    assert [int(v) for v in out.split()] == want


def test_quantize_refusals():
    lib = tr.load_library()
    ok = dict(rows=4, K=64, dtype=B.BF16, bits=8, x=FAKE, q=FAR, s=FAR + 4096)
    for kw, status in ((dict(rows=-1), -1), (dict(K=0), -1), (dict(K=48), -2), (dict(K=(1 << 22) + 32), -2),
                       (dict(dtype=2), -1), (dict(bits=6), -1), (dict(rows=1 << 35), -2), (dict(x=None), -1),
                       (dict(x=FAKE + 8), -1), (dict(q=None), -1), (dict(q=FAR + 4), -1), (dict(s=None), -1),
                       (dict(q=FAKE + 496), -1), (dict(s=FAKE + 511), -1), (dict(s=FAR + 255), -1)):
        a = {**ok, **kw}
        assert lib.moe_quantize_mx(*a.values(), None) == status, kw
        assert lib.moe_last_error()
    assert lib.moe_quantize_mx(0, 64, B.BF16, 4, None, None, None, None) == 0


def test_norm_refusals():
    lib = tr.load_library()
    d0 = dict(T=4, H=64, dtype=B.BF16, eps=1e-6)
    a0 = dict(x=FAKE, residual=FAKE + (1 << 20), weight=FAKE + (2 << 20), y=FAR, residual_out=FAR + (1 << 20),
              q=FAR + (2 << 20), s=FAR + (3 << 20))

    def call(d, a):
        return lib.moe_rms_norm(C.byref(B.NormDesc(**{**d0, **d})), *{**a0, **a}.values(), None)

    for d, status in ((dict(T=-1), -1), (dict(T=1 << 31), -2), (dict(H=0), -1), (dict(H=12), -2),
                      (dict(H=40), -2), (dict(H=(1 << 22) + 32), -2), (dict(dtype=3), -1),
                      (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1)):
        assert call(d, {}) == status, d
    for a in (dict(x=None), dict(weight=None), dict(y=None, q=None, s=None), dict(q=None), dict(s=None),
              dict(x=FAKE + 8), dict(residual=FAKE + 8), dict(weight=FAKE + 2), dict(y=FAR + 4), dict(q=FAR + 8),
              dict(residual_out=FAR + 2), dict(y=FAKE + 16), dict(residual_out=FAKE + 496),
              dict(q=FAKE), dict(s=FAKE + (1 << 20) + 511), dict(residual_out=FAR + 256), dict(q=FAR + 496),
              dict(s=FAR), dict(s=FAR + (1 << 20) + 511), dict(s=FAR + (2 << 20) + 255),
              dict(y=FAKE + (2 << 20) + 112), dict(s=FAKE + (2 << 20))):
        assert call({}, a) == -1, a
        assert lib.moe_last_error()
    assert lib.moe_rms_norm(None, *a0.values(), None) == -1
    assert call(dict(T=0), {k: None for k in a0}) == 0


def test_expert_refusals():
    lib = tr.load_library()
    d0 = dict(T=8, R=8, K=64, N=128, E=4, bits=8, swiglu=1, out=1)
    a0 = dict(x=FAKE, xs=FAKE + (1 << 20), w=FAKE + (2 << 20), ws=FAKE + (3 << 20), offsets=FAKE + (4 << 20),
              rows=FAKE + (5 << 20), y=FAR, ys=FAR + (1 << 20))

    def call(d, a):
        return lib.moe_expert_linear(C.byref(B.ExpertDesc(**{**d0, **d})), *{**a0, **a}.values(), None)

    for d, status in ((dict(T=-1), -1), (dict(R=-1), -1), (dict(T=1 << 31), -2), (dict(R=1 << 31), -2),
                      (dict(T=0), -1), (dict(K=0), -1), (dict(K=40), -2), (dict(K=(1 << 22) + 32), -2),
                      (dict(N=0), -1), (dict(N=127), -1), (dict(N=96), -2), (dict(N=100, swiglu=0), -2),
                      (dict(N=1 << 26), -2), (dict(E=0), -1), (dict(E=1025), -1), (dict(bits=6), -1),
                      (dict(swiglu=2), -1), (dict(out=2), -1), (dict(kernel=5), -1), (dict(kernel=-1), -1),
                      (dict(reserved=1), -1), (dict(kernel=2), -2), (dict(kernel=4), -2)):
        assert call(d, {}) == status, d
        assert lib.moe_last_error()
    for a in (dict(x=None), dict(xs=None), dict(w=None), dict(ws=None), dict(offsets=None), dict(y=None),
              dict(ys=None), dict(x=FAKE + 8), dict(w=FAKE + 4), dict(y=FAR + 8), dict(offsets=FAKE + 2),
              dict(rows=FAKE + 1), dict(y=FAKE + 496), dict(ys=FAKE + 511), dict(y=FAKE + (1 << 20)),
              dict(ys=FAR + 511)):
        assert call({}, a) == -1, a
    assert call(dict(out=0), {}) == -1              # scales given, and none asked for
    assert call(dict(T=7), dict(rows=None)) == -1   # a row of x for each of the result's
    # a block for each tile: too many for a launch
    most = dict(T=1, R=1 << 22, K=256, N=1 << 16, out=0, swiglu=0)
    for kernel in (2, 3):
        assert call(dict(most, kernel=kernel), dict(y=FAR * 2, ys=None)) == -2
    assert lib.moe_expert_linear(None, *a0.values(), None) == -1
    assert call(dict(R=0, T=0), {k: None for k in a0}) == 0


def test_linear4_refusals():
    lib = tr.load_library()
    d0 = dict(T=4, K=64, N=48, dtype=B.BF16, reserved=0)
    a0 = dict(x=FAKE, w=FAKE + (1 << 20), wscale=FAKE + (2 << 20), y=FAR, ws=FAKE + (4 << 20), n=1 << 40)

    def call(d, a):
        return lib.moe_linear_mx4(C.byref(B.Linear4Desc(**{**d0, **d})), *{**a0, **a}.values(), None)

    for d, status in ((dict(T=-1), -1), (dict(T=1 << 31), -2), (dict(K=0), -1), (dict(K=16), -2),
                      (dict(K=(1 << 22) + 32), -2), (dict(N=0), -1), (dict(N=(1 << 22) + 1), -2),
                      (dict(T=1 << 30, N=1 << 11), -2), (dict(dtype=2), -1), (dict(reserved=1), -1)):
        assert call(d, {}) == status, d
        assert lib.moe_last_error()
        assert lib.moe_linear_mx4_workspace(C.byref(B.Linear4Desc(**{**d0, **d}))) == 0
    for a in (dict(x=None), dict(w=None), dict(wscale=None), dict(y=None), dict(x=FAKE + 8), dict(w=FAKE + 4),
              dict(y=FAR + 2), dict(y=FAKE + 496)):
        assert call({}, a) == -1, a
    assert lib.moe_linear_mx4(None, *a0.values(), None) == -1
    assert call(dict(T=0), {k: v if k == "n" else None for k, v in a0.items()}) == 0
    # some rows, few tiles: a workspace for the parts' sums
    big = dict(T=40, K=4096, N=256)
    need = lib.moe_linear_mx4_workspace(C.byref(B.Linear4Desc(**{**d0, **big})))
    assert need >= 2 * 40 * 256 * 4 and need == tr.linear_mx4_workspace_size(40, 4096, 256)
    for a, status in ((dict(ws=None), -1), (dict(ws=FAKE + 128), -1), (dict(n=need - 1), -3)):
        assert call(big, a) == status, a
    assert tr.linear_mx4_workspace_size(4, 64, 48) == 256


def test_forward_refusals():
    lib = tr.load_library()

    def call(bits=8, **kw):
        p = B.PlanStruct()
        p.d = B.make_desc(**{**dict(T=4, K=2, E=4, H=64, I=32), **kw})
        p.ws = FAKE
        p.R_cap = p.d.T * p.d.K
        a = [FAKE] * 2 + [None, bits] + [FAKE] * 4 + [FAR]
        return lib.moe_forward_mx(C.byref(p), *a, None)

    for kw in (dict(dtype=torch.float32), dict(H=40), dict(I=40)):
        assert call(**kw) == -2, kw
    assert call(bits=5) == -1
    assert lib.moe_forward_mx(None, *[None] * 3, 8, *[None] * 6) == -1


def cpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=torch.float32).to(dtype)


def test_the_binding_refuses_what_is_not_on_the_gpu():
    x, w = cpu(4, 64), cpu(64)
    for call in (lambda: tr.rms_norm(x, w), lambda: tr.quantize_mx(x),
                 lambda: tr.linear_mx4(x, M.quantize(cpu(8, 64), 4)),
                 lambda: tr.expert_linear(M.quantize(x), M.quantize(cpu(2, 8, 64)), torch.zeros(3, dtype=torch.int32))):
        with pytest.raises(ValueError, match="must be on the GPU"):
            call()
    with pytest.raises(TypeError):
        tr.expert_linear(x, M.quantize(cpu(2, 8, 64)), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        tr.quantize_mx(x, bits=6)


def test_plain_blocks():
    """The oracle's own quantization, by hand."""
    v = torch.zeros(3, 32, dtype=torch.float64)
    v[0, :4] = torch.tensor([448.0, -17.0, 0.3, 2.0 ** -9])
    v[1, :4] = torch.tensor([449.0, 1.0, -1.5, 0.0])
    q, s = M.quantize(v, 8)
    assert s.view(torch.uint8).flatten().tolist() == [127, 128, 0]
    assert M.value(q, s)[0, :4].tolist() == [448.0, -16.0, 0.3125, 2.0 ** -9]
    assert M.value(q, s)[1, :3].tolist() == [448.0, 1.0, -1.5]     # 224.5 is 224 in steps of 16
    v[0, :8] = torch.tensor([6.0, 5.0, 2.5, 1.75, -0.25, 0.75, 3.5, -1.25])
    q, s = M.quantize(v[:1], 4)
    assert s.view(torch.uint8).flatten().tolist() == [127]
    assert M.value(q, s)[0, :8].tolist() == [6.0, 4.0, 2.0, 2.0, -0.0, 1.0, 4.0, -1.0]
