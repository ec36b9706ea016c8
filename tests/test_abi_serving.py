"""C ABI checks of the router, the layer and the adapter projection that need
no GPU: struct layouts match the binding's mirror, and bad arguments are
refused on the host before anything is launched."""

import ctypes as C
import os
import subprocess

import torch

import top_reduce_amd as tr
from top_reduce_amd import _binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = C.c_void_p(1 << 40)       # never dereferenced: the checks fail first
FAR = C.c_void_p(1 << 44)
BIG = 1 << 40                    # workspace bytes claimed


def test_struct_layouts_match_the_binding(tmp_path):
    pairs = [("tr_route_desc", B.RouteDesc), ("tr_layer_desc", B.LayerDesc),
             ("tr_adapter_desc", B.AdapterDesc)]
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "topreduce.h"', "int main(void){"]
    want = []
    for name, cls in pairs:
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


def route(**kw):
    d = dict(T=4, H=64, G=16, K=2, dtype=B.BF16, idx_dtype=B.IDX_I64, score=0, renorm=1, scale=1.0)
    d.update(kw)
    return B.RouteDesc(**d)


BAD_ROUTE = [(dict(T=-1), -1), (dict(H=0), -1), (dict(H=12), -2), (dict(H=1 << 23), -2),
             (dict(G=0), -1), (dict(G=4097), -2), (dict(K=0), -1), (dict(K=17), -1),
             (dict(G=64, K=33), -1), (dict(dtype=2), -1), (dict(idx_dtype=5), -1),
             (dict(score=2), -1), (dict(renorm=2), -1), (dict(scale=float("inf")), -1),
             (dict(scale=float("nan")), -1), (dict(reserved=1), -1), (dict(T=1 << 31), -2)]


def test_route_refusals():
    lib = tr.load_library()
    for kw, status in BAD_ROUTE:
        d = route(**kw)
        assert lib.moe_route_topk_workspace(C.byref(d)) == 0, kw
        assert lib.moe_route_topk(C.byref(d), FAKE, FAKE, None, FAKE, FAKE, FAKE, BIG, None) == status, kw
        assert lib.moe_last_error()
    d = route()
    need = lib.moe_route_topk_workspace(C.byref(d))
    assert need > 0
    bad = C.c_void_p((1 << 40) + 4)
    ok = [FAKE, FAKE, None, FAKE, FAKE, FAKE, need]
    for at, v, status in ((0, None, -1), (0, bad, -1), (1, None, -1), (1, bad, -1),
                          (2, C.c_void_p((1 << 40) + 2), -1), (3, None, -1), (3, bad, -1),
                          (4, None, -1), (4, C.c_void_p((1 << 40) + 2), -1), (5, None, -1),
                          (5, bad, -1), (6, need - 1, -3)):
        args = list(ok)
        args[at] = v
        assert lib.moe_route_topk(C.byref(d), *args, None) == status, (at, v)
    assert lib.moe_route_topk(None, *ok, None) == -1
    # no rows: nothing is read, nothing launched
    d = route(T=0)
    assert lib.moe_route_topk_workspace(C.byref(d)) > 0
    assert lib.moe_route_topk(C.byref(d), None, None, None, None, None, FAKE, 256, None) == 0


def test_layer_refusals():
    lib = tr.load_library()

    def desc(r=None, **kw):
        d = dict(route=r or route(), I=32, expert_begin=0, E=4)
        d.update(kw)
        return B.LayerDesc(**d)

    def call(d, ws=BIG, **kw):
        a = dict(x=FAKE, gate=FAKE, bias=None, w1=FAKE, w2=FAKE, y=FAKE, idx=FAKE, w=FAKE)
        a.update(kw)
        return lib.moe_layer(C.byref(d), a["x"], a["gate"], a["bias"], a["w1"], a["w2"], a["y"],
                             a["idx"], a["w"], FAKE, ws, None)

    for kw, status in BAD_ROUTE:
        d = desc(route(**kw))
        assert lib.moe_layer_workspace(C.byref(d)) == 0 and call(d) == status, kw
    for kw, status in ((dict(E=0), -1), (dict(E=1025), -1), (dict(I=0), -1), (dict(expert_begin=13), -1),
                       (dict(expert_begin=-1), -1), (dict(reserved=3), -1), (dict(I=(1 << 22) + 1), -2),
                       (dict(I=1 << 24), -2)):
        d = desc(**kw)
        assert lib.moe_layer_workspace(C.byref(d)) == 0 and call(d) == status, kw
    for T in (4, 100):
        d = desc(route(T=T))
        need = lib.moe_layer_workspace(C.byref(d))
        assert need > 0 and call(d, ws=need - 1) == -3
        for name in ("x", "gate", "w1", "w2", "y", "idx", "w"):
            assert call(d, **{name: None}) == -1, name
            if name != "w":
                assert call(d, **{name: C.c_void_p((1 << 40) + 4)}) == -1, name
    assert call(desc(route(T=0)), x=None, gate=None, w1=None, w2=None, y=None, idx=None, w=None) == 0


def test_adapter_refusals():
    lib = tr.load_library()

    def desc(**kw):
        d = dict(T=4, H=64, N=48, R=8, A=3, dtype=B.BF16)
        d.update(kw)
        return B.AdapterDesc(**d)

    def call(d, ws=BIG, **kw):
        a = dict(x=FAKE, w=FAKE, a=FAKE, b=FAKE, ids=FAKE, scales=None, y=FAR)
        a.update(kw)
        return lib.moe_adapter_linear(C.byref(d), a["x"], a["w"], a["a"], a["b"], a["ids"],
                                      a["scales"], a["y"], FAKE, ws, None)

    for kw, status in ((dict(T=-1), -1), (dict(T=1 << 31), -2), (dict(H=0), -1), (dict(H=20), -2),
                       (dict(H=(1 << 22) + 8), -2), (dict(N=0), -1), (dict(N=(1 << 22) + 1), -2),
                       (dict(R=0), -1), (dict(R=257), -2), (dict(A=0), -1), (dict(A=(1 << 20) + 1), -2),
                       (dict(dtype=3), -1), (dict(reserved=1), -1),
                       (dict(T=(1 << 31) - 1, N=1 << 22), -2)):
        d = desc(**kw)
        assert lib.moe_adapter_linear_workspace(C.byref(d)) == 0 and call(d) == status, kw
    for T in (4, 100):
        d = desc(T=T)
        need = lib.moe_adapter_linear_workspace(C.byref(d))
        assert need > 0 and call(d, ws=need - 1) == -3
        for name in ("x", "w", "a", "b", "ids", "y"):
            assert call(d, **{name: None}) == -1, name
            assert call(d, **{name: C.c_void_p((1 << 40) + 2)}) == -1, name
        assert call(d, scales=C.c_void_p((1 << 40) + 2)) == -1
        assert call(d, y=FAKE) == -1                                    # y over x
        assert call(d, y=C.c_void_p((1 << 40) + T * 128 - 16)) == -1    # its start over x's end
        assert b"overlap" in lib.moe_last_error()
    assert call(desc(T=0), x=None, w=None, a=None, b=None, ids=None, y=None) == 0


def test_workspace_sizes_grow_with_the_work():
    assert tr.route_workspace_size(1, 3584, 896, 16) >= 896 * 4
    assert tr.route_workspace_size(16384, 7168, 256, 8) >= 16384 * 256 * 4
    assert tr.adapter_workspace_size(8, 3584, 3584, 16, 8) >= 8 * 3584 * 4
    assert tr.adapter_workspace_size(100, 512, 512, 16, 8, dtype=torch.float32) >= 100 * 16 * 4
    few = tr.layer_workspace_size(64, 7168, 2048, 32, 256, 8)
    assert few >= 64 * 8 * 2048 * 4 and few < tr.layer_workspace_size(65, 7168, 2048, 32, 256, 8)
