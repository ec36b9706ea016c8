"""Host checks of the entry points for rows and weights in 8 and 4 bits at the ends of their
sizes: no rows, workspaces of the smallest size. No GPU needed; every call is made in a
process of its own where it could end the process."""

import ctypes as C
import os
import subprocess
import sys

import pytest
import torch

import top_reduce_amd as tr
from top_reduce_amd import _binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("dtype", [B.BF16, B.F32])
@pytest.mark.parametrize("K,N", [(32, 1), (256, 16384), (4096, 16), (7168, 7168), (7168, 131072), (1 << 22, 1 << 22)])
def test_a_projection_of_no_rows(K, N, dtype):
    code = ("import ctypes as C, top_reduce_amd as tr\n"
            "from top_reduce_amd import _binding as B\n"
            f"lib, d = tr.load_library(), B.Linear4Desc(T=0, K={K}, N={N}, dtype={dtype}, reserved=0)\n"
            "assert lib.moe_linear_mx4_workspace(C.byref(d)) == 256\n"
            "assert lib.moe_linear_mx4(C.byref(d), None, None, None, None, None, 0, None) == 0\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stderr[-2000:])


def test_a_workspace_that_is_needed_is_not_taken_for_none():
    """Every size of few products: where the call wants a workspace the size says so."""
    lib = tr.load_library()
    fake = 1 << 40      # never dereferenced
    wanted = set()
    for K in (2816, 4096, 8192, 16384, 32768, 1 << 20):
        for T in (1, 2, 3, 4, 8, 16, 17, 33, 64):
            for N in (1, 2, 3, 4, 8, 16, 64, 100):
                d = B.Linear4Desc(T=T, K=K, N=N, dtype=B.F32, reserved=0)
                need = lib.moe_linear_mx4_workspace(C.byref(d))
                # no bytes: refused where some are needed; x is misaligned, so that the call ends on
                # the host either way
                status = lib.moe_linear_mx4(C.byref(d), fake + 8, fake, fake, 2 * fake, fake, 0, None)
                assert status == (-3 if need > 256 else -1), (K, T, N, need)
                if need > 256:
                    wanted.add(need)
                    assert lib.moe_linear_mx4(C.byref(d), fake + 8, fake, fake, 2 * fake, fake, need, None) == -1
    assert min(wanted) == 512 and tr.linear_mx4_workspace_size(1, 4096, 16, torch.float32) == 512
