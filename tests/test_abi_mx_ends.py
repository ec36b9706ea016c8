"""Host checks of the entry points for rows and weights in 8 and 4 bits at the ends of their
sizes: no rows, workspaces of the smallest size. No GPU needed; every call is made in a
process of its own where it could end the process."""

import os
import subprocess
import sys

import pytest

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
