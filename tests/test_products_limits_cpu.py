"""Sizes at the ends of what lq_gemm_ep, lq_gemm_grouped, lq_gemm_join and lq_route take: answered or
refused on the host (no GPU needed).  Each runs in a process of its own, so that one that ends the
process fails its test and not the session."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F32, F16, BF16 = 0, 1, 2
OK, SHAPE = 0, 2


def status(name, *sizes):
    """What the size query returns, and the bytes."""
    code = ("import ctypes\nfrom bit_lifted_gemv_amd import lq\nn = ctypes.c_size_t(0)\n"
            f"print(lq.load_library().{name}(*{sizes!r}, ctypes.byref(n)), n.value)")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])
    return tuple(int(x) for x in r.stdout.split()[-2:])


@pytest.mark.parametrize("name,sizes", [
    ("lq_gemm_grouped_workspace_size", (4, 1, 128, 100, 100, BF16)),
    ("lq_gemm_ep_workspace_size", (1, 65536, 25000, BF16)),
    ("lq_gemm_ep_workspace_size", (1, 65536, 15000, F32)),
    ("lq_gemm_ep_workspace_size", (3, 65536, 20000, F16)),
    ("lq_gemm_join_workspace_size", (4, 1, 128, 100, 50, 2, F16)),
])
def test_one_row_of_weights(name, sizes):
    st, need = status(name, *sizes)
    assert st == OK and need > 0


@pytest.mark.parametrize("T,k", [(1 << 62, 4), (1 << 59, 32), ((1 << 63) - 1, 2), (1 << 31, 1), (1 << 30, 2)])
def test_too_many_choices_are_refused(T, k):
    """T * k < 2^31, also where the product of the two wraps round to a small number."""
    assert status("lq_route_workspace_size", T, 64, k)[0] == SHAPE
    assert status("lq_gemm_join_workspace_size", 4, 64, 128, 10, T, k, BF16)[0] == SHAPE
