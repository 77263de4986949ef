"""Calls on empty plans of the operators around experts, whose pointers are all given: sizes of
zero are allowed everywhere, and what the host works out from them must end in a status code.
Without a GPU every launch is refused by the runtime, so a call that gets that far returns the
code of a HIP error; in a process of its own, that a signal would end."""

import os
import signal
import subprocess
import sys

import pytest

import software_pipelined_tiled_gemm_amd as spg

CHILD = """
import ctypes, itertools, sys
import software_pipelined_tiled_gemm_amd as spg
L = spg.lib()
h = ctypes.c_void_p()
p, big = 4096, 1 << 40
which = sys.argv[1]

def plan(create, *a):
    assert getattr(L, create)(ctypes.byref(h), *a) == 0, (create, a)
    print(create, a, flush=True)
    return h

if which == "grouped":
    for rows, N, K, tokens, layout in itertools.product((0, 1), (0, 1, 64), (0, 1, 64), (-1, 0, 16), (0, 1)):
        # with no rows a source may be given or not, whatever the plan has
        for src in {p if tokens >= 0 else 0, p if rows == 0 else 0 if tokens < 0 else p}:
            plan("gemm_grouped_create", rows, N, K, 4, tokens, 1, layout)
            print(L.gemm_grouped_run(h, p, p, p, src, p, p, big, 0), flush=True)
            for dx, dw in ((p, p), (p, 0), (0, p), (0, 0)):
                print(L.gemm_grouped_backward(h, p, p, p, p, src, dx, dw, p, big, 0), flush=True)
            L.gemm_grouped_destroy(h)
            plan("gemm_experts_create", rows, N, K, 4, tokens, 1, layout, 1)
            print(L.gemm_experts_run(h, p, p, p, p, src, p, p, p, p, big, 0), flush=True)
            print(L.gemm_experts_backward(h, p, p, p, p, p, p, p, src, p, p, p, p, big, 0), flush=True)
            L.gemm_experts_destroy(h)
elif which == "norm":
    for rows, K in itertools.product((0, 1, 5000), (0, 1, 64, 20000)):
        plan("gemm_norm_create", rows, K, 1, 2, 1e-5)
        print(L.gemm_norm_run(h, p, p, p, p, p, p, 0), flush=True)
        for dw, db in ((p, p), (0, p), (0, 0)):
            print(L.gemm_norm_backward(h, p, p, p, p, p, p, dw, db, p, big, 0), flush=True)
        L.gemm_norm_destroy(h)
elif which == "route":
    for tokens, E, k in ((0, 1, 1), (0, 64, 8), (1, 1, 1), (5000, 64, 8)):
        plan("gemm_route_create", tokens, E, k, 2, 0)
        print(L.gemm_route_run(h, p, p, p, p, p, p, p, big, 0), flush=True)
        print(L.gemm_route_backward(h, p, p, p, p, 0), flush=True)
        L.gemm_route_destroy(h)
else:
    for tokens, rows, N in itertools.product((0, 1), (0, 2), (0, 1, 64)):
        plan("gemm_combine_create", tokens, 2, rows, N, 1)
        print(L.gemm_combine_run(h, p, p, p, p, 0), flush=True)
        for dgate in (p, 0):
            print(L.gemm_combine_backward(h, p, p, p, p, p, dgate, 0), flush=True)
        L.gemm_combine_destroy(h)
print("through")
"""


@pytest.mark.parametrize("which", ["grouped", "norm", "route", "combine"])
def test_empty_plans(which):
    if not os.path.exists(spg.LIB_PATH):
        pytest.fail("libspgemm.so is not built; run __graft_entry__.build()")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    # the pointers are made up: no device may be seen
    env = dict(os.environ, HIP_VISIBLE_DEVICES="-1", ROCR_VISIBLE_DEVICES="", CUDA_VISIBLE_DEVICES="-1", PYTHONPATH=root)
    r = subprocess.run([sys.executable, "-c", CHILD, which], cwd=root, env=env, capture_output=True, text=True, timeout=300)
    end = signal.Signals(-r.returncode).name if r.returncode < 0 else r.returncode
    assert r.returncode == 0 and r.stdout.endswith("through\n"), (end, r.stdout.splitlines()[-2:], r.stderr[-500:])
