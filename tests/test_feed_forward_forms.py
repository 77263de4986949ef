"""The sizes of tests/feed_forward_forms.py reach every kernel that the feed-forward operators'
choice of tiles launches anywhere in a sweep of sizes.  csrc/product.hip's host side is compiled
for the CPU with its launches replaced by a record of them, so it is the code's own choice."""

import ctypes
import os
import shutil
import subprocess

import pytest

from tests import feed_forward_forms as listed

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

DRIVER = r"""
#include <hip/hip_runtime.h>
#undef hipLaunchKernelGGL
#define hipLaunchKernelGGL(...) ((void)0)
#define hipGetLastError() hipSuccess
#include "product.hip"

struct Record { int product, reg, tile, tail, split, merged, kt; };
static Record g_rec[16];
static int g_n;

namespace spg {
gemm_status hip_fail(hipError_t) { return GEMM_ERR_HIP; }
static void note(int p, int et, bool reg, int tile, const ProductArgs& a, int merged) {
    // the kernels that launch_tile (product_launch.hpp) compiles with and without tails
    const bool tail = p != kGradW && p != kGradXNK && kTileM[tile] == 256 && !reg && a.K * (et == kElI8 ? 1 : 2) % 16 != 0;
    g_rec[g_n++] = Record{p, reg, tile, tail, a.split > 1, merged, a.kt_part};
}
template <int ET, int P, bool REG>
void launch_product(int tile, const ProductArgs& a, dim3, hipStream_t) { note(P, ET, REG, tile, a, 0); }
template <int ET, int P, bool REG>
void launch_gradients(int tile, const ProductArgs& x, const ProductArgs& w, int, dim3, hipStream_t) {
    note(P, ET, REG, tile, x, 1);
    note(kGradW, ET, REG, tile, w, 1);
}
}  // namespace spg

// what: 0 gated, 1 its backward pass, 2 int8; flag: weights [N,K], or gated; out: Records
extern "C" int launches(int what, int64_t M, int64_t N, int64_t K, int flag, int off, int* out) {
    char* p = (char*)(((uintptr_t)1 << 40) + off);
    char* w = (char*)((uintptr_t)1 << 41);
    gemm_status e;
    g_n = 0;
    if (what == 2) {
        gemm_quantized_handle h;
        if (gemm_quantized_create(&h, M, N, K, GEMM_F32, flag ? GEMM_ACT_SILU : GEMM_ACT_NONE)) return -1;
        e = gemm_quantized_run(h, (int8_t*)p, (float*)w, (int8_t*)p, (float*)w, flag ? (int8_t*)p : nullptr,
                               flag ? (float*)w : nullptr, p, w, INT64_MAX, 0);
        gemm_quantized_destroy(h);
    } else {
        gemm_gated_handle h;
        if (gemm_gated_create(&h, M, N, K, GEMM_BF16, flag ? GEMM_B_NK : GEMM_B_KN, GEMM_ACT_SILU)) return -1;
        e = what == 0 ? gemm_gated_run(h, p, p, p, p, p, p, w, INT64_MAX, 0)
                      : gemm_gated_backward(h, p, p, p, p, p, p, p, p, p, w, INT64_MAX, 0);
        gemm_gated_destroy(h);
    }
    if (e != GEMM_OK) return -1;
    for (int i = 0; i < g_n; ++i) ((Record*)out)[i] = g_rec[i];
    return g_n;
}
"""

# rows, and columns and reductions, on both sides of what separates the tiles, with every
# alignment of a row: whole lines, 16 bytes, words, odd
ROWS = [1, 16, 17, 33, 64, 65, 100, 128, 130, 200, 256, 300, 400, 512, 520, 700, 1000, 1024, 1300, 1536, 2048, 2050,
        2100, 3000, 4096, 5000, 6000, 8192, 8200, 12288]
WIDTHS = [8, 40, 64, 72, 78, 128, 136, 200, 256, 334, 500, 512, 832, 1001, 1002, 1003, 1024, 1365, 1536, 2046, 2048,
          2050, 2051, 2731, 3000, 4096, 4100, 8192, 12288]
GROUPS = {0: (1, 1, 1, 2, 4, 1), 1: (1, 1, 1, 1, 4, 1)}      # wave groups over K of a tile class


@pytest.fixture(scope="module")
def forms(tmp_path_factory):
    if shutil.which("hipcc") is None:
        pytest.skip("no hipcc")
    d = tmp_path_factory.mktemp("forms")
    src, out = d / "forms.hip", d / "forms.so"
    src.write_text(DRIVER)
    subprocess.run(["hipcc", "--offload-host-only", "-O1", "-std=c++17", "-fPIC", "-shared", "-w",
                    "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "software_pipelined_tiled_gemm_amd", "csrc"),
                    str(src), "-o", str(out)], check=True)
    L = ctypes.CDLL(str(out))
    i, q = ctypes.c_int, ctypes.c_int64
    L.launches.argtypes = [i, q, q, q, i, i, ctypes.POINTER(i)]
    buf = (i * 128)()

    def of(what, *case):
        """{form: whether it multiplies seven k-tiles or more in a row}"""
        n = L.launches(what, *case, buf)
        assert n >= 0, (what, case)
        recs = [tuple(buf[7 * k:7 * k + 7]) for k in range(n)]
        return [(r[:6], r[6] >= 7 * GROUPS[r[1]][r[2]]) for r in recs]

    return of


def test_the_listed_sizes_reach_every_kernel(forms):
    reached = {f for what, cases in enumerate((listed.GATED, listed.BACKWARD, listed.INT8))
               for c in cases for f in forms(what, *c)}
    wanted = set()
    for M in ROWS:
        for N in WIDTHS:
            for K in WIDTHS:
                for off in (0, 2):
                    for flag in (0, 1):
                        for what in (0, 1, 2):
                            wanted.update(forms(what, M, N, K, flag, off))
    # every product, both stagings
    assert {f[:2] for f, _ in wanted} == {(p, r) for p in range(7) for r in (0, 1)}
    long = {f for f, many in wanted if many}
    missing = [f for f in long if (f, True) not in reached]
    missing += [f for f, _ in wanted if f not in long and (f, False) not in reached]
    assert not missing, sorted(missing)
