"""Workspaces of the layer norm's backward pass, on a machine without a GPU: what every kind of row
needs, and that less is refused before any HIP call."""

import ctypes
import os

import pytest

import software_pipelined_tiled_gemm_amd as spg

P = 4096


@pytest.mark.parametrize("rows,K,needs", [(256, 4, False), (257, 4, True), (1 << 29, 1, True), (200, 20000, False), (3000, 20000, True),
                                          (1, 4096, True), (9, 520, True), (0, 4, False), (0, 4096, False), (0, 20000, False),
                                          (100000, 0, False), (300, 1 << 29, False)])
def test_backward(rows, K, needs):
    if not os.path.exists(spg.LIB_PATH):
        pytest.fail("libspgemm.so is not built; run __graft_entry__.build()")
    L, h = spg.lib(), ctypes.c_void_p()
    assert L.gemm_norm_create(ctypes.byref(h), rows, K, 1, 2, 1e-5) == 0
    ws = L.gemm_norm_workspace(h)
    assert (ws > 0) == needs
    # no more than a float a column, gradient and workgroup
    assert ws <= 2048 * 2 * (K + 7) * 4
    if needs:
        for a in ((0, ws), (P, ws - 1), (P + 8, ws)):
            assert L.gemm_norm_backward(h, P, P, P, P, P, P, P, P, *a, 0) == 1
            assert L.gemm_norm_backward(h, P, P, P, P, P, P, P, 0, *a, 0) == 1
    L.gemm_norm_destroy(h)
