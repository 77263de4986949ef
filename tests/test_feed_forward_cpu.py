"""Refusals of the feed-forward operators on a machine without a GPU: every argument check
runs before any HIP call, through the C ABI and through the Python wrappers."""

import ctypes
import os

import pytest

import software_pipelined_tiled_gemm_amd as spg


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(spg.LIB_PATH):
        pytest.fail("libspgemm.so is not built; run __graft_entry__.build()")
    return spg.lib()


def test_gated_plans(L):
    h = ctypes.c_void_p()
    make = lambda *a: L.gemm_gated_create(ctypes.byref(h), *a)
    assert L.gemm_gated_create(None, 8, 8, 8, 1, 1, 1) == 1
    assert make(-1, 8, 8, 1, 1, 1) == 1 and make(8, -1, 8, 1, 1, 1) == 1 and make(8, 8, -1, 1, 1, 1) == 1
    assert make(8, 8, 8, 2, 1, 1) == 1     # fp32 operands
    assert make(8, 8, 8, 3, 1, 1) == 1
    assert make(8, 8, 8, 1, 2, 1) == 1     # layout
    assert make(8, 8, 8, 1, 1, 0) == 1     # no activation
    assert make(8, 8, 8, 1, 1, 4) == 1
    assert make(1 << 31, 8, 8, 1, 1, 1) == 2
    assert not h.value
    assert L.gemm_gated_workspace(None) == -1
    assert L.gemm_gated_destroy(None) == 0


def test_gated_calls(L):
    h = spg.gemm_gated_create(64, 256, 128, "bf16", "kn", "silu")
    ws = spg.gemm_gated_workspace(h)
    assert ws >= 64 * 256 * 2 * 2          # dG and dU
    p = 4096
    run = lambda *a: L.gemm_gated_run(h, *a)
    assert L.gemm_gated_run(None, p, p, p, p, 0, 0, p, ws, 0) == 1
    assert run(0, p, p, p, 0, 0, p, ws, 0) == 1
    assert run(p, 0, p, p, 0, 0, p, ws, 0) == 1
    assert run(p, p, 0, p, 0, 0, p, ws, 0) == 1
    assert run(p, p, p, 0, 0, 0, p, ws, 0) == 1
    assert run(p, p, p, p, p, 0, p, ws, 0) == 1        # G without U
    assert run(p, p, p, p, 0, p, p, ws, 0) == 1
    good = [p] * 9
    for i in range(9):
        bad = list(good)
        bad[i] = 0
        assert L.gemm_gated_backward(h, *bad, p, ws, 0) == 1, i
    assert L.gemm_gated_backward(None, *good, p, ws, 0) == 1
    assert L.gemm_gated_backward(h, *good, 0, ws, 0) == 1
    assert L.gemm_gated_backward(h, *good, p, ws - 1, 0) == 1
    assert L.gemm_gated_backward(h, *good, p + 8, ws, 0) == 1
    spg.gemm_gated_destroy(h)


def test_a_split_reduction_asks_for_its_workspace(L):
    # few tiles and a long reduction: parts, whose sums need memory
    h = spg.gemm_gated_create(96, 256, 8192, "bf16", "kn", "silu")
    p = 4096
    assert spg.gemm_gated_workspace(h) > 0
    assert L.gemm_gated_run(h, p, p, p, p, 0, 0, 0, 0, 0) == 1
    assert L.gemm_gated_run(h, p, p, p, p, 0, 0, p, 16, 0) == 1
    spg.gemm_gated_destroy(h)
    q = spg.gemm_quantized_create(100, 128, 16384, "f32", "none")
    assert spg.gemm_quantized_workspace(q) > 0
    assert L.gemm_quantized_run(q, p, p, p, p, 0, 0, p, 0, 0, 0) == 1
    spg.gemm_quantized_destroy(q)


def test_empty_calls_are_no_ops(L):
    h = spg.gemm_gated_create(0, 256, 128, "f16", "nk", "relu")
    assert L.gemm_gated_run(h, 0, 0, 0, 0, 0, 0, 0, 0, 0) == 0
    spg.gemm_gated_destroy(h)
    h = spg.gemm_gated_create(4, 8, 0, "f16", "nk", "relu")
    assert L.gemm_gated_backward(h, *[0] * 9, 0, 0, 0) == 0
    spg.gemm_gated_destroy(h)
    q = spg.gemm_quantized_create(4, 0, 64, "bf16", "none")
    assert L.gemm_quantized_run(q, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0) == 0
    spg.gemm_quantized_destroy(q)
    assert L.gemm_quantize_rows(0, 1, 0, 64, 0, 0, 0) == 0


def test_quantized_plans_and_calls(L):
    h = ctypes.c_void_p()
    make = lambda *a: L.gemm_quantized_create(ctypes.byref(h), *a)
    assert L.gemm_quantized_create(None, 8, 8, 8, 1, 0) == 1
    assert make(-1, 8, 8, 1, 0) == 1 and make(8, 8, 8, 3, 0) == 1 and make(8, 8, 8, 1, 4) == 1
    assert make(8, 8, 131072, 1, 0) == 2   # the int32 sums could overflow
    assert make(8, 8, 131071, 1, 0) == 0
    L.gemm_quantized_destroy(h)
    assert L.gemm_quantized_workspace(None) == -1 and L.gemm_quantized_destroy(None) == 0
    p = 4096
    q = spg.gemm_quantized_create(8, 64, 64, "bf16", "none")
    good = [p, p, p, p, 0, 0, p]
    assert L.gemm_quantized_run(None, *good, 0, 0, 0) == 1
    for i in (0, 1, 2, 3, 6):
        bad = list(good)
        bad[i] = 0
        assert L.gemm_quantized_run(q, *bad, 0, 0, 0) == 1, i
    assert L.gemm_quantized_run(q, p, p, p, p, p, p, p, 0, 0, 0) == 1   # B2 without an activation
    spg.gemm_quantized_destroy(q)
    q = spg.gemm_quantized_create(8, 64, 64, "bf16", "silu")
    assert L.gemm_quantized_run(q, p, p, p, p, 0, p, p, 0, 0, 0) == 1
    assert L.gemm_quantized_run(q, p, p, p, p, p, 0, p, 0, 0, 0) == 1
    spg.gemm_quantized_destroy(q)


def test_quantize_rows_arguments(L):
    p = 4096
    assert L.gemm_quantize_rows(p, 1, -1, 8, p, p, 0) == 1
    assert L.gemm_quantize_rows(p, 1, 8, -1, p, p, 0) == 1
    assert L.gemm_quantize_rows(p, 3, 8, 8, p, p, 0) == 1
    assert L.gemm_quantize_rows(0, 1, 8, 8, p, p, 0) == 1
    assert L.gemm_quantize_rows(p, 1, 8, 8, 0, p, 0) == 1
    assert L.gemm_quantize_rows(p, 1, 8, 8, p, 0, 0) == 1
    assert L.gemm_quantize_rows(p, 1, 1 << 31, 8, p, p, 0) == 2


def test_wrappers_check_tensors():
    torch = pytest.importorskip("torch")
    x, w, h = torch.zeros(4, 16), torch.zeros(32, 16), torch.zeros(4, 32)
    b = torch.bfloat16
    with spg.Gated(4, 32, 16, "bf16", "nk", "silu") as plan:
        for args in ((x, w.to(b), w.to(b), h.to(b)),                     # type
                     (x.to(b), w.to(b).t(), w.to(b), h.to(b)),           # shape
                     (x.to(b), w.to(b), torch.zeros(16, 32).to(b).t(), h.to(b)),   # strides
                     (x.to(b), w.to(b), w.to(b), h.to(b))):              # host memory
            with pytest.raises(spg.GemmError) as e:
                plan(*args)
            assert e.value.status == 1
    with spg.QuantizedGemm(4, 32, 16, "f32") as q:
        with pytest.raises(spg.GemmError):
            q(x, torch.zeros(4), w.to(torch.int8), torch.zeros(32), h)
    with pytest.raises(spg.GemmError):
        spg.gemm_quantize_rows(x, torch.zeros(4, 15, dtype=torch.int8), torch.zeros(4))
    with pytest.raises(KeyError):
        spg.Gated(4, 32, 16, "f64")


def test_serving_needs_no_room_for_the_backward_pass(L):
    assert L.gemm_gated_run_workspace(None) == -1
    with spg.Gated(8192, 12288, 4096, "bf16", "nk", "silu") as plan:
        assert plan.workspace_bytes(backward=False) == 0
        assert plan.workspace_bytes() >= 8192 * 12288 * 2 * 2
    p = 4096
    for layout, K in (("kn", 8192), ("nk", 8192), ("kn", 1001), ("nk", 1001)):
        h = spg.gemm_gated_create(96, 256, K, "bf16", layout, "silu")
        run, both = spg.gemm_gated_run_workspace(h), spg.gemm_gated_workspace(h)
        assert 0 <= run <= both
        if K == 8192:      # split: the projection asks for its own part and for no more
            assert run > 0 and L.gemm_gated_run(h, p, p, p, p, 0, 0, p, run - 1, 0) == 1
        spg.gemm_gated_destroy(h)
