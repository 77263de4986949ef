"""Refusals of the operators of a mixture of experts on a machine without a GPU: every argument
check runs before any HIP call, through the C ABI and through the Python wrappers; what the
wrappers pass on, with the entry points replaced by recorders."""

import ctypes
import os

import pytest

import software_pipelined_tiled_gemm_amd as spg
from tests.test_feed_forward_calls import Like, OnDevice, P, Recorder

torch = pytest.importorskip("torch")

p = 4096


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(spg.LIB_PATH):
        pytest.fail("libspgemm.so is not built; run __graft_entry__.build()")
    return spg.lib()


def test_norm_plans(L):
    h = ctypes.c_void_p()
    make = lambda *a: L.gemm_norm_create(ctypes.byref(h), *a)
    assert L.gemm_norm_create(None, 8, 8, 1, 1, 1e-5) == 1
    assert make(-1, 8, 1, 1, 1e-5) == 1 and make(8, -1, 1, 1, 1e-5) == 1
    assert make(8, 8, 3, 1, 1e-5) == 1 and make(8, 8, 1, 0, 1e-5) == 1 and make(8, 8, 2, 1, 1e-5) == 1
    for eps in (-1e-5, float("nan"), float("inf")):
        assert make(8, 8, 1, 1, eps) == 1
    assert make(1 << 31, 8, 1, 1, 1e-5) == 2 and make(8, 1 << 31, 1, 1, 1e-5) == 2
    assert not h.value and L.gemm_norm_workspace(None) == -1 and L.gemm_norm_destroy(None) == 0
    assert make(0, 0, 2, 2, 0.0) == 0
    L.gemm_norm_destroy(h)


def test_norm_calls(L):
    h = ctypes.c_void_p()
    assert L.gemm_norm_create(ctypes.byref(h), 64, 4096, 1, 2, 1e-5) == 0
    ws = L.gemm_norm_workspace(h)
    good = [p] * 6
    assert L.gemm_norm_run(None, *good, 0) == 1
    for i in (0, 3, 4, 5):                               # X, Y; mean without rstd and the reverse
        bad = list(good)
        bad[i] = 0
        assert L.gemm_norm_run(h, *bad, 0) == 1, i
    good = [p] * 8
    assert L.gemm_norm_backward(None, *good, p, ws, 0) == 1
    for i in (0, 1, 3, 4, 5):                            # dY, X, mean, rstd, dX
        bad = list(good)
        bad[i] = 0
        assert L.gemm_norm_backward(h, *bad, p, ws, 0) == 1, i
    if ws:
        assert L.gemm_norm_backward(h, *good, 0, ws, 0) == 1
        assert L.gemm_norm_backward(h, *good, p, ws - 1, 0) == 1
        assert L.gemm_norm_backward(h, *good, p + 8, ws, 0) == 1
    L.gemm_norm_destroy(h)


def test_route_plans_and_calls(L):
    h = ctypes.c_void_p()
    make = lambda *a: L.gemm_route_create(ctypes.byref(h), *a)
    assert L.gemm_route_create(None, 8, 8, 2, 2, 0) == 1
    assert make(-1, 8, 2, 2, 0) == 1 and make(8, 0, 1, 2, 0) == 1 and make(8, 8, 0, 2, 0) == 1
    assert make(8, 8, 9, 2, 0) == 1 and make(8, 200, 65, 2, 0) == 1       # more choices than experts, than 64
    assert make(8, 8, 2, 3, 0) == 1 and make(8, 8, 2, 2, 2) == 1
    assert make(8, 1025, 2, 2, 0) == 2 and make(1 << 30, 8, 2, 2, 0) == 2
    assert not h.value and L.gemm_route_workspace(None) == -1 and L.gemm_route_destroy(None) == 0
    assert make(5000, 64, 8, 1, 1) == 0
    ws = L.gemm_route_workspace(h)
    assert ws > 0
    for i in range(6):
        bad = [p] * 6
        bad[i] = 0
        assert L.gemm_route_run(h, *bad, p, ws, 0) == 1, i
    assert L.gemm_route_run(None, *[p] * 6, p, ws, 0) == 1
    assert L.gemm_route_run(h, *[p] * 6, 0, ws, 0) == 1 and L.gemm_route_run(h, *[p] * 6, p, ws - 1, 0) == 1
    for i in range(4):
        bad = [p] * 4
        bad[i] = 0
        assert L.gemm_route_backward(h, *bad, 0) == 1, i
    L.gemm_route_destroy(h)


def test_grouped_plans(L):
    h = ctypes.c_void_p()
    for make in (lambda *a: L.gemm_grouped_create(ctypes.byref(h), *a),
                 lambda *a: L.gemm_experts_create(ctypes.byref(h), *a, 1)):
        assert make(-1, 8, 8, 2, -1, 1, 1) == 1 and make(8, -1, 8, 2, -1, 1, 1) == 1 and make(8, 8, -1, 2, -1, 1, 1) == 1
        assert make(8, 8, 8, 0, -1, 1, 1) == 1 and make(8, 8, 8, 2, -2, 1, 1) == 1
        assert make(8, 8, 8, 2, -1, 2, 1) == 1 and make(8, 8, 8, 2, -1, 1, 2) == 1
        assert make(8, 8, 8, 65536, -1, 1, 1) == 2 and make(1 << 31, 8, 8, 2, -1, 1, 1) == 2
        assert make(8, 8, 8, 2, 1 << 31, 1, 1) == 2
        assert not h.value
    assert L.gemm_grouped_create(None, 8, 8, 8, 2, -1, 1, 1) == 1
    assert L.gemm_experts_create(None, 8, 8, 8, 2, -1, 1, 1, 1) == 1
    for act in (0, 4):
        assert L.gemm_experts_create(ctypes.byref(h), 8, 8, 8, 2, -1, 1, 1, act) == 1
    for f in (L.gemm_grouped_workspace, L.gemm_grouped_run_workspace, L.gemm_experts_workspace, L.gemm_experts_run_workspace):
        assert f(None) == -1
    assert L.gemm_grouped_destroy(None) == 0 and L.gemm_experts_destroy(None) == 0


@pytest.mark.parametrize("tokens", [-1, 40])
@pytest.mark.parametrize("layout", [0, 1])
def test_grouped_calls(L, layout, tokens):
    src = 0 if tokens < 0 else p
    wrong = p - src                                      # a source that the plan has not, or none where it has
    h = ctypes.c_void_p()
    assert L.gemm_grouped_create(ctypes.byref(h), 96, 256, 512, 4, tokens, 1, layout) == 0
    ws = L.gemm_grouped_workspace(h)
    good = [p, p, p, src, p]                             # X W offsets source Y
    run = lambda a, *s: L.gemm_grouped_run(h, *a, *(s or (p, 1 << 40)), 0)
    for i in (0, 1, 2, 4):
        assert run(good[:i] + [0] + good[i + 1:]) == 1, i
    assert run(good[:3] + [wrong] + good[4:]) == 1
    assert L.gemm_grouped_run(None, *good, p, 1 << 40, 0) == 1
    need = L.gemm_grouped_run_workspace(h)
    if need:
        assert run(good, 0, need) == 1 and run(good, p, need - 1) == 1 and run(good, p + 8, need) == 1
    good = [p, p, p, p, src, p, p]                       # dY X W offsets source dX dW
    back = lambda a, *s: L.gemm_grouped_backward(h, *a, *(s or (p, 1 << 40)), 0)
    for i in (0, 1, 2, 3):
        assert back(good[:i] + [0] + good[i + 1:]) == 1, i
    assert back(good[:4] + [wrong] + good[5:]) == 1
    if ws:
        assert back(good, 0, ws) == 1 and back(good, p, ws - 1) == 1 and back(good, p + 8, ws) == 1
    assert back(good[:5] + [0, 0]) == 0                  # neither gradient: nothing to do
    L.gemm_grouped_destroy(h)

    assert L.gemm_experts_create(ctypes.byref(h), 96, 256, 512, 4, tokens, 1, layout, 1) == 0
    ws = L.gemm_experts_workspace(h)
    assert ws >= 96 * 256 * 2 * 2                        # dG and dU
    good = [p, p, p, p, src, p, p, p]                    # X Wg Wu offsets source H G U
    run = lambda a: L.gemm_experts_run(h, *a, p, 1 << 40, 0)
    for i in (0, 1, 2, 3, 5, 6, 7):
        assert run(good[:i] + [0] + good[i + 1:]) == 1, i
    assert run(good[:4] + [wrong] + good[5:]) == 1
    good = [p] * 7 + [src] + [p] * 3                     # dH X Wg Wu G U offsets source dX dWg dWu
    back = lambda a, *s: L.gemm_experts_backward(h, *a, *(s or (p, 1 << 40)), 0)
    for i in range(11):
        if i != 7:
            assert back(good[:i] + [0] + good[i + 1:]) == 1, i
    assert back(good[:7] + [wrong] + good[8:]) == 1
    assert back(good, 0, ws) == 1 and back(good, p, ws - 1) == 1 and back(good, p + 8, ws) == 1
    assert L.gemm_experts_backward(None, *good, p, ws, 0) == 1
    L.gemm_experts_destroy(h)


def test_combine_plans_and_calls(L):
    h = ctypes.c_void_p()
    make = lambda *a: L.gemm_combine_create(ctypes.byref(h), *a)
    assert L.gemm_combine_create(None, 8, 2, 16, 8, 1) == 1
    assert make(-1, 2, 16, 8, 1) == 1 and make(8, 0, 16, 8, 1) == 1 and make(8, 65, 16, 8, 1) == 1
    assert make(8, 2, -1, 8, 1) == 1 and make(8, 2, 16, -1, 1) == 1 and make(8, 2, 16, 8, 3) == 1
    assert make(1 << 30, 2, 16, 8, 1) == 2 and make(8, 2, 1 << 31, 8, 1) == 2 and make(8, 2, 16, 1 << 31, 1) == 2
    assert not h.value and L.gemm_combine_destroy(None) == 0
    assert make(8, 2, 16, 64, 1) == 0
    assert L.gemm_combine_run(None, p, p, p, p, 0) == 1
    for a in ((0, p, p, p), (p, 0, p, p), (p, p, p, 0)):
        assert L.gemm_combine_run(h, *a, 0) == 1
    for a in ((0, p, p, p, p, p), (p, 0, p, p, p, p), (p, p, 0, p, p, p), (p, p, p, p, 0, p)):
        assert L.gemm_combine_backward(h, *a, 0) == 1
    L.gemm_combine_destroy(h)


ENTRIES = ["gemm_norm_run", "gemm_norm_backward", "gemm_route_run", "gemm_route_backward", "gemm_grouped_run",
           "gemm_grouped_backward", "gemm_experts_run", "gemm_experts_backward", "gemm_combine_run", "gemm_combine_backward"]


@pytest.fixture
def lib(monkeypatch):
    """The library with recorders in place of the entry points that launch, behind the Python
    call path."""
    real = spg.lib()

    class Lib:
        def __getattr__(self, name):
            return getattr(real, name)

    fake = Lib()
    for name in ENTRIES:
        setattr(fake, name, Recorder())
    monkeypatch.setattr(spg, "_lib", fake)
    monkeypatch.setattr(spg, "_calls", None)
    return fake


B, F, I = torch.bfloat16, torch.float32, torch.int32
T, E, K_, R, N, D = 40, 6, 2, 80, 72, 136


def passes(lib):
    """(entry point, call on tensors, their shapes and types in the call's order, the C order's index of each)"""
    norm, route = spg.LayerNorm(T, D, "bf16", "f32"), spg.Router(T, E, K_, "f32")
    plain = spg.GroupedGemm(R, N, D, E, "bf16", "nk")
    gated = spg.GroupedGated(R, N, D, E, "bf16", "kn", tokens=T)
    comb = spg.Combine(T, K_, R, N, "bf16")
    x, h, w, wk = ((T, D), B), ((R, N), B), ((E, N, D), B), ((E, D, N), B)
    off, src, tk, tki = ((E + 1,), I), ((R,), I), ((T, K_), F), ((T, K_), I)
    par, row, xs, lg, o = ((D,), F), ((T,), F), ((R, D), B), ((T, E), F), ((T, N), B)
    return [
        (lib.gemm_norm_run, lambda a, **k: norm(*a[:4], mean=a[4], rstd=a[5], **k), [x, par, par, x, row, row]),
        (lib.gemm_norm_backward, lambda a, **k: norm.backward(*a, **k), [x, x, par, row, row, x, par, par]),
        (lib.gemm_route_run, lambda a, **k: route(*a, **k), [lg, tk, tki, tki, src, off]),
        (lib.gemm_route_backward, lambda a, **k: route.backward(*a, **k), [lg, tki, tk, lg]),
        (lib.gemm_grouped_run, lambda a, **k: plain(*a, **k), [xs, w, off, h]),
        (lib.gemm_grouped_backward, lambda a, **k: plain.backward(*a, **k), [h, xs, w, off, xs, w]),
        (lib.gemm_experts_run, lambda a, **k: gated(*a[:5], source=a[5], G=a[6], U=a[7], **k),
         [x, wk, wk, off, h, src, h, h]),
        (lib.gemm_experts_backward, lambda a, **k: gated.backward(*a[:10], source=a[10], **k),
         [h, x, wk, wk, h, h, off, xs, wk, wk, src]),
        (lib.gemm_combine_run, lambda a, **k: comb(*a, **k), [h, tki, tk, o]),
        (lib.gemm_combine_backward, lambda a, **k: comb.backward(*a, **k), [o, h, tki, tk, h, tk]),
    ]


@pytest.mark.parametrize("which", range(len(ENTRIES)))
def test_tensors_that_do_not_fit(lib, which):
    fn, call, specs = passes(lib)[which]
    good = [Like(s, t) for s, t in specs]
    for i, (shape, dtype) in enumerate(specs):
        for bad in (Like(shape[:-1] + (shape[-1] + 1,), dtype), Like(shape + (1,), dtype),
                    Like(shape, torch.float64), Like(shape, dtype, device=1 if i else 2),
                    torch.empty(shape, dtype=dtype), torch.empty(shape + (2,), dtype=dtype)[..., 0]):
            with pytest.raises(spg.GemmError) as e:
                call(good[:i] + [bad] + good[i + 1:], stream=0)
            assert e.value.status == 1 and not fn.calls, (i, bad.shape)
    call(good, stream=7)
    assert len(fn.calls) == 1 and fn.calls[0][-1] == 7


@pytest.mark.parametrize("which", [1, 2, 4, 5, 6, 7])
def test_workspaces_that_do_not_fit(lib, which):
    fn, call, specs = passes(lib)[which]
    good = [Like(s, t) for s, t in specs]
    for bad, why in ((torch.empty(64, dtype=torch.uint8), "not on a GPU"),
                     (torch.empty(1, dtype=torch.uint8).expand(64), "not contiguous"),
                     (OnDevice(64, device=1), "on another device")):
        with pytest.raises(spg.GemmError, match="workspace is " + why):
            call(good, workspace=bad, stream=0)
        assert not fn.calls
    call(good, workspace=OnDevice(64), stream=0)
    call(good, workspace=None, stream=0)
    call(good, workspace=torch.empty(0, dtype=torch.uint8), stream=0)
    assert [c[-3:-1] for c in fn.calls] == [(P, 64), (None, 0), (None, 0)]


def test_raw_pointers(lib):
    for fn, call, specs in passes(lib):
        call([P + 16 * i for i in range(len(specs))], stream=0)
        assert len(fn.calls) == 1


def test_plans_that_cannot_be(L):
    for make in (lambda: spg.LayerNorm(4, 8, "bf16", "f16"), lambda: spg.Router(4, 8, 9), lambda: spg.GroupedGemm(4, 8, 8, 0),
                 lambda: spg.GroupedGated(4, 8, 8, 2, act="none"), lambda: spg.Combine(4, 0, 4, 8),
                 lambda: spg.GroupedGemm(4, 8, 8, 2, "f32")):
        with pytest.raises(spg.GemmError) as e:
            make()
        assert e.value.status == 1
    with pytest.raises(KeyError):
        spg.LayerNorm(4, 8, "f64")


def test_closed_plans_are_refused(L):
    plan = spg.Combine(4, 2, 8, 16)
    plan.close()
    plan.close()
    with pytest.raises(spg.GemmError) as e:
        plan(P, P, P, P, stream=0)
    assert e.value.status == 1
