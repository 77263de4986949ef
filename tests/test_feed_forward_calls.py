"""What the Python wrappers of the feed-forward operators pass on and what they refuse, with the
C entry points replaced by recorders: nothing is launched, no GPU is needed."""

import pytest

import software_pipelined_tiled_gemm_amd as spg

torch = pytest.importorskip("torch")

P = 1 << 20      # a raw device pointer


class Recorder:
    """Stands for a C entry point: keeps the arguments, succeeds."""

    def __init__(self):
        self.calls = []

    def __call__(self, *args):
        self.calls.append(args)
        return 0


class OnDevice:
    """The attributes of a dense uint8 device tensor that the wrappers read."""

    dtype, is_cuda = torch.uint8, True

    def __init__(self, n, device=0):
        self.shape, self.nbytes, self.device = (n,), n, device

    def get_device(self):
        return self.device

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return P


class Like(OnDevice):
    """... of an operand."""

    def __init__(self, shape, dtype, device=0):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, device


@pytest.fixture
def lib(monkeypatch):
    """The library with recorders in place of the entry points that launch, behind the Python
    call path."""
    real = spg.lib()

    class Lib:
        def __getattr__(self, name):
            return getattr(real, name)

    fake = Lib()
    for name in ("gemm_gated_run", "gemm_gated_backward", "gemm_quantized_run", "gemm_quantize_rows"):
        setattr(fake, name, Recorder())
    monkeypatch.setattr(spg, "_lib", fake)
    monkeypatch.setattr(spg, "_calls", None)
    monkeypatch.setattr(spg, "_address", lambda fn: 0)
    return fake


M, N, K = 96, 256, 8192


def calls(lib):
    """(entry point, call with a workspace) of every operator that takes one: the classes, then
    the functions of the entry points' names."""
    gated, q = spg.Gated(M, N, K), spg.QuantizedGemm(M, N, K)
    return [
        (lib.gemm_gated_run, gated.workspace_bytes(), lambda **kw: gated(P, P, P, P, stream=0, **kw)),
        (lib.gemm_gated_backward, gated.workspace_bytes(), lambda **kw: gated.backward(*[P] * 9, stream=0, **kw)),
        (lib.gemm_quantized_run, q.workspace_bytes(), lambda **kw: q(P, P, P, P, P, stream=0, **kw)),
        (lib.gemm_gated_run, gated.workspace_bytes(),
         lambda **kw: spg.gemm_gated_run(gated.handle, P, P, P, P, stream=0, **kw)),
        (lib.gemm_gated_backward, gated.workspace_bytes(),
         lambda **kw: spg.gemm_gated_backward(gated.handle, *[P] * 9, stream=0, **kw)),
        (lib.gemm_quantized_run, q.workspace_bytes(),
         lambda **kw: spg.gemm_quantized_run(q.handle, P, P, P, P, P, stream=0, **kw)),
    ]


@pytest.mark.parametrize("which", range(6))
def test_workspaces_that_the_kernels_could_not_write(lib, which):
    fn, n, call = calls(lib)[which]
    assert n > 0
    for bad, why in ((torch.empty(n, dtype=torch.uint8), "not on a GPU"),
                     (torch.empty(1, dtype=torch.uint8).expand(n), "not contiguous"),
                     (torch.empty(2 * n, dtype=torch.uint8)[::2], "not contiguous")):
        with pytest.raises(spg.GemmError, match="workspace is " + why) as e:
            call(workspace=bad)
        assert e.value.status == 1 and not fn.calls
    call(workspace=OnDevice(n))
    call(workspace=None)
    assert [c[-3:-1] for c in fn.calls] == [(P, n), (None, 0)]


def test_a_size_beyond_the_workspace(lib):
    for fn, n, call in calls(lib)[3:]:
        with pytest.raises(spg.GemmError, match="workspace has") as e:
            call(workspace=OnDevice(n), workspace_bytes=n + 1)
        assert e.value.status == 1 and not fn.calls
        call(workspace=OnDevice(n + 16), workspace_bytes=n)
        call(workspace=P, workspace_bytes=n)
        assert [c[-3:-1] for c in fn.calls] == [(P, n), (P, n)]
        fn.calls.clear()


def test_a_workspace_on_another_device(lib):
    b, i8, f32 = torch.bfloat16, torch.int8, torch.float32
    x, w, h = Like((M, K), b), Like((N, K), b), Like((M, N), b)
    with spg.Gated(M, N, K) as plan, spg.QuantizedGemm(M, N, K) as q:
        for fn, n, call in (
                (lib.gemm_gated_run, plan.workspace_bytes(), lambda ws: plan(x, w, w, h, workspace=ws, stream=0)),
                (lib.gemm_gated_backward, plan.workspace_bytes(),
                 lambda ws: plan.backward(h, x, w, w, h, h, x, w, w, workspace=ws, stream=0)),
                (lib.gemm_quantized_run, q.workspace_bytes(),
                 lambda ws: q(Like((M, K), i8), Like((M,), f32), Like((N, K), i8), Like((N,), f32), h, workspace=ws, stream=0))):
            with pytest.raises(spg.GemmError, match="workspace is on another device"):
                call(OnDevice(n, device=1))
            assert not fn.calls
            call(OnDevice(n))
            assert len(fn.calls) == 1


def test_quantising_from_a_raw_pointer_checks_the_tensors(lib, monkeypatch):
    fn = lib.gemm_quantize_rows
    i8, f32 = torch.int8, torch.float32
    a, s = Like((4, 16), i8), Like((4,), f32)
    args = dict(dtype="bf16", shape=(4, 16))
    for A, scale in ((torch.zeros(4, 16, dtype=i8), s), (a, torch.zeros(4)), (Like((4, 15), i8), s), (Like((4, 16), f32), s),
                     (a, Like((3,), f32)), (a, Like((4,), i8)), (a, Like((4,), f32, device=1))):
        with pytest.raises(spg.GemmError) as e:
            spg.gemm_quantize_rows(P, A, scale, stream=0, **args)
        assert e.value.status == 1 and not fn.calls
    # the tensors' device gives the stream, as for every other call
    monkeypatch.setattr(spg, "_raw_stream", lambda device: 1000 + device)
    spg.gemm_quantize_rows(P, Like((2, 2, 16), i8, device=3), Like((2, 2), f32, device=3), **args)
    spg.gemm_quantize_rows(P, P, P, **args)
    assert [c[-1] for c in fn.calls] == [1003, None] and all(c[:4] == (P, 1, 4, 16) for c in fn.calls)


def test_an_exchange_interface_of_another_kind(monkeypatch):
    # a torch whose interface cannot be read: the Python path, not an error out of a plan
    import ctypes
    import os
    if not os.path.exists(os.path.join(os.path.dirname(spg.__file__), "_calls.so")):
        pytest.fail("_calls.so is not built; run __graft_entry__.build()")
    new = ctypes.pythonapi.PyCapsule_New
    new.restype, new.argtypes = ctypes.py_object, [ctypes.c_void_p, ctypes.c_char_p, ctypes.c_void_p]
    for other in (new(P, b"dlpack_exchange_api_of_another_version", None), new(P, None, None), object()):
        monkeypatch.setattr(torch.Tensor, "__dlpack_c_exchange_api__", other, raising=False)
        monkeypatch.setattr(spg, "_calls", False)
        with spg.Gated(4, 32, 16) as plan:
            assert plan._calls is None


def test_the_build_without_torch_or_headers(monkeypatch, tmp_path, capsys):
    # the library itself needs neither: its C users build without the wrappers' call path
    import sys
    from software_pipelined_tiled_gemm_amd import build
    out = tmp_path / "_calls.so"
    with monkeypatch.context() as m:
        m.setitem(sys.modules, "torch", None)
        assert build.build_calls(str(out)) is None
        assert "torch" in capsys.readouterr().err
    with monkeypatch.context() as m:
        m.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
        assert build.build_calls(str(out)) is None
        assert "Python.h" in capsys.readouterr().err
    assert not list(tmp_path.iterdir())
    assert build.build_calls(str(out)) == str(out) and out.exists()


def test_raw_workspaces_through_the_classes(lib):
    # a raw pointer is taken at its word, as raw operands are: workspace_bytes() of memory
    for fn, n, call in calls(lib)[:3]:
        call(workspace=P)
        assert fn.calls[-1][-3:-1] == (P, n)
    # the functions of the entry points' names take the size
    for fn, n, call in calls(lib)[3:]:
        call(workspace=P)
        assert fn.calls[-1][-3:-1] == (P, 0)


def test_empty_workspaces(lib):
    # workspace_bytes() may be 0: a tensor without bytes is no workspace, wherever it is
    for fn, n, call in calls(lib):
        call(workspace=torch.empty(0, dtype=torch.uint8))
        assert fn.calls[-1][-3:-1] == (None, 0)
