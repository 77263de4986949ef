"""Python binding of the MI355X software-pipelined tiled GEMM and the feed-forward operators
(C ABI in include/spgemm.h) and of the standalone elementwise GELU (include/spgelu.h).

Argument marshalling only: every step of C = epi(A . B) runs in the HIP
kernels of ``libspgemm.so``.  PyTorch is used by callers for device memory and
streams; this module accepts torch tensors (device pointer + current stream are
taken from them) or raw integer device pointers.

If the shared library has not been built, importing works but every call raises
``GemmError`` -- there is no CPU fallback.
"""

from __future__ import annotations

import ctypes
import math
import os
import struct
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libspgemm.so")
# The poison library: the same C ABI built with -DSPG_POISON from a subset of the
# configurations, every released ring region overwritten with NaN (a race detector
# for the GPU tests; build.build_poison()).
POISON_LIB_PATH = os.path.join(_HERE, "libspgemm_poison.so")

GEMM_OK = 0
STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported", 3: "out of memory",
          4: "HIP runtime error", 5: "internal error"}
DTYPES = {"f16": 0, "bf16": 1, "f32": 2}
B_LAYOUTS = {"kn": 0, "nk": 1}
EPILOGUES = {"none": 0, "gelu_tanh": 1, "relu": 2}
ACTIVATIONS = {"none": 0, "silu": 1, "gelu_tanh": 2, "relu": 3}
STAGING = {0: "direct", 1: "vgpr", 2: "direct-spread", 3: "producer-wave", 4: "direct-a-deep",
           5: "direct-late-release", 6: "direct-b-deep", 7: "vgpr-any-alignment"}


class GemmError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS.get(status, status)} (status {status})")
        self.status = status


class TileConfig(ctypes.Structure):
    _fields_ = [("block_m", ctypes.c_int32), ("block_n", ctypes.c_int32),
                ("block_k", ctypes.c_int32), ("stages", ctypes.c_int32),
                ("wave_m", ctypes.c_int32), ("wave_n", ctypes.c_int32),
                ("swizzle", ctypes.c_int32), ("group_m", ctypes.c_int32),
                ("xcd_remap", ctypes.c_int32), ("staging", ctypes.c_int32),
                ("lookahead", ctypes.c_int32), ("schedule", ctypes.c_int32),
                ("persistent", ctypes.c_int32), ("store", ctypes.c_int32),
                ("mfma", ctypes.c_int32)]

    def __init__(self, **kw):
        kw.setdefault("lookahead", 1)
        super().__init__(**kw)

    def as_dict(self):
        return {k: int(getattr(self, k)) for k, _ in self._fields_}

    @classmethod
    def from_dict(cls, d):
        c = cls()
        for k, _ in cls._fields_:
            setattr(c, k, int(d.get(k, 1 if k == "lookahead" else 0)))
        return c

    def __repr__(self):
        d = self.as_dict()
        return (f"TileConfig({d['block_m']}x{d['block_n']}x{d['block_k']}, S={d['stages']}, "
                f"wave {d['wave_m']}x{d['wave_n']}, swizzle={d['swizzle']}, "
                f"group_m={d['group_m']}, xcd_remap={d['xcd_remap']}, "
                f"staging={STAGING.get(d['staging'], d['staging'])}, lookahead={d['lookahead']}, "
                f"schedule={('manual', 'compiler', 'ping-pong')[d['schedule']] if 0 <= d['schedule'] <= 2 else d['schedule']}"
                f"{', persistent' if d['persistent'] else ''}{', direct store' if d['store'] else ''}"
                f"{', mfma 16x16x32' if d['mfma'] == 16 else ''})")


EXPORTED = ("gemm_create", "gemm_run", "gemm_destroy", "gemm_get_config", "gemm_launch_config",
            "gemm_autotune",
            "gemm_num_configs", "gemm_list_config", "gemm_lds_bytes", "gemm_status_string",
            "gemm_last_hip_error", "gemm_wait_timeouts", "gelu_run",
            "gemm_gated_create", "gemm_gated_workspace", "gemm_gated_run_workspace",
            "gemm_gated_run", "gemm_gated_backward",
            "gemm_gated_destroy", "gemm_quantized_create", "gemm_quantized_workspace",
            "gemm_quantized_run", "gemm_quantized_destroy", "gemm_quantize_rows")

_lib = None
_poison_lib = None


def lib():
    """Load libspgemm.so (raises GemmError if it is missing: no fallback path exists)."""
    global _lib
    if _lib is None:
        _lib = _load(LIB_PATH)
    return _lib


def poison_lib():
    """Load libspgemm_poison.so, the race-detecting test build of the same C ABI."""
    global _poison_lib
    if _poison_lib is None:
        _poison_lib = _load(POISON_LIB_PATH)
    return _poison_lib


def _load(path):
    if not os.path.exists(path):
        raise GemmError(5, f"HIP library {path} is not built (run __graft_entry__.build())")
    # PyTorch-ROCm ships its own libamdhip64 / libhsa-runtime64.  Load it first so this
    # library binds (by soname) to that same HIP runtime instead of a second copy from
    # /opt/rocm: two HIP runtimes in one process do not share devices.
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    L = ctypes.CDLL(path)
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    L.gemm_create.restype = ctypes.c_int
    L.gemm_create.argtypes = [ctypes.POINTER(vp), i64, i64, i64, ctypes.c_int, ctypes.c_int,
                              ctypes.c_int, ctypes.c_int, ctypes.POINTER(TileConfig)]
    L.gemm_run.restype = ctypes.c_int
    L.gemm_run.argtypes = [vp, vp, vp, vp, vp]
    L.gemm_destroy.restype = ctypes.c_int
    L.gemm_destroy.argtypes = [vp]
    L.gemm_get_config.restype = ctypes.c_int
    L.gemm_get_config.argtypes = [vp, ctypes.POINTER(TileConfig)]
    L.gemm_launch_config.restype = ctypes.c_int
    L.gemm_launch_config.argtypes = [vp, vp, vp, vp, ctypes.POINTER(TileConfig)]
    L.gemm_autotune.restype = ctypes.c_int
    L.gemm_autotune.argtypes = [vp, vp, vp, vp, vp, ctypes.c_int, ctypes.POINTER(ctypes.c_double)]
    L.gemm_num_configs.restype = i32
    L.gemm_num_configs.argtypes = []
    L.gemm_list_config.restype = ctypes.c_int
    L.gemm_list_config.argtypes = [i32, ctypes.POINTER(TileConfig)]
    L.gemm_lds_bytes.restype = i64
    L.gemm_lds_bytes.argtypes = [ctypes.POINTER(TileConfig)]
    L.gemm_status_string.restype = ctypes.c_char_p
    L.gemm_status_string.argtypes = [ctypes.c_int]
    L.gemm_last_hip_error.restype = ctypes.c_char_p
    L.gemm_last_hip_error.argtypes = []
    L.gemm_wait_timeouts.restype = ctypes.c_int
    L.gemm_wait_timeouts.argtypes = [ctypes.POINTER(ctypes.c_uint32), i32]
    L.gelu_run.restype = ctypes.c_int
    L.gelu_run.argtypes = [vp, vp, i64, ctypes.c_int, vp]
    en = ctypes.c_int
    for name, res, args in (
            ("gemm_gated_create", en, [ctypes.POINTER(vp), i64, i64, i64, en, en, en]),
            ("gemm_gated_workspace", i64, [vp]),
            ("gemm_gated_run_workspace", i64, [vp]),
            ("gemm_gated_run", en, [vp] * 8 + [i64, vp]),
            ("gemm_gated_backward", en, [vp] * 11 + [i64, vp]),
            ("gemm_gated_destroy", en, [vp]),
            ("gemm_quantized_create", en, [ctypes.POINTER(vp), i64, i64, i64, en, en]),
            ("gemm_quantized_workspace", i64, [vp]),
            ("gemm_quantized_run", en, [vp] * 9 + [i64, vp]),
            ("gemm_quantized_destroy", en, [vp]),
            ("gemm_quantize_rows", en, [vp, en, i64, i64, vp, vp, vp])):
        f = getattr(L, name)
        f.restype, f.argtypes = res, args
    return L


def _check(status: int, what: str):
    if status != GEMM_OK:
        if status == 4:
            what = f"{what} [{gemm_last_hip_error()}]"
        raise GemmError(status, what)


def _ptr(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return int(x.data_ptr())  # torch tensor


def _stream(stream, *tensors) -> Optional[int]:
    if stream is not None:
        return stream if isinstance(stream, int) else int(stream.cuda_stream)
    for t in tensors:
        if t is not None and not isinstance(t, int) and getattr(t, "is_cuda", False):
            import torch
            return int(torch.cuda.current_stream(t.device).cuda_stream)
    return None


# ---- the C entry points, same names --------------------------------------------------

def gemm_create(M: int, N: int, K: int, in_dtype: str = "bf16", out_dtype: str = "bf16",
                b_layout: str = "kn", epilogue: str = "none",
                force: Optional[TileConfig] = None) -> int:
    h = ctypes.c_void_p()
    st = lib().gemm_create(ctypes.byref(h), M, N, K, DTYPES[in_dtype], DTYPES[out_dtype],
                           B_LAYOUTS[b_layout], EPILOGUES[epilogue],
                           ctypes.byref(force) if force is not None else None)
    _check(st, "gemm_create")
    return int(h.value)


def gemm_run(handle: int, A, B, C, stream=None) -> None:
    st = lib().gemm_run(handle, _ptr(A), _ptr(B), _ptr(C), _stream(stream, A, B, C))
    _check(st, "gemm_run")


def gemm_destroy(handle: Optional[int]) -> None:
    _check(lib().gemm_destroy(handle), "gemm_destroy")


def gemm_get_config(handle: int) -> TileConfig:
    c = TileConfig()
    _check(lib().gemm_get_config(handle, ctypes.byref(c)), "gemm_get_config")
    return c


def gemm_launch_config(handle: int, A, B, C) -> TileConfig:
    """The configuration gemm_run would launch with these operands (their alignment)."""
    c = TileConfig()
    _check(lib().gemm_launch_config(handle, _ptr(A), _ptr(B), _ptr(C), ctypes.byref(c)),
           "gemm_launch_config")
    return c


def gemm_autotune(handle: int, A, B, C, stream=None, reps: int = 10) -> float:
    us = ctypes.c_double()
    st = lib().gemm_autotune(handle, _ptr(A), _ptr(B), _ptr(C), _stream(stream, A, B, C), reps,
                             ctypes.byref(us))
    _check(st, "gemm_autotune")
    return float(us.value)


def gemm_num_configs() -> int:
    return int(lib().gemm_num_configs())


def gemm_list_config(index: int) -> TileConfig:
    c = TileConfig()
    _check(lib().gemm_list_config(index, ctypes.byref(c)), "gemm_list_config")
    return c


def gemm_lds_bytes(cfg: TileConfig) -> int:
    return int(lib().gemm_lds_bytes(ctypes.byref(cfg)))


def gemm_status_string(status: int) -> str:
    return lib().gemm_status_string(status).decode()


def gemm_last_hip_error() -> str:
    return lib().gemm_last_hip_error().decode()


def gemm_wait_timeouts(reset: bool = False) -> int:
    """Bounded waits of the wave-specialized ring that gave up on the current device
    (synchronizes the device; reset clears the count after reading it)."""
    n = ctypes.c_uint32()
    _check(lib().gemm_wait_timeouts(ctypes.byref(n), 1 if reset else 0), "gemm_wait_timeouts")
    return int(n.value)


def gelu_run(x, y, n: int, dtype: str = "bf16", stream=None) -> None:
    """y[i] = gelu(x[i]) for n contiguous elements of dtype (include/spgelu.h)."""
    st = lib().gelu_run(_ptr(x), _ptr(y), n, DTYPES[dtype], _stream(stream, x, y))
    _check(st, "gelu_run")


# ---- the feed-forward operators --------------------------------------------------------

def gemm_gated_create(M: int, N: int, K: int, dtype: str = "bf16", layout: str = "nk",
                      act: str = "silu") -> int:
    h = ctypes.c_void_p()
    st = lib().gemm_gated_create(ctypes.byref(h), M, N, K, DTYPES[dtype], B_LAYOUTS[layout],
                                 ACTIVATIONS[act])
    _check(st, "gemm_gated_create")
    return int(h.value)


def gemm_gated_workspace(handle: int) -> int:
    return int(lib().gemm_gated_workspace(handle))


def gemm_gated_run_workspace(handle: int) -> int:
    return int(lib().gemm_gated_run_workspace(handle))


def gemm_gated_run(handle: int, X, Wg, Wu, H, G=None, U=None, workspace=None,
                   workspace_bytes: Optional[int] = None, stream=None) -> None:
    ws = _scratch("gemm_gated_run", workspace, workspace_bytes)
    st = lib().gemm_gated_run(handle, _ptr(X), _ptr(Wg), _ptr(Wu), _ptr(H), _ptr(G), _ptr(U),
                              *ws, _stream(stream, X, H))
    _check(st, "gemm_gated_run")


def gemm_gated_backward(handle: int, dH, X, Wg, Wu, G, U, dX, dWg, dWu, workspace=None,
                        workspace_bytes: Optional[int] = None, stream=None) -> None:
    ws = _scratch("gemm_gated_backward", workspace, workspace_bytes)
    st = lib().gemm_gated_backward(handle, _ptr(dH), _ptr(X), _ptr(Wg), _ptr(Wu), _ptr(G), _ptr(U),
                                   _ptr(dX), _ptr(dWg), _ptr(dWu), *ws, _stream(stream, dH, X, dX))
    _check(st, "gemm_gated_backward")


def gemm_gated_destroy(handle: Optional[int]) -> None:
    _check(lib().gemm_gated_destroy(handle), "gemm_gated_destroy")


def gemm_quantized_create(M: int, N: int, K: int, out_dtype: str = "bf16", act: str = "none") -> int:
    h = ctypes.c_void_p()
    st = lib().gemm_quantized_create(ctypes.byref(h), M, N, K, DTYPES[out_dtype], ACTIVATIONS[act])
    _check(st, "gemm_quantized_create")
    return int(h.value)


def gemm_quantized_workspace(handle: int) -> int:
    return int(lib().gemm_quantized_workspace(handle))


def gemm_quantized_run(handle: int, A, scale_a, B, scale_b, C, B2=None, scale_b2=None, workspace=None,
                       workspace_bytes: Optional[int] = None, stream=None) -> None:
    ws = _scratch("gemm_quantized_run", workspace, workspace_bytes)
    st = lib().gemm_quantized_run(handle, _ptr(A), _ptr(scale_a), _ptr(B), _ptr(scale_b), _ptr(B2),
                                  _ptr(scale_b2), _ptr(C), *ws, _stream(stream, A, C))
    _check(st, "gemm_quantized_run")


def gemm_quantized_destroy(handle: Optional[int]) -> None:
    _check(lib().gemm_quantized_destroy(handle), "gemm_quantized_destroy")


def gemm_quantize_rows(X, A, scale, stream=None, dtype: Optional[str] = None,
                       shape: Optional[tuple] = None) -> None:
    """Quantise the rows of X into A (int8) and scale (fp32).  For tensors the type and the
    [rows, K] shape are X's; with raw device pointers they are given."""
    calls = _calls_module()
    if calls is not None and dtype is None and shape is None:
        st = calls.rows(_address(lib().gemm_quantize_rows), X, A, scale, _raw(stream))
        if st >= 0:
            if st:
                _check(st, "gemm_quantize_rows")
            return
    if not isinstance(X, int) and X is not None:
        names, full = _torch_names(), X.shape
        if len(full) < 1 or X.dtype not in names or names[X.dtype] not in DTYPES:
            raise GemmError(1, f"gemm_quantize_rows: X is {X.dtype} of shape {tuple(full)}")
        device, (X_, A_, s_) = _dense("gemm_quantize_rows", ("X", X, X.dtype, full),
                                      ("A", A, _torch_type("i8"), full),
                                      ("scale", scale, _torch_type("f32"), full[:-1]))
        dtype, shape = names[X.dtype], (full[:-1].numel(), full[-1])
    else:
        if dtype is None or shape is None:
            raise GemmError(1, "gemm_quantize_rows: a raw X needs dtype and shape")
        rows, K = shape

        def any_shape(t, want):
            # tensors of any number of dimensions, as many values
            return t.shape if hasattr(t, "shape") and t.shape.numel() == math.prod(want) else want

        device, (A_, s_) = _dense("gemm_quantize_rows", ("A", A, _torch_type("i8"), any_shape(A, (rows, K))),
                                  ("scale", scale, _torch_type("f32"), any_shape(scale, (rows,))))
        X_ = X
    st = lib().gemm_quantize_rows(X_, DTYPES[dtype], shape[0], shape[1], A_, s_, _stream_on(stream, device))
    if st:
        _check(st, "gemm_quantize_rows")


def _scratch(what: str, workspace, given: Optional[int] = None, device: Optional[int] = None, raw: int = 0) -> tuple:
    """Pointer and bytes of a workspace.  A tensor has to be dense memory of the operands' GPU
    (`device`, where they tell): the kernels write as many bytes as its size promises.  A raw
    pointer without a given size has `raw` bytes: the plan's need, as raw operands have its shapes."""
    if workspace is None:
        return None, given or 0
    if isinstance(workspace, int):
        return workspace, raw if given is None else given
    if workspace.nbytes == 0 and not given:
        return None, 0
    if not workspace.is_contiguous():
        raise GemmError(1, f"{what}: workspace is not contiguous")
    if not workspace.is_cuda:
        raise GemmError(1, f"{what}: workspace is not on a GPU")
    if device is not None and workspace.get_device() != device:
        raise GemmError(1, f"{what}: workspace is on another device")
    if given is not None and given > workspace.nbytes:
        raise GemmError(1, f"{what}: workspace has {workspace.nbytes} bytes, not {given}")
    return workspace.data_ptr(), workspace.nbytes if given is None else given


_names = _types = None


def _torch_names():
    """torch dtype -> this library's name."""
    global _names, _types
    if _names is None:
        import torch
        _names = {torch.float16: "f16", torch.bfloat16: "bf16", torch.float32: "f32", torch.int8: "i8"}
        _types = {v: k for k, v in _names.items()}
    return _names


def _torch_type(name: str):
    """This library's name -> torch dtype (None without torch: raw pointers only)."""
    if _types is None:
        try:
            _torch_names()
        except ImportError:
            return None
    return _types[name]


def _refuse(what: str, tensors) -> None:
    """Raise for the first of (name, tensor, dtype, shape) that is not a dense GPU tensor of
    that type and shape on the first one's device."""
    device = None
    for name, t, dtype, shape in tensors:
        if t is None or isinstance(t, int):
            continue
        if t.shape != shape:
            raise GemmError(1, f"{what}: {name} has shape {tuple(t.shape)}, not {tuple(shape)}")
        if t.dtype is not dtype:
            raise GemmError(1, f"{what}: {name} is {t.dtype}, not {dtype}")
        if not t.is_contiguous():
            raise GemmError(1, f"{what}: {name} is not contiguous")
        if not t.is_cuda:
            raise GemmError(1, f"{what}: {name} is not on a GPU")
        if device is None:
            device = t.get_device()
        elif t.get_device() != device:
            raise GemmError(1, f"{what}: {name} is on another device")


def _dense(what: str, *tensors) -> tuple:
    """Check (name, tensor, dtype, shape) -- the kernels read dense memory of exactly that
    shape; raw device pointers and None pass -- and return the device index (None without a
    tensor) and the pointers.  Written for its cost: a call on one token is over in a few
    microseconds, and each attribute of a tensor takes a tenth of one to read."""
    device, ptrs = None, []
    for _, t, dtype, shape in tensors:
        if t is None or isinstance(t, int):
            ptrs.append(t)
            continue
        d = t.get_device()
        if device is None:
            device = d
        if d != device or d < 0 or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
            _refuse(what, tensors)
        ptrs.append(t.data_ptr())
    return device, ptrs


_calls = False


def _calls_module():
    """The compiled call path for torch tensors (csrc/binding.cpp): the checks of _dense and
    the call in one step, in a tenth of the time.  None where it is not built, or for a torch
    without the DLPack C exchange API: the Python path makes the same checks."""
    global _calls
    if _calls is False:
        _calls = None
        path = os.path.join(_HERE, "_calls.so")
        try:
            import torch
            api = getattr(torch.Tensor, "__dlpack_c_exchange_api__", None)
            if api is not None and os.path.exists(path):
                import importlib.machinery
                import importlib.util
                loader = importlib.machinery.ExtensionFileLoader("_calls", path)
                m = importlib.util.module_from_spec(importlib.util.spec_from_loader("_calls", loader))
                loader.exec_module(m)
                if m.setup(api, torch.Tensor, torch.nn.Parameter):
                    _calls = m
        except ImportError:
            pass
    return _calls


def _address(fn) -> int:
    """Address of a C entry point (kept with the function object)."""
    a = getattr(fn, "address", None)
    if a is None:
        a = fn.address = ctypes.cast(fn, ctypes.c_void_p).value
    return a


def _raw(stream):
    return stream if stream is None or isinstance(stream, int) else int(stream.cuda_stream)


def _specs(*tensors) -> bytes:
    """(dtype, shape) of each tensor of a call as csrc/binding.cpp reads them."""
    codes = {"f16": (2, 16), "bf16": (4, 16), "f32": (2, 32), "i8": (0, 8)}   # DLPack's
    out = b""
    for dtype, shape in tensors:
        code, bits = codes[dtype]
        out += struct.pack("4i2q", code, bits, len(shape), 0, *shape, *[0] * (2 - len(shape)))
    return out


_raw_stream = None


def _stream_on(stream, device: Optional[int]) -> Optional[int]:
    """The caller's stream, or the current one of `device`."""
    if stream is not None:
        return stream if isinstance(stream, int) else int(stream.cuda_stream)
    if device is None:
        return None
    global _raw_stream
    if _raw_stream is None:
        import torch
        # torch's own accessor of the handle where there is one: it makes no Stream object
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda d: int(torch.cuda.current_stream(d).cuda_stream))
    return _raw_stream(device)


class Gated:
    """The gated projection H = act(X Wg) * (X Wu) of a feed-forward block, and its backward
    pass (gemm_gated_* in include/spgemm.h).

    X [M,K]; Wg, Wu [N,K] ("nk") or [K,N] ("kn"); H, G, U [M,N].  Pass G and U to keep the
    pre-activations for ``backward``.  ``workspace`` is a uint8 tensor of at least
    ``workspace_bytes()``, or a raw pointer to that much memory; where only the projection is
    called, ``workspace_bytes(backward=False)`` is enough.  Calls in flight on different streams
    need one each."""

    def __init__(self, M, N, K, dtype="bf16", layout="nk", act="silu"):
        self.handle = 0
        self.M, self.N, self.K = M, N, K
        self.dtype, self.layout, self.act = dtype, layout, act
        self.handle = gemm_gated_create(M, N, K, dtype, layout, act)
        self._ws = gemm_gated_workspace(self.handle)
        self._ws_run = gemm_gated_run_workspace(self.handle)
        self._x, self._h = (M, K), (M, N)
        self._w = (N, K) if layout == "nk" else (K, N)
        self._run, self._back = lib().gemm_gated_run, lib().gemm_gated_backward
        self._type = _torch_type(dtype)
        x, w, h = ((dtype, s) for s in (self._x, self._w, self._h))
        self._calls = _calls_module()
        self._run_spec = _address(self._run), _specs(x, w, w, h, h, h)
        self._back_spec = _address(self._back), _specs(h, x, w, w, h, h, x, w, w)

    def workspace_bytes(self, backward: bool = True) -> int:
        """Bytes for the plan's calls; without ``backward`` for the projection alone."""
        return gemm_gated_workspace(self.handle) if backward else gemm_gated_run_workspace(self.handle)

    def __call__(self, X, Wg, Wu, H, G=None, U=None, workspace=None, stream=None):
        if self._calls is not None:
            fn, spec = self._run_spec
            st = self._calls.run(fn, self.handle, spec, (X, Wg, Wu, H, G, U), workspace, _raw(stream))
            if st >= 0:
                if st:
                    _check(st, "gemm_gated_run")
                return H
        d, x, w, h = self._type, self._x, self._w, self._h
        dev, p = _dense("Gated", ("X", X, d, x), ("Wg", Wg, d, w), ("Wu", Wu, d, w), ("H", H, d, h),
                        ("G", G, d, h), ("U", U, d, h))
        st = self._run(self.handle, *p, *_scratch("Gated", workspace, device=dev, raw=self._ws_run), _stream_on(stream, dev))
        if st:
            _check(st, "gemm_gated_run")
        return H

    def backward(self, dH, X, Wg, Wu, G, U, dX, dWg, dWu, workspace=None, stream=None):
        if self._calls is not None:
            fn, spec = self._back_spec
            st = self._calls.run(fn, self.handle, spec, (dH, X, Wg, Wu, G, U, dX, dWg, dWu), workspace, _raw(stream))
            if st >= 0:
                if st:
                    _check(st, "gemm_gated_backward")
                return dX, dWg, dWu
        d, x, w, h = self._type, self._x, self._w, self._h
        dev, p = _dense("Gated.backward", ("dH", dH, d, h), ("X", X, d, x), ("Wg", Wg, d, w),
                        ("Wu", Wu, d, w), ("G", G, d, h), ("U", U, d, h), ("dX", dX, d, x),
                        ("dWg", dWg, d, w), ("dWu", dWu, d, w))
        st = self._back(self.handle, *p, *_scratch("Gated.backward", workspace, device=dev, raw=self._ws), _stream_on(stream, dev))
        if st:
            _check(st, "gemm_gated_backward")
        return dX, dWg, dWu

    def close(self):
        if self.handle:
            gemm_gated_destroy(self.handle)
            self.handle = 0

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class QuantizedGemm:
    """C = (A B^T) scaled by row and by column, int8 operands (gemm_quantized_* in
    include/spgemm.h); with an activation C = act(C1) * C2 from B and B2.

    A [M,K] int8 with scale_a [M]; B, B2 [N,K] int8 with scale_b, scale_b2 [N]; C [M,N];
    ``workspace`` as in ``Gated``."""

    def __init__(self, M, N, K, out_dtype="bf16", act="none"):
        self.handle = 0
        self.M, self.N, self.K = M, N, K
        self.out_dtype, self.act = out_dtype, act
        self.handle = gemm_quantized_create(M, N, K, out_dtype, act)
        self._ws = gemm_quantized_workspace(self.handle)
        self._a, self._b, self._c, self._m, self._n = (M, K), (N, K), (M, N), (M,), (N,)
        self._run = lib().gemm_quantized_run
        self._calls = _calls_module()
        m, n, b = ("f32", self._m), ("f32", self._n), ("i8", self._b)
        self._run_spec = _address(self._run), _specs(("i8", self._a), m, b, n, b, n, (out_dtype, self._c))
        self._i8, self._f32, self._out = _torch_type("i8"), _torch_type("f32"), _torch_type(out_dtype)

    def workspace_bytes(self) -> int:
        return gemm_quantized_workspace(self.handle)

    def __call__(self, A, scale_a, B, scale_b, C, B2=None, scale_b2=None, workspace=None, stream=None):
        if self._calls is not None:
            fn, spec = self._run_spec
            st = self._calls.run(fn, self.handle, spec, (A, scale_a, B, scale_b, B2, scale_b2, C), workspace, _raw(stream))
            if st >= 0:
                if st:
                    _check(st, "gemm_quantized_run")
                return C
        i8, f32, m, n, b = self._i8, self._f32, self._m, self._n, self._b
        dev, p = _dense("QuantizedGemm", ("A", A, i8, self._a), ("scale_a", scale_a, f32, m), ("B", B, i8, b),
                        ("scale_b", scale_b, f32, n), ("B2", B2, i8, b), ("scale_b2", scale_b2, f32, n),
                        ("C", C, self._out, self._c))
        st = self._run(self.handle, *p, *_scratch("QuantizedGemm", workspace, device=dev, raw=self._ws), _stream_on(stream, dev))
        if st:
            _check(st, "gemm_quantized_run")
        return C

    def close(self):
        if self.handle:
            gemm_quantized_destroy(self.handle)
            self.handle = 0

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Gemm:
    """RAII wrapper around one plan: ``with Gemm(M, N, K, ...) as g: g(A, B, C)``."""

    def __init__(self, M, N, K, in_dtype="bf16", out_dtype="bf16", b_layout="kn",
                 epilogue="none", force: Optional[TileConfig] = None):
        self.M, self.N, self.K = M, N, K
        self.in_dtype, self.out_dtype, self.b_layout, self.epilogue = (
            in_dtype, out_dtype, b_layout, epilogue)
        self.handle = gemm_create(M, N, K, in_dtype, out_dtype, b_layout, epilogue, force)

    def __call__(self, A, B, C, stream=None):
        gemm_run(self.handle, A, B, C, stream)
        return C

    def config(self) -> TileConfig:
        return gemm_get_config(self.handle)

    def launch_config(self, A, B, C) -> TileConfig:
        return gemm_launch_config(self.handle, A, B, C)

    def autotune(self, A, B, C, stream=None, reps=10) -> float:
        return gemm_autotune(self.handle, A, B, C, stream, reps)

    def close(self):
        if self.handle:
            gemm_destroy(self.handle)
            self.handle = 0

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
