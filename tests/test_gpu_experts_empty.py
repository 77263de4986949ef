"""GPU tests of empty plans of the products by group that are given every pointer, as a program
with buffers of a fixed size does for an empty batch: the matrices' gradients are zeros, and
nothing else is written or read."""

import pytest

import software_pipelined_tiled_gemm_amd as spg
from tests.test_gpu_feed_forward import Buf, _dt, _t, _workspace

pytestmark = pytest.mark.gpu


# tiled, register-staged, odd addresses, without MFMAs, without columns
@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("size", [(64, 64, 0), (264, 136, 0), (77, 1001, 0), (72, 200, 1), (6, 5, 0), (0, 64, 0)], ids=str)
@pytest.mark.parametrize("tokens", [None, 0, 16])
def test_no_rows_and_a_source(size, layout, tokens):
    torch = _t()
    N, K, off = size
    E, dt = 4, _dt("bf16")
    shape = (E, N, K) if layout == "nk" else (E, K, N)
    w, dw, dwg, dwu = (Buf(shape, dt, off) for _ in range(4))
    w.t.zero_()
    spare = Buf((64, 1024), dt)                          # any rows, in and out
    source = torch.full((64,), 3, dtype=torch.int32, device="cuda")
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    p, s = spare.t.data_ptr(), source.data_ptr()
    torch.cuda.synchronize()                             # raw pointers run on the default stream
    with spg.GroupedGemm(0, N, K, E, "bf16", layout, tokens=tokens) as plan:
        ws = _workspace(plan.workspace_bytes())
        ws = ws if ws is None else ws.data_ptr()
        plan(p, w.t.data_ptr(), offsets.data_ptr(), p, source=s, workspace=ws)
        plan.backward(p, p, w.t.data_ptr(), offsets.data_ptr(), p, dw.t.data_ptr(), source=s, workspace=ws)
    with spg.GroupedGated(0, N, K, E, "bf16", layout, "silu", tokens=tokens) as plan:
        ws = _workspace(plan.workspace_bytes())
        ws = ws if ws is None else ws.data_ptr()
        q = w.t.data_ptr()
        plan(p, q, q, offsets.data_ptr(), p, source=s, G=p, U=p, workspace=ws)
        plan.backward(p, p, q, q, p, p, offsets.data_ptr(), p, dwg.t.data_ptr(), dwu.t.data_ptr(), source=s, workspace=ws)
    torch.cuda.synchronize()
    for b in (dw, dwg, dwu):
        assert bool((b.t == 0).all()) and b.intact()
    assert bool((spare.t.view(torch.int16) == 0x5A).all()) and spare.intact()
