"""GPU tests of the gated projection's gradients by group against differences of the loss and its
autograd, in 64 bits, with tolerances that a halved, negated or incomplete gradient does not meet
(tests/test_grouped_gradients_check.py plants those)."""

import pytest

import software_pipelined_tiled_gemm_amd as spg
from tests import grouped_gradients
from tests.test_gpu_feed_forward import _dt, _gen, _half_ulp, _normal, _t, _workspace
from tests.test_gpu_grouped import GROUPS, _offsets, _weights

pytestmark = pytest.mark.gpu


def _kn(w, layout):
    return (w.transpose(1, 2) if layout == "nk" else w).double().contiguous()


# streamed and tiled, one k-tile and several, odd, without MFMAs
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("kind,N,K,tokens", [("few", 40, 48, None), ("few", 130, 77, 30), ("ragged", 72, 200, None), ("ragged", 264, 136, 90),
                                             ("single", 96, 1536, 5), ("few", 5, 6, None)])
def test_gated(kind, N, K, tokens, layout, act, dtype):
    torch = _t()
    o, rows, offsets = _offsets(kind)
    E, dt = len(GROUPS[kind][1]), _dt(dtype)
    x = _normal(_gen(1), (rows if tokens is None else tokens, K), 1.0).to(dt)
    source = None if tokens is None else torch.randint(0, tokens, (rows,), generator=_gen(5), device="cuda").int()
    wg, wu = (_weights(E, N, K, dtype, layout, 2 + i, 0).t for i in (0, 1))
    dh = _normal(_gen(4), (rows, N), 0.3).to(dt)
    h, g, u = (torch.zeros(rows, N, device="cuda", dtype=dt) for _ in range(3))
    dx, dwg, dwu = torch.zeros(rows, K, device="cuda", dtype=dt), torch.full_like(wg, 7), torch.full_like(wu, 7)
    with spg.GroupedGated(rows, N, K, E, dtype, layout, act, tokens=tokens) as plan:
        ws = _workspace(plan.workspace_bytes())
        plan(x, wg, wu, offsets, h, source=source, G=g, U=u, workspace=ws)
        plan.backward(dh, x, wg, wu, g, u, offsets, dx, dwg, dwu, source=source, workspace=ws)
    xs = (x if source is None else x[source.long()]).double()
    grouped_gradients.check((dx, _kn(dwg, layout), _kn(dwu, layout)), xs, _kn(wg, layout), _kn(wu, layout), dh.double(), o, act,
                            _half_ulp(dtype))
