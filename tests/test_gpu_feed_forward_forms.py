"""Every kernel that the feed-forward operators' choice of tiles can launch (the sizes of
tests/feed_forward_forms.py), against the formulas in 64 bits with the tolerances of
test_gpu_feed_forward.py, and bit for bit against the poisoned library, whose released ring
slots are NaN."""

import pytest

import software_pipelined_tiled_gemm_amd as spg
from tests import feed_forward_forms as listed
from tests.test_gpu_feed_forward import (SLOPE, U32, Buf, _act, _check_backward, _check_forward, _dt, _gated_case, _gen,
                                         _half_ulp, _ints, _normal, _t, _tiny, _within, _workspace)
from tests.test_gpu_feed_forward_poison import _both, _same

pytestmark = pytest.mark.gpu


def _types(cases):
    """fp16 and bf16 in turn."""
    return [(*c, ("bf16", "f16")[i % 2]) for i, c in enumerate(cases)]


@pytest.mark.parametrize("case", _types(listed.GATED), ids=str)
def test_projection(case, monkeypatch):
    torch = _t()
    M, N, K, nk, off, dtype = case
    layout = "nk" if nk else "kn"
    x, wg, wu = _gated_case(M, N, K, dtype, layout, 201, off // 2)

    def step():
        out = [Buf((M, N), _dt(dtype), off // 2) for _ in range(3)]
        with spg.Gated(M, N, K, dtype, layout, "silu") as plan:
            ws = _workspace(plan.workspace_bytes(backward=False))
            plan(x.t, wg.t, wu.t, out[0].t, G=out[1].t, U=out[2].t, workspace=ws)
        torch.cuda.synchronize()
        assert all(b.intact() for b in (x, wg, wu, *out))
        return [b.t for b in out]

    want, got = _both(step, monkeypatch)
    _check_forward(x.t, wg.t, wu.t, *want, dtype, layout, "silu")
    _same(want, got)


@pytest.mark.parametrize("case", _types(listed.BACKWARD), ids=str)
def test_gradients(case, monkeypatch):
    torch = _t()
    M, N, K, nk, off, dtype = case
    layout, dt = "nk" if nk else "kn", _dt(dtype)
    x, wg, wu = _gated_case(M, N, K, dtype, layout, 202, off // 2)
    gen = _gen(203)
    g, u, dh = (Buf((M, N), dt, off // 2, _normal(gen, (M, N), std).to(dt)) for std in (1.0, 1.0, 0.3))

    def step():
        out = [Buf(b.t.shape, dt, off // 2) for b in (x, wg, wu)]
        with spg.Gated(M, N, K, dtype, layout, "gelu_tanh") as plan:
            ws = _workspace(plan.workspace_bytes())
            plan.backward(dh.t, x.t, wg.t, wu.t, g.t, u.t, *(b.t for b in out), workspace=ws)
        torch.cuda.synchronize()
        assert all(b.intact() for b in (x, wg, wu, g, u, dh, *out))
        return [b.t for b in out]

    want, got = _both(step, monkeypatch)
    _check_backward(dh.t, x.t, wg.t, wu.t, g.t, u.t, *want, dtype, layout, "gelu_tanh")
    _same(want, got)


@pytest.mark.parametrize("case", listed.INT8, ids=str)
def test_int8_product(case, monkeypatch):
    torch = _t()
    M, N, K, gated, off = case
    act = "silu" if gated else "none"
    gen = _gen(204)
    a = Buf((M, K), torch.int8, off, _ints(gen, (M, K)))
    b = [Buf((N, K), torch.int8, off, _ints(gen, (N, K))) for _ in range(1 + gated)]
    sa = torch.empty(M, device="cuda").uniform_(0.5, 1.5, generator=gen)
    sb = [torch.empty(N, device="cuda").uniform_(0.5, 1.5, generator=gen) / (74.0 * 74.0 * K ** 0.5) for _ in b]

    def step():
        c = Buf((M, N), torch.float32)
        with spg.QuantizedGemm(M, N, K, "f32", act) as plan:
            ws = _workspace(plan.workspace_bytes())
            plan(a.t, sa, b[0].t, sb[0], c.t, B2=b[1].t if gated else None, scale_b2=sb[1] if gated else None, workspace=ws)
        torch.cuda.synchronize()
        assert all(t.intact() for t in (a, c, *b))
        return [c.t]

    want, got = _both(step, monkeypatch)
    # three roundings of the sums to scaled fp32 (test_quantized_product), then the gate's
    p = [(a.t.double() @ w.t.double().t()) * sa.double()[:, None] * s.double() for w, s in zip(b, sb)]
    e, tiny = _half_ulp("f32"), _tiny("f32")
    if not gated:
        value, tol = p[0], (e + 3.01 * U32) * p[0].abs() + tiny
    else:
        A = _act(p[0], act)
        value = A * p[1]
        tol = (e * value.abs() + SLOPE * 3.01 * U32 * p[0].abs() * p[1].abs() * 1.01
               + 4.02 * U32 * value.abs() + 2.0 ** -20 * p[0].abs() * p[1].abs() + tiny)
    _within(want[0], value, tol, f"C {act}")
    _same(want, got)
