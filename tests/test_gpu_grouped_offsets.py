"""GPU tests of the products by group on offsets that no routing makes: outside the rows, falling,
overlapping.  Offsets count as the nearest that there is and a group that ends before it starts is
empty; where groups overlap no result is specified, and nothing outside the operands may change."""

import pytest

import software_pipelined_tiled_gemm_amd as spg
from tests.test_gpu_feed_forward import Buf, _as_kn, _dt, _gen, _normal, _t, _workspace
from tests.test_gpu_grouped import _check_rows, _check_weight, _weights

pytestmark = pytest.mark.gpu

LOW, HIGH = -2 ** 31, 2 ** 31 - 1
# rows, offsets
APART = {
    "outside": (300, [-5, 130, HIGH, HIGH]),
    "below": (300, [LOW, -1, 0, 77]),
    "falling": (300, [200, 100, 40, 260]),
    "beyond": (300, [301, 5000, HIGH, HIGH]),
    "single": (3, [LOW, 1, 2, HIGH]),
}
OVERLAPPING = {
    "twice": (300, [0, 300, 0, 300]),
    "in turn": (300, [0, 300] * 40),
    "mixed": (300, [HIGH, LOW, 200, 50, 260, -3, 299]),
    "many": (700, [0, 700] * 400),
    "few rows": (5, [0, 5] * 30),
}
# streamed, tiled, register-staged, reductions in parts, without MFMAs
SIZES = [(48, 64), (264, 512), (131, 77), (96, 4200), (4200, 96), (6, 5)]


def _run(rows, o, N, K, layout, tokens):
    torch = _t()
    E, dt = len(o) - 1, _dt("bf16")
    offsets = torch.tensor(o, dtype=torch.int32, device="cuda")
    xr = rows if tokens is None else tokens
    x = Buf((xr, K), dt, 0, _normal(_gen(1), (xr, K), 1.0).to(dt))
    w = [_weights(E, N, K, "bf16", layout, 2 + i, 0) for i in (0, 1)]
    dy = Buf((rows, N), dt, 0, _normal(_gen(4), (rows, N), 0.3).to(dt))
    source = None if tokens is None else torch.randint(0, tokens, (rows,), generator=_gen(5), device="cuda").int()
    y, h, g, u = (Buf((rows, N), dt) for _ in range(4))
    dx, dx1 = (Buf((rows, K), dt) for _ in range(2))
    dw, dwg, dwu = (Buf(w[0].t.shape, dt) for _ in range(3))
    with spg.GroupedGemm(rows, N, K, E, "bf16", layout, tokens=tokens) as plan:
        ws = Buf((max(1, plan.workspace_bytes()),), torch.uint8)
        plan(x.t, w[0].t, offsets, y.t, source=source, workspace=ws.t)
        plan.backward(dy.t, x.t, w[0].t, offsets, dx.t, dw.t, source=source, workspace=ws.t)
    with spg.GroupedGated(rows, N, K, E, "bf16", layout, "silu", tokens=tokens) as plan:
        ws1 = Buf((max(1, plan.workspace_bytes()),), torch.uint8)
        plan(x.t, w[0].t, w[1].t, offsets, h.t, source=source, G=g.t, U=u.t, workspace=ws1.t)
        plan.backward(dy.t, x.t, w[0].t, w[1].t, g.t, u.t, offsets, dx1.t, dwg.t, dwu.t, source=source, workspace=ws1.t)
    torch.cuda.synchronize()
    assert all(b.intact() for b in (x, dy, y, h, g, u, dx, dx1, dw, dwg, dwu, ws, ws1, *w))
    xs = x.t if source is None else x.t[source.long()]
    return xs, w[0].t, dy.t, y.t, dx.t, dw.t


@pytest.mark.parametrize("tokens", [None, 37])
@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("kind", list(APART))
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_apart(size, kind, layout, tokens):
    torch = _t()
    rows, o = APART[kind]
    xs, w, dy, y, dx, dw = _run(rows, o, *size, layout, tokens)
    inside = [min(max(v, 0), rows) for v in o]
    written = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for e, (a, b) in enumerate(zip(inside, inside[1:])):
        if a >= b:
            assert bool((dw[e] == 0).all())
            continue
        written[a:b] = True
        wd = _as_kn(w[e], layout)
        _check_rows(xs[a:b], wd, y[a:b], "bf16", f"Y of group {e}")
        _check_rows(dy[a:b], wd.t().contiguous(), dx[a:b], "bf16", f"dX of group {e}")
        _check_weight(xs[a:b], dy[a:b], dw[e], "bf16", layout, f"dW of group {e}")
    for t in (y, dx):
        assert bool((t.view(torch.int16)[~written] == 0x5A).all())


@pytest.mark.parametrize("tokens", [None, 37])
@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("kind", list(OVERLAPPING))
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_overlapping(size, kind, layout, tokens):
    # a matrix's gradient is its own group's: it does not depend on the others
    rows, o = OVERLAPPING[kind]
    if len(o) > 100 and size[0] * size[1] > 50000:
        size = (72, 200)
    xs, w, dy, y, dx, dw = _run(rows, o, *size, layout, tokens)
    inside = [min(max(v, 0), rows) for v in o]
    for e in {0, 1, len(o) // 2, len(o) - 2}:
        a, b = inside[e], inside[e + 1]
        if a >= b:
            assert bool((dw[e] == 0).all())
        else:
            _check_weight(xs[a:b], dy[a:b], dw[e], "bf16", layout, f"dW of group {e}")
