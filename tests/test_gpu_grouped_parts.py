"""GPU tests of the products by group on few tiles with long reductions, which are split over the
CUs and joined: every small tile, both layouts and alignments, reductions that end inside a k-tile
and inside a 16-byte chunk, rows by their source, forward, input and matrix gradients.  Formulas and
tolerances of test_gpu_grouped.py; parts are sums in fp32 like any other order of them."""

import pytest

import software_pipelined_tiled_gemm_amd as spg
from tests.test_gpu_feed_forward import Buf, _as_kn, _check_backward, _dt, _gen, _normal, _t, _workspace
from tests.test_gpu_grouped import _check_rows, _check_weight, _gathered, _source, _weights, run_gated, run_plain

pytestmark = pytest.mark.gpu

# (N, K): the forward pass's reduction is K, the input gradient's N
SIZES = [(96, 4200), (89, 3001), (40, 6000), (520, 2056), (4200, 96), (3001, 89), (8, 12288), (2056, 2050)]


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("kind", ["one", "single", "few", "tile", "ragged", "skewed", "empty"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_plain(size, kind, layout):
    run_plain(kind, *size, "bf16", layout, 0, None, 200)
    run_plain(kind, *size, "f16", layout, 1, 37, 210)


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("kind", ["one", "few", "tile", "skewed"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_gated(size, kind, layout):
    run_gated(kind, *size, "bf16", layout, "silu", 0, 50, True, 220)
    run_gated(kind, *size, "f16", layout, "gelu_tanh", 1, None, True, 230)


# rows of the groups, N, K: few small matrices and many rows, whose gradients are split along the
# rows; groups of fewer k-tiles than parts, of none, odd sizes
ROWS = [([3000, 0, 1700, 5], 72, 136), ([9000], 64, 200), ([4100, 2500], 33, 65), ([2049, 64, 5000, 1, 0, 3000], 130, 64),
        ([7000, 20], 264, 72), ([4160] * 3, 200, 8)]


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("case", ROWS, ids=str)
def test_gradients_of_many_rows(case, layout):
    counts, N, K = case
    o = [3 + sum(counts[:i]) for i in range(len(counts) + 1)]
    rows, E = o[-1] + 2, len(counts)
    torch = _t()
    offsets = torch.tensor(o, dtype=torch.int32, device="cuda")
    for dtype, off, tokens in (("bf16", 0, 500), ("f16", 1, None)):
        dt = _dt(dtype)
        xr = rows if tokens is None else tokens
        x = Buf((xr, K), dt, off, _normal(_gen(1), (xr, K), 1.0).to(dt))
        w = [_weights(E, N, K, dtype, layout, 2 + i, off) for i in (0, 1)]
        dh = Buf((rows, N), dt, off, _normal(_gen(4), (rows, N), 0.3).to(dt))
        source = None if tokens is None else _source(rows, tokens, 5)
        h, g, u, dx, dx1 = (Buf((rows, n), dt, off) for n in (N, N, N, K, K))
        dwg, dwu, dw, again = (Buf(w[0].t.shape, dt, off) for _ in range(4))
        with spg.GroupedGated(rows, N, K, E, dtype, layout, "silu", tokens=tokens) as plan:
            ws = _workspace(plan.workspace_bytes())
            plan(x.t, w[0].t, w[1].t, offsets, h.t, source=source, G=g.t, U=u.t, workspace=ws)
            plan.backward(dh.t, x.t, w[0].t, w[1].t, g.t, u.t, offsets, dx.t, dwg.t, dwu.t, source=source, workspace=ws)
        with spg.GroupedGemm(rows, N, K, E, dtype, layout, tokens=tokens) as plan:
            ws = _workspace(plan.workspace_bytes())
            plan.backward(dh.t, x.t, w[0].t, offsets, dx1.t, dw.t, source=source, workspace=ws)
            plan.backward(dh.t, x.t, w[0].t, offsets, None, again.t, source=source, workspace=ws)
        torch.cuda.synchronize()
        xs = _gathered(x.t, source)
        for e in range(E):
            r = slice(o[e], o[e + 1])
            if o[e] == o[e + 1]:
                assert all(bool((b.t[e] == 0).all()) for b in (dwg, dwu, dw, again))
                continue
            _check_backward(dh.t[r], xs[r], w[0].t[e], w[1].t[e], g.t[r], u.t[r], dx.t[r], dwg.t[e], dwu.t[e], dtype, layout, "silu")
            _check_weight(xs[r], dh.t[r], dw.t[e], dtype, layout, f"dW of group {e}")
            _check_weight(xs[r], dh.t[r], again.t[e], dtype, layout, f"dW alone of group {e}")
            _check_rows(dh.t[r], _as_kn(w[0].t[e], layout).t().contiguous(), dx1.t[r], dtype, f"dX of group {e}")
        assert all(b.intact() for b in (x, dh, h, g, u, dx, dx1, dwg, dwu, dw, again, *w))
