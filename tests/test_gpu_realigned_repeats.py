"""GPU tests of every kernel that realigns 16-byte chunks in registers, over grids that fill the
device, many times: chunks that ended inside a row once came out wrong in some of a kernel's runs and
not in others.  The first run is held against the formulas, all later ones against its bits."""

import pytest

import software_pipelined_tiled_gemm_amd as spg
from tests.test_gpu_feed_forward import Buf, _as_kn, _check_backward, _check_forward, _dt, _gen, _normal, _t, _workspace
from tests.test_gpu_grouped import _check_rows, _check_weight, _source, _gathered, _weights

pytestmark = pytest.mark.gpu

TIMES = 12


def _equal(p, q):
    torch = _t()
    return all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(p, q))


# K that end at every element of a chunk; B stored [N,K], and [K,N] with as many odd rows
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K,layout,off", [(2048, 1100, 1001 + i, "nk", 0) for i in range(7)] +
                         [(2048, 1100, 1024, "nk", 1), (2048, 1101, 1000, "kn", 0), (1030, 2055, 777, "kn", 1)])
def test_gemm(M, N, K, layout, off, dtype):
    torch = _t()
    dt = _dt(dtype)
    a = Buf((M, K), dt, off, _normal(_gen(1), (M, K), 1.0).to(dt))
    shape = (N, K) if layout == "nk" else (K, N)
    b = Buf(shape, dt, off, _normal(_gen(2), shape, K ** -0.5).to(dt))
    c = torch.zeros(M, N, dtype=dt, device="cuda")
    with spg.Gemm(M, N, K, dtype, dtype, layout) as g:
        g(a.t, b.t, c)
        first = c.clone()
        _check_rows(a.t, _as_kn(b.t, layout), first, dtype, "C")
        for _ in range(TIMES):
            c.zero_()
            g(a.t, b.t, c)
            assert _equal([c], [first])


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K", [(300, 2731, 1001), (511, 1365, 500), (1, 4097, 1003), (1300, 2051, 1005)])
def test_gated(M, N, K, dtype, layout):
    torch = _t()
    dt = _dt(dtype)
    x, dh = _normal(_gen(1), (M, K), 1.0).to(dt), _normal(_gen(4), (M, N), 0.3).to(dt)
    shape = (N, K) if layout == "nk" else (K, N)
    wg, wu = (_normal(_gen(2 + i), shape, K ** -0.5).to(dt) for i in (0, 1))
    h, g, u = (torch.empty_like(dh) for _ in range(3))
    dx, dwg, dwu = torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)
    out = (h, g, u, dx, dwg, dwu)
    first = None
    with spg.Gated(M, N, K, dtype, layout, "silu") as plan:
        ws = _workspace(plan.workspace_bytes())
        for _ in range(1 + TIMES):
            for t in out:
                t.fill_(7)
            plan(x, wg, wu, h, G=g, U=u, workspace=ws)
            plan.backward(dh, x, wg, wu, g, u, dx, dwg, dwu, workspace=ws)
            if first is None:
                first = [t.clone() for t in out]
                _check_forward(x, wg, wu, h, g, u, dtype, layout, "silu")
                _check_backward(dh, x, wg, wu, g, u, dx, dwg, dwu, dtype, layout, "silu")
            assert _equal(out, first)


# streamed and tiled, rows in order and by their source, reductions that end inside chunks
@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("counts,N,K,tokens", [([32, 0] * 30, 1912, 54, None), ([5, 0, 1, 16] * 12, 1911, 331, 90), ([70, 3, 129, 64] * 4, 801, 1001, None),
                                               ([300, 41, 200], 1365, 203, 150), ([20] * 64, 1001, 49, None)])
def test_by_group(counts, N, K, tokens, layout):
    torch = _t()
    o = [sum(counts[:i]) for i in range(len(counts) + 1)]
    rows, E = o[-1], len(counts)
    offsets = torch.tensor(o, dtype=torch.int32, device="cuda")
    xr = rows if tokens is None else tokens
    x, dy = _normal(_gen(1), (xr, K), 1.0).bfloat16(), _normal(_gen(4), (rows, N), 0.3).bfloat16()
    source = None if tokens is None else _source(rows, tokens, 5)
    w = _weights(E, N, K, "bf16", layout, 2, 0).t
    y, dx, dw = torch.empty_like(dy), torch.empty(rows, K, dtype=torch.bfloat16, device="cuda"), torch.empty_like(w)
    out, first = (y, dx, dw), None
    with spg.GroupedGemm(rows, N, K, E, "bf16", layout, tokens=tokens) as plan:
        ws = _workspace(plan.workspace_bytes())
        for _ in range(1 + TIMES):
            for t in out:
                t.fill_(7)
            plan(x, w, offsets, y, source=source, workspace=ws)
            plan.backward(dy, x, w, offsets, dx, dw, source=source, workspace=ws)
            if first is None:
                first = [t.clone() for t in out]
                xs = _gathered(x, source)
                for e in range(0, E, max(1, E // 6)):
                    r = slice(o[e], o[e + 1])
                    if o[e] < o[e + 1]:
                        wd = _as_kn(w[e], layout)
                        _check_rows(xs[r], wd, y[r], "bf16", f"Y of group {e}")
                        _check_rows(dy[r], wd.t().contiguous(), dx[r], "bf16", f"dX of group {e}")
                        _check_weight(xs[r], dy[r], dw[e], "bf16", layout, f"dW of group {e}")
            assert _equal(out, first)
