"""GPU tests of the products by group, plain and gated, against plain formulas in 64 bits, group
by group.  Tolerances as in test_gpu_feed_forward.py: a sum of K products in fp32 in any order is
off by at most K 2^-24 S, S the sum of the products' magnitudes; each result is rounded once more;
the gated ones' share is that file's."""

import pytest

import software_pipelined_tiled_gemm_amd as spg
from tests.test_gpu_feed_forward import (U32, Buf, _as_kn, _check_backward, _check_forward, _dt, _gen, _half_ulp, _normal, _t,
                                         _tiny, _within, _workspace)

pytestmark = pytest.mark.gpu

# rows of each group; the first and the last number are rows in front of and behind the groups
GROUPS = {
    "one": (0, [1], 0),
    "single": (0, [1, 0, 1, 1], 3),
    "few": (2, [0, 3, 16, 17, 0, 1], 5),
    "tile": (0, [64, 65, 63, 128], 0),
    "ragged": (5, [130, 0, 1, 257, 77, 0], 40),
    "many": (0, [i % 7 for i in range(130)], 9),
    "skewed": (0, [0, 900, 3, 0, 0, 41], 0),
    "long": (0, [513, 700, 300], 1),
    "empty": (3, [0, 0, 0], 4),
    "thousand": (1, [1 if i % 5 == 0 else 0 for i in range(1000)], 2),
}
# (N, K): narrow, odd, one k-tile, many, rows on words and off them, shorter than a 16-byte chunk
SIZES = [(48, 40), (130, 64), (72, 200), (33, 9), (7, 3), (264, 512), (257, 320), (500, 1365), (64, 2048), (96, 1536), (520, 196),
         (1024, 78)]


def _offsets(kind):
    torch = _t()
    front, counts, behind = GROUPS[kind]
    o = [front]
    for n in counts:
        o.append(o[-1] + n)
    return o, o[-1] + behind, torch.tensor(o, dtype=torch.int32, device="cuda")


def _weights(E, N, K, dtype, layout, seed, off):
    shape = (E, N, K) if layout == "nk" else (E, K, N)
    return Buf(shape, _dt(dtype), off, _normal(_gen(seed), shape, max(K, 1) ** -0.5).to(_dt(dtype)))


def _source(rows, tokens, seed):
    """Rows of X in any order, some read often, a few out of range (rows of zeros)."""
    torch = _t()
    s = torch.randint(0, tokens, (rows,), generator=_gen(seed), device="cuda").int()
    if rows > 4:
        s[rows // 2], s[rows // 3] = -1, tokens
    return s


def _gathered(x, source):
    if source is None:
        return x
    ok = (source >= 0) & (source < x.shape[0])
    return x[source.clamp(0, x.shape[0] - 1).long()] * ok[:, None]


def _outside(t, offsets):
    """Rows in front of the first group and behind the last."""
    return t[: offsets[0]], t[offsets[-1]:]


def _untouched(b, offsets):
    torch = _t()
    raw = b.t.view(torch.int16)
    return all(bool((part == 0x5A).all()) for part in _outside(raw, offsets))


def _check_rows(x, w, y, dtype, what):
    """y = x w, w as [K,N] in 64 bits."""
    K = x.shape[1]
    xd = x.double()
    want = xd @ w
    tol = _half_ulp(dtype) * want.abs() + 1.01 * K * U32 * (xd.abs() @ w.abs()) + _tiny(dtype)
    _within(y, want, tol, what)


def _check_weight(x, dy, dw, dtype, layout, what):
    xd, dd = x.double(), dy.double()
    want = xd.t() @ dd
    tol = _half_ulp(dtype) * want.abs() + 1.01 * x.shape[0] * U32 * (xd.abs().t() @ dd.abs()) + _tiny(dtype)
    if layout == "nk":
        want, tol = want.t(), tol.t()
    _within(dw, want, tol, what)


def run_plain(kind, N, K, dtype, layout, off, tokens, seed):
    torch = _t()
    o, rows, offsets = _offsets(kind)
    E = len(o) - 1
    dt = _dt(dtype)
    x = Buf((rows if tokens is None else tokens, K), dt, off, _normal(_gen(seed), (rows if tokens is None else tokens, K), 1.0).to(dt))
    w = _weights(E, N, K, dtype, layout, seed + 1, off)
    dy = Buf((rows, N), dt, off, _normal(_gen(seed + 2), (rows, N), 0.3).to(dt))
    source = None if tokens is None else _source(rows, tokens, seed + 3)
    for part in _outside(dy.t, o) + (_outside(x.t, o) if source is None else ()):
        part.fill_(float("nan"))                             # not read
    y, dx, dw = Buf((rows, N), dt, off), Buf((rows, K), dt, off), Buf(w.t.shape, dt, off)
    with spg.GroupedGemm(rows, N, K, E, dtype, layout, tokens=tokens) as plan:
        plan(x.t, w.t, offsets, y.t, source=source, workspace=_workspace(plan.workspace_bytes(backward=False)))
        plan.backward(dy.t, x.t, w.t, offsets, dx.t, dw.t, source=source, workspace=_workspace(plan.workspace_bytes()))
    torch.cuda.synchronize()
    xs = _gathered(x.t, source)
    for e in range(E):
        r = slice(o[e], o[e + 1])
        if o[e] == o[e + 1]:
            continue
        wd = _as_kn(w.t[e], layout)
        _check_rows(xs[r], wd, y.t[r], dtype, f"Y of group {e}")
        _check_rows(dy.t[r], wd.t().contiguous(), dx.t[r], dtype, f"dX of group {e}")
        _check_weight(xs[r], dy.t[r], dw.t[e], dtype, layout, f"dW of group {e}")
    empty = [e for e in range(E) if o[e] == o[e + 1]]
    assert bool((dw.t[empty] == 0).all())
    assert _untouched(y, o) and _untouched(dx, o)
    assert all(b.intact() for b in (x, w, dy, y, dx, dw))


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("kind", list(GROUPS))
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_plain(size, kind, layout):
    N, K = size
    if kind == "thousand" and N * K > 50000:
        N, K = 72, 200
    run_plain(kind, N, K, "bf16", layout, 0, None, 100)
    run_plain(kind, N, K, "f16", layout, 0, 37, 110)
    run_plain(kind, N, K, "f16", layout, 1, None, 120)
    run_plain(kind, N, K, "bf16", layout, 2, 900, 130)


def run_gated(kind, N, K, dtype, layout, act, off, tokens, keep, seed):
    torch = _t()
    o, rows, offsets = _offsets(kind)
    E = len(o) - 1
    dt = _dt(dtype)
    x = Buf((rows if tokens is None else tokens, K), dt, off, _normal(_gen(seed), (rows if tokens is None else tokens, K), 1.0).to(dt))
    wg, wu = (_weights(E, N, K, dtype, layout, seed + 1 + i, off) for i in (0, 1))
    dh = Buf((rows, N), dt, off, _normal(_gen(seed + 3), (rows, N), 0.3).to(dt))
    source = None if tokens is None else _source(rows, tokens, seed + 4)
    for part in _outside(dh.t, o) + (_outside(x.t, o) if source is None else ()):
        part.fill_(float("nan"))
    h, g, u, dx = (Buf((rows, n), dt, off) for n in (N, N, N, K))
    dwg, dwu = Buf(wg.t.shape, dt, off), Buf(wg.t.shape, dt, off)
    with spg.GroupedGated(rows, N, K, E, dtype, layout, act, tokens=tokens) as plan:
        plan(x.t, wg.t, wu.t, offsets, h.t, source=source, G=g.t if keep else None, U=u.t if keep else None,
             workspace=_workspace(plan.workspace_bytes(backward=False)))
        if keep:
            plan.backward(dh.t, x.t, wg.t, wu.t, g.t, u.t, offsets, dx.t, dwg.t, dwu.t, source=source,
                          workspace=_workspace(plan.workspace_bytes()))
    torch.cuda.synchronize()
    xs = _gathered(x.t, source)
    for e in range(E):
        r = slice(o[e], o[e + 1])
        if o[e] == o[e + 1]:
            continue
        _check_forward(xs[r], wg.t[e], wu.t[e], h.t[r], g.t[r] if keep else None, u.t[r], dtype, layout, act)
        if keep:
            _check_backward(dh.t[r], xs[r], wg.t[e], wu.t[e], g.t[r], u.t[r], dx.t[r], dwg.t[e], dwu.t[e], dtype, layout, act)
    if keep:
        empty = [e for e in range(E) if o[e] == o[e + 1]]
        assert bool((dwg.t[empty] == 0).all()) and bool((dwu.t[empty] == 0).all())
    assert all(_untouched(b, o) for b in (h, g, u, dx))
    assert all(b.intact() for b in (x, wg, wu, dh, h, g, u, dx, dwg, dwu))


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("kind", list(GROUPS))
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_gated(size, kind, layout):
    N, K = size
    if kind == "thousand" and N * K > 50000:
        N, K = 72, 200
    run_gated(kind, N, K, "bf16", layout, "silu", 0, 37, True, 200)
    run_gated(kind, N, K, "f16", layout, "gelu_tanh", 0, None, True, 210)
    run_gated(kind, N, K, "bf16", layout, "relu", 1, None, True, 220)
    run_gated(kind, N, K, "f16", layout, "silu", 2, 900, False, 230)


@pytest.mark.parametrize("layout", ["nk", "kn"])
def test_offsets_outside_the_rows(layout):
    # they count as the nearest end; a group that would end before it starts is empty
    torch = _t()
    rows, N, K, E = 50, 72, 136, 5
    x = _normal(_gen(1), (rows, K), 1.0).bfloat16()
    w = _weights(E, N, K, "bf16", layout, 2, 0).t
    bad = torch.tensor([-9, 20, 20, 30, 1 << 30, 40], dtype=torch.int32, device="cuda")
    good = [(0, 20), (20, 20), (20, 30), (30, 50), (50, 50)]
    for gated in (False, True):
        y = Buf((rows, N), torch.bfloat16)
        if gated:
            with spg.GroupedGated(rows, N, K, E, "bf16", layout, "silu") as plan:
                plan(x, w, w, bad, y.t, workspace=_workspace(plan.workspace_bytes()))
        else:
            with spg.GroupedGemm(rows, N, K, E, "bf16", layout) as plan:
                plan(x, w, bad, y.t, workspace=_workspace(plan.workspace_bytes()))
        torch.cuda.synchronize()
        assert y.intact()
        for e, (a, b) in enumerate(good):
            if a == b:
                continue
            if gated:
                _check_forward(x[a:b], w[e], w[e], y.t[a:b], None, None, "bf16", layout, "silu")
            else:
                _check_rows(x[a:b], _as_kn(w[e], layout), y.t[a:b], "bf16", f"group {e}")
    dw = Buf(w.shape, torch.bfloat16)
    dy = _normal(_gen(3), (rows, N), 0.3).bfloat16()
    dx = torch.empty_like(x)
    with spg.GroupedGemm(rows, N, K, E, "bf16", layout) as plan:
        plan.backward(dy, x, w, bad, dx, dw.t, workspace=_workspace(plan.workspace_bytes()))
    torch.cuda.synchronize()
    assert dw.intact()
    for e, (a, b) in enumerate(good):
        _check_weight(x[a:b], dy[a:b], dw.t[e], "bf16", layout, f"dW of group {e}")


def test_either_gradient_alone_and_nothing_to_do():
    torch = _t()
    o, rows, offsets = _offsets("ragged")
    N, K, E = 72, 136, len(o) - 1
    dt = torch.bfloat16
    x, dy = _normal(_gen(1), (rows, K), 1.0).to(dt), _normal(_gen(2), (rows, N), 0.3).to(dt)
    w = _weights(E, N, K, "bf16", "nk", 3, 0).t
    with spg.GroupedGemm(rows, N, K, E, "bf16", "nk") as plan:
        ws = _workspace(plan.workspace_bytes())
        both = torch.zeros_like(x), torch.zeros_like(w)
        alone = torch.zeros_like(x), torch.zeros_like(w)
        plan.backward(dy, x, w, offsets, *both, workspace=ws)
        plan.backward(dy, None, w, offsets, alone[0], None, workspace=ws)
        plan.backward(dy, x, None, offsets, None, alone[1], workspace=ws)
        # one launch or two: the tiles may differ and with them the order of a sum, so each result
        # is held to the formula (both orders are within its tolerance) and not to the other's bits
        for dx, dw in (both, alone):
            for e in range(E):
                r = slice(o[e], o[e + 1])
                _check_rows(dy[r], _as_kn(w[e], "nk").t().contiguous(), dx[r], "bf16", f"dX of group {e}")
                _check_weight(x[r], dy[r], dw[e], "bf16", "nk", f"dW of group {e}")
    # no rows: the weights' gradients are zero; K = 0: products of nothing are zero
    none = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    for Z in (spg.GroupedGemm(0, N, K, E), spg.GroupedGated(0, N, K, E)):
        with Z as plan:
            ex, ey = torch.empty(0, K, device="cuda", dtype=dt), torch.empty(0, N, device="cuda", dtype=dt)
            d = [torch.full_like(w, 5.0) for _ in range(2)]
            if isinstance(plan, spg.GroupedGemm):
                plan(ex, w, none, ey)
                plan.backward(ey, ex, w, none, ex, d[0])
                d[1].zero_()
            else:
                plan(ex, w, w, none, ey)
                plan.backward(ey, ex, w, w, ey, ey, none, ex, *d)
            assert all(bool((v == 0).all()) for v in d)
    y = torch.full((rows, N), 3.0, device="cuda", dtype=dt)
    with spg.GroupedGemm(rows, N, 0, E) as plan:
        plan(torch.empty(rows, 0, device="cuda", dtype=dt), torch.empty(E, N, 0, device="cuda", dtype=dt), offsets, y)
    assert bool((y[o[0]:o[-1]] == 0).all()) and bool((y[:o[0]] == 3).all()) and bool((y[o[-1]:] == 3).all())


@pytest.mark.parametrize("layout", ["nk", "kn"])
def test_infinities_stay_in_their_group(layout):
    # neighbouring rows and matrices hold what would spoil a product that reads past its own
    torch = _t()
    for N, K in ((72, 136), (40, 1001), (130, 70)):
        o, rows, offsets = _offsets("ragged")
        E = len(o) - 1
        x = _normal(_gen(1), (rows, K), 1.0).half()
        w = _weights(E, N, K, "f16", layout, 2, 0).t
        dy = _normal(_gen(3), (rows, N), 0.3).half()
        bad = 3                                              # of 257 rows
        r = slice(o[bad], o[bad + 1])
        x[r], w[bad], dy[r] = float("inf"), float("nan"), float("nan")
        y, dx, dw = torch.zeros(rows, N, device="cuda").half(), torch.zeros_like(x), torch.zeros_like(w)
        with spg.GroupedGemm(rows, N, K, E, "f16", layout) as plan:
            ws = _workspace(plan.workspace_bytes())
            plan(x, w, offsets, y, workspace=ws)
            plan.backward(dy, x, w, offsets, dx, dw, workspace=ws)
        for t in (y, dx):
            assert bool(torch.isfinite(t[: o[bad]]).all()) and bool(torch.isfinite(t[o[bad + 1]:]).all()), (N, K)
            assert bool(torch.isnan(t[r]).all())
        fine = [e for e in range(E) if e != bad]
        assert bool(torch.isfinite(dw[fine]).all()) and bool(torch.isnan(dw[bad]).all())


@pytest.mark.parametrize("layout", ["nk", "kn"])
def test_gradients_against_differences(layout):
    # the plain product is linear in X and in W, so a difference of any step is exact; the gated
    # one's central difference, in 64 bits, is off by h^2 / 6 of the third derivative
    torch = _t()
    o, rows, offsets = _offsets("few")
    N, K, E, h = 40, 48, len(o) - 1, 1e-3
    x = _normal(_gen(1), (rows, K), 1.0).half()
    wg, wu = (_weights(E, N, K, "f16", layout, 2 + i, 0).t for i in (0, 1))
    dh = _normal(_gen(4), (rows, N), 0.3).half()
    hh, g, u = (torch.zeros(rows, N, device="cuda", dtype=torch.float16) for _ in range(3))
    dx, dwg, dwu = torch.zeros_like(x), torch.zeros_like(wg), torch.zeros_like(wu)
    with spg.GroupedGated(rows, N, K, E, "f16", layout, "silu") as plan:
        ws = _workspace(plan.workspace_bytes())
        plan(x, wg, wu, offsets, hh, G=g, U=u, workspace=ws)
        plan.backward(dh, x, wg, wu, g, u, offsets, dx, dwg, dwu, workspace=ws)

    def loss(x, wg, wu):
        s = 0.0
        for e in range(E):
            r = slice(o[e], o[e + 1])
            a, b = x[r] @ _as_kn(wg[e], layout), x[r] @ _as_kn(wu[e], layout)
            s = s + (dh[r].double() * a * torch.sigmoid(a) * b).sum()
        return s

    for grad, which in ((dx, 0), (dwg, 1), (dwu, 2)):
        for i in range(3):
            d = _normal(_gen(10 + i), grad.shape, 1.0).double()
            hi, lo = [v.double() for v in (x, wg, wu)], [v.double() for v in (x, wg, wu)]
            hi[which], lo[which] = hi[which] + h * d, lo[which] - h * d
            want = float((loss(*hi) - loss(*lo)) / (2 * h))
            got = float((grad.double() * d).sum())
            # G, U, dG, dU and the gradient rounded to fp16: 5 half ulps of each product's terms,
            # whose magnitudes are below 16 times the gradient's
            tol = 80 * _half_ulp("f16") * float((grad.double().abs() * d.abs()).sum()) + 1e-3
            assert abs(got - want) <= tol, (which, got, want, tol)


@pytest.mark.parametrize("layout", ["nk", "kn"])
def test_results_repeat(layout):
    torch = _t()
    o, rows, offsets = _offsets("long")
    N, K, E = 520, 776, len(o) - 1
    x = _normal(_gen(1), (rows, K), 1.0).bfloat16()
    wg, wu = (_weights(E, N, K, "bf16", layout, 2 + i, 0).t for i in (0, 1))
    dh = _normal(_gen(4), (rows, N), 0.3).bfloat16()
    seen = []
    with spg.GroupedGated(rows, N, K, E, "bf16", layout, "silu") as plan:
        for _ in range(3):
            h, g, u = (torch.zeros(rows, N, device="cuda", dtype=torch.bfloat16) for _ in range(3))
            dx, dwg, dwu = torch.zeros_like(x), torch.zeros_like(wg), torch.zeros_like(wu)
            ws = _workspace(plan.workspace_bytes())
            plan(x, wg, wu, offsets, h, G=g, U=u, workspace=ws)
            plan.backward(dh, x, wg, wu, g, u, offsets, dx, dwg, dwu, workspace=ws)
            seen.append((h, g, u, dx, dwg, dwu))
    for other in seen[1:]:
        assert all(torch.equal(p, q) for p, q in zip(seen[0], other))


@pytest.mark.parametrize("K", [46, 54, 62, 214, 44, 50])
def test_rows_that_end_inside_a_chunk_many_times(K):
    # groups of more rows than one MFMA tile, a reduction that ends inside a 16-byte chunk, and
    # enough workgroups to fill the device: realigned chunks came out wrong in some of them
    torch = _t()
    counts = [32, 0] * 30
    o = [sum(counts[:i]) for i in range(len(counts) + 1)]
    offsets = torch.tensor(o, dtype=torch.int32, device="cuda")
    rows, N, E = o[-1], 1912, len(counts)
    x = _normal(_gen(1), (rows, K), 1.0).bfloat16()
    w = _weights(E, N, K, "bf16", "nk", 2, 0).t
    with spg.GroupedGemm(rows, N, K, E, "bf16", "nk") as plan:
        ws = _workspace(plan.workspace_bytes())
        for _ in range(6):
            y = torch.zeros(rows, N, device="cuda", dtype=torch.bfloat16)
            plan(x, w, offsets, y, workspace=ws)
            for e in range(0, E, 2):
                _check_rows(x[o[e]:o[e + 1]], _as_kn(w[e], "nk"), y[o[e]:o[e + 1]], "bf16", f"group {e}")


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("case", [([1300, 1100, 0, 900], 2304, 4160), ([2050], 4096, 6154), ([300, 515, 257, 600, 256, 1024, 70], 2050, 4096)],
                         ids=["groups", "one", "many"])
def test_last_round_in_parts(case, layout):
    # grids of a little more than a round of 256x256 tiles with long reductions: the last tiles are
    # split along the sum; rows cut on both sides of a tile's half, columns cut, G and U kept
    torch = _t()
    counts, N, K = case
    o = [3 + sum(counts[:i]) for i in range(len(counts) + 1)]
    rows, E = o[-1] + 2, len(counts)
    offsets = torch.tensor(o, dtype=torch.int32, device="cuda")
    tokens = 1500
    for dtype, src in (("bf16", True), ("f16", False)):
        dt = _dt(dtype)
        xr = tokens if src else rows
        x = Buf((xr, K), dt, 0, _normal(_gen(1), (xr, K), 1.0).to(dt))
        w = [_weights(E, N, K, dtype, layout, 2 + i, 0) for i in (0, 1)]
        dh = Buf((rows, N), dt, 0, _normal(_gen(4), (rows, N), 0.3).to(dt))
        source = _source(rows, tokens, 5) if src else None
        h, g, u, dx, y, dx1 = (Buf((rows, n), dt) for n in (N, N, N, K, N, K))
        dwg, dwu, dw = (Buf(w[0].t.shape, dt) for _ in range(3))
        t = tokens if src else None
        with spg.GroupedGated(rows, N, K, E, dtype, layout, "silu", tokens=t) as plan:
            plan(x.t, w[0].t, w[1].t, offsets, h.t, source=source, G=g.t, U=u.t,
                 workspace=_workspace(plan.workspace_bytes(backward=False)))
            plan.backward(dh.t, x.t, w[0].t, w[1].t, g.t, u.t, offsets, dx.t, dwg.t, dwu.t, source=source,
                          workspace=_workspace(plan.workspace_bytes()))
        with spg.GroupedGemm(rows, N, K, E, dtype, layout, tokens=t) as plan:
            plan(x.t, w[0].t, offsets, y.t, source=source, workspace=_workspace(plan.workspace_bytes(backward=False)))
            plan.backward(dh.t, x.t, w[0].t, offsets, dx1.t, dw.t, source=source, workspace=_workspace(plan.workspace_bytes()))
        torch.cuda.synchronize()
        xs = _gathered(x.t, source)
        for e in range(E):
            r = slice(o[e], o[e + 1])
            if o[e] == o[e + 1]:
                continue
            _check_forward(xs[r], w[0].t[e], w[1].t[e], h.t[r], g.t[r], u.t[r], dtype, layout, "silu")
            _check_backward(dh.t[r], xs[r], w[0].t[e], w[1].t[e], g.t[r], u.t[r], dx.t[r], dwg.t[e], dwu.t[e], dtype, layout, "silu")
            wd = _as_kn(w[0].t[e], layout)
            _check_rows(xs[r], wd, y.t[r], dtype, f"Y of group {e}")
            _check_rows(dh.t[r], wd.t().contiguous(), dx1.t[r], dtype, f"dX of group {e}")
        assert all(_untouched(b, o) for b in (h, g, u, dx, y, dx1))
        assert all(b.intact() for b in (x, *w, dh, h, g, u, dx, y, dx1, dwg, dwu, dw))
