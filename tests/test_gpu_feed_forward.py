"""GPU tests of the feed-forward operators (gated projection, its backward pass, int8
products, quantisation of rows) against plain formulas in 64 bits.

Tolerances, derived from the arithmetic and applied to every element.  With e the output
type's epsilon, an output y rounded once is off by e/2 |y|.  A sum of K products in fp32 in
any order is off by at most K 2^-24 S, S the sum of the products' magnitudes.  The
activations and their slopes are evaluated in fp32 from a sigmoid with relative error below
2^-20: act is off by 2^-20 |g|, act' by 2^-19 (1 + |g|); |act'| < 1.13 for all three.
fp16 results below 2^-14 are rounded to multiples of 2^-24: half of that is added.  In the
backward pass dG and dU are rounded to the operands' type before the products.
"""

import pytest

import software_pipelined_tiled_gemm_amd as spg
from tests import gpu_util

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
SLOPE = 1.13


def _t():
    import torch
    return torch


def _dt(name):
    torch = _t()
    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[name]


def _half_ulp(name):
    return _t().finfo(_dt(name)).eps / 2


def _tiny(name):
    return 2.0 ** -25 if name == "f16" else 2.0 ** -134


class Buf:
    """A tensor inside a larger allocation, `off` elements past a 16-byte boundary, with
    guard elements on both sides that must stay untouched."""

    def __init__(self, shape, dtype, off=0, value=None):
        torch = _t()
        n = 1
        for d in shape:
            n *= d
        self.n, self.lo = n, 64 + off
        raw = {1: torch.int8, 2: torch.int16, 4: torch.int32}[torch.empty(0, dtype=dtype).element_size()]
        self.raw = torch.full((n + 128 + off,), 0x5A, dtype=raw, device=gpu_util.torch_dev())
        self.t = self.raw.view(dtype)[self.lo:self.lo + n].view(shape)
        if value is not None:
            self.t.copy_(value)

    def intact(self):
        return bool((self.raw[:self.lo] == 0x5A).all()) and bool((self.raw[self.lo + self.n:] == 0x5A).all())


def _normal(gen, shape, std):
    torch = _t()
    return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=gen)


def _gen(seed):
    g = _t().Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _act(g, act):
    torch = _t()
    if act == "relu":
        return g.clamp(min=0)
    z = g if act == "silu" else 2 * 0.7978845608 * (g + 0.044715 * g ** 3)
    return g * torch.sigmoid(z)


def _slope(g, act):
    torch = _t()
    if act == "relu":
        return (g > 0).double()
    if act == "silu":
        z, dz = g, 1.0
    else:
        z, dz = 2 * 0.7978845608 * (g + 0.044715 * g ** 3), 2 * 0.7978845608 * (1 + 3 * 0.044715 * g * g)
    s = torch.sigmoid(z)
    return s + g * s * (1 - s) * dz


def _within(got, want, tol, what):
    torch = _t()
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    if bool(bad.any()):
        i = int(bad.flatten().nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at flat index {i}: "
                             f"got {got.flatten()[i].item()}, want {want.flatten()[i].item()}, "
                             f"tol {tol.flatten()[i].item()}")
    return float((err / tol.clamp(min=1e-300)).max()) if err.numel() else 0.0


# (M, N, K): few rows (1, 16, 17, 33, 64), tiles cut on every side, odd rows, one k-tile,
# more parts of the reduction than one, grids of the 256-wide tile, odd rows that are laid
# out again, rows of whole words that end inside a 16-byte chunk
SIZES = [(1, 48, 40), (1, 4096, 1001), (3, 130, 64), (16, 72, 200), (17, 96, 136), (33, 40, 8), (48, 56, 777),
         (64, 264, 512), (65, 100, 64), (129, 257, 320), (200, 64, 2048), (300, 2731, 1001), (511, 520, 500),
         (70, 33, 9), (96, 1536, 4096), (1280, 2304, 192), (1300, 2051, 1003),
         (60, 130, 70), (150, 262, 1002), (520, 2050, 196), (2100, 2050, 78)]


def _gated_case(M, N, K, dtype, layout, seed, off=0):
    gen = _gen(seed)
    dt = _dt(dtype)
    w = (N, K) if layout == "nk" else (K, N)
    x = Buf((M, K), dt, off, _normal(gen, (M, K), 1.0).to(dt))
    wg = Buf(w, dt, off, _normal(gen, w, K ** -0.5).to(dt))
    wu = Buf(w, dt, off, _normal(gen, w, K ** -0.5).to(dt))
    return x, wg, wu


def _as_kn(w, layout):
    d = w.double()
    return d.t().contiguous() if layout == "nk" else d


def _check_forward(x, wg, wu, h, g, u, dtype, layout, act):
    K = x.shape[1]
    xd, gd, ud = x.double(), _as_kn(wg, layout), _as_kn(wu, layout)
    G, U = xd @ gd, xd @ ud
    sg, su = K * U32 * (xd.abs() @ gd.abs()), K * U32 * (xd.abs() @ ud.abs())
    e, tiny = _half_ulp(dtype), _tiny(dtype)
    A = _act(G, act)
    want = A * U
    tol = e * want.abs() + SLOPE * sg * (U.abs() + su) + A.abs() * su + 2.0 ** -20 * G.abs() * U.abs() + tiny
    r = _within(h, want, tol, "H")
    if g is not None:
        _within(g, G, e * G.abs() + 1.01 * sg + tiny, "G")
        _within(u, U, e * U.abs() + 1.01 * su + tiny, "U")
    return r


def _workspace(nbytes):
    torch = _t()
    # filled with NaN patterns: nothing may be read before it is written
    return torch.full((max(nbytes, 1),), 0xFF, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_gated_forward(size, layout):
    torch = _t()
    M, N, K = size
    for i, (dtype, act, off, keep) in enumerate((("bf16", "silu", 0, False), ("f16", "gelu_tanh", 0, True),
                                                 ("bf16", "relu", 1, True), ("f16", "silu", 2, False))):
        x, wg, wu = _gated_case(M, N, K, dtype, layout, 100 + i, off)
        h, g, u = (Buf((M, N), _dt(dtype), off) for _ in range(3))
        with spg.Gated(M, N, K, dtype, layout, act) as plan:
            ws = _workspace(plan.workspace_bytes())
            plan(x.t, wg.t, wu.t, h.t, G=g.t if keep else None, U=u.t if keep else None, workspace=ws)
        torch.cuda.synchronize()
        _check_forward(x.t, wg.t, wu.t, h.t, g.t if keep else None, u.t if keep else None, dtype, layout, act)
        assert all(b.intact() for b in (x, wg, wu, h, g, u))


def _slopes(dh, g, u, dtype, act):
    """dG and dU, and what the rounded ones may be off by."""
    e, tiny = _half_ulp(dtype), _tiny(dtype)
    D, G, U = dh.double(), g.double(), u.double()
    dG, dU = D * U * _slope(G, act), D * _act(G, act)
    tg = e * dG.abs() + 1.01 * 2.0 ** -19 * D.abs() * U.abs() * (1 + G.abs()) + tiny
    tu = e * dU.abs() + 1.01 * 2.0 ** -20 * D.abs() * G.abs() + tiny
    return dG, dU, tg, tu


def _check_dx(dh, wg, wu, g, u, dx, dtype, layout, act):
    N = g.shape[1]
    e, tiny = _half_ulp(dtype), _tiny(dtype)
    gd, ud = _as_kn(wg, layout), _as_kn(wu, layout)
    dG, dU, tg, tu = _slopes(dh, g, u, dtype, act)
    want = dG @ gd.t() + dU @ ud.t()
    tol = e * want.abs() + 1.01 * (tg @ gd.abs().t() + tu @ ud.abs().t()) + tiny
    tol += 2 * N * U32 * ((dG.abs() + tg) @ gd.abs().t() + (dU.abs() + tu) @ ud.abs().t())
    _within(dx, want, tol, "dX")


def _check_dw(dh, x, g, u, dwg, dwu, dtype, layout, act):
    M = x.shape[0]
    e, tiny = _half_ulp(dtype), _tiny(dtype)
    X = x.double()
    dG, dU, tg, tu = _slopes(dh, g, u, dtype, act)
    for name, got, d, t in (("dWg", dwg, dG, tg), ("dWu", dwu, dU, tu)):
        w = X.t() @ d
        tol = e * w.abs() + 1.01 * (X.abs().t() @ t) + M * U32 * (X.abs().t() @ (d.abs() + t)) + tiny
        if layout == "nk":
            w, tol = w.t(), tol.t()
        _within(got, w, tol, name)


def _check_backward(dh, x, wg, wu, g, u, dx, dwg, dwu, dtype, layout, act):
    _check_dx(dh, wg, wu, g, u, dx, dtype, layout, act)
    _check_dw(dh, x, g, u, dwg, dwu, dtype, layout, act)


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("size", SIZES + [(2048, 1024, 256), (1000, 24, 1536)], ids=str)
def test_gated_backward(size, layout):
    torch = _t()
    M, N, K = size
    for i, (dtype, act, off) in enumerate((("bf16", "silu", 0), ("f16", "gelu_tanh", 0), ("bf16", "relu", 1),
                                           ("f16", "silu", 2))):
        x, wg, wu = _gated_case(M, N, K, dtype, layout, 200 + i, off)
        gen = _gen(300 + i)
        dt = _dt(dtype)
        g = Buf((M, N), dt, off, _normal(gen, (M, N), 1.0).to(dt))
        u = Buf((M, N), dt, off, _normal(gen, (M, N), 1.0).to(dt))
        dh = Buf((M, N), dt, off, _normal(gen, (M, N), 0.3).to(dt))
        dx, dwg, dwu = Buf(x.t.shape, dt, off), Buf(wg.t.shape, dt, off), Buf(wu.t.shape, dt, off)
        with spg.Gated(M, N, K, dtype, layout, act) as plan:
            ws = _workspace(plan.workspace_bytes())
            plan.backward(dh.t, x.t, wg.t, wu.t, g.t, u.t, dx.t, dwg.t, dwu.t, workspace=ws)
        torch.cuda.synchronize()
        _check_backward(dh.t, x.t, wg.t, wu.t, g.t, u.t, dx.t, dwg.t, dwu.t, dtype, layout, act)
        assert all(b.intact() for b in (x, wg, wu, g, u, dh, dx, dwg, dwu))


def test_gradient_against_differences():
    # sum(R * H) differenced along random directions of X, Wg and Wu in 64 bits (central
    # differences, error O(t^2)), against the fp16 gradients.  The gradients carry the
    # roundings of G, U, dG, dU and their own: five of 2^-11 each, random in sign over more
    # than 10^4 terms; 2^-8 of the norm of the products leaves each of them whole.
    torch = _t()
    M, N, K = 96, 160, 128
    for act in ("silu", "gelu_tanh"):
        for layout in ("nk", "kn"):
            x, wg, wu = (b.t for b in _gated_case(M, N, K, "f16", layout, 7))
            R = _normal(_gen(8), (M, N), 0.5).half()
            h, g, u = (torch.empty(M, N, dtype=torch.float16, device="cuda") for _ in range(3))
            dx, dwg, dwu = torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)
            with spg.Gated(M, N, K, "f16", layout, act) as plan:
                ws = _workspace(plan.workspace_bytes())
                plan(x, wg, wu, h, G=g, U=u, workspace=ws)
                plan.backward(R, x, wg, wu, g, u, dx, dwg, dwu, workspace=ws)
            for which, grad in ((0, dx), (1, dwg), (2, dwu)):
                p = [x.double(), wg.double(), wu.double()]
                v = _normal(_gen(20 + which), p[which].shape, 1.0).double()

                def loss(t):
                    q = list(p)
                    q[which] = q[which] + t * v
                    a, b = (q[i].t() if layout == "nk" else q[i] for i in (1, 2))
                    return (R.double() * _act(q[0] @ a, act) * (q[0] @ b)).sum()

                t = 1e-5
                slope = float((loss(t) - loss(-t)) / (2 * t))
                scale = float((grad.double() * v).norm())
                assert abs(float((grad.double() * v).sum()) - slope) <= 2.0 ** -8 * scale + 1e-6, (act, layout, which)


def test_gated_infinities_stay_in_their_row_and_column():
    # a value of one row never reaches another row, whatever lies past a row's end
    torch = _t()
    for layout in ("nk", "kn"):
        for M, N, K in ((5, 40, 72), (5, 40, 75), (100, 136, 72), (100, 130, 75), (100, 130, 74), (20, 130, 75),
                        (300, 520, 200), (300, 522, 202), (1100, 2306, 90)):
            x, wg, wu = (b.t for b in _gated_case(M, N, K, "bf16", layout, 11))
            x[2, :] = float("inf")
            x[M - 1, 0] = float("nan")
            wgk = wg if layout == "nk" else wg.t()
            wgk[7, 0] = float("nan")
            wgk[N - 1, K - 1] = float("inf")
            h = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
            with spg.Gated(M, N, K, "bf16", layout, "silu") as plan:
                plan(x, wg, wu, h, workspace=_workspace(plan.workspace_bytes()))
            ok = torch.isfinite(h.float())
            rows = [m for m in range(M) if m not in (2, M - 1)]
            cols = [n for n in range(N) if n not in (7, N - 1)]
            assert bool(ok[rows][:, cols].all()), (layout, M, N, K)
            assert bool(torch.isnan(h[:, 7].float()).all()) and bool(torch.isnan(h[M - 1].float()).all())


@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "relu"])
def test_slopes_of_extreme_preactivations(act):
    # one row and X = 1: dWg and dWu are dG and dU
    torch = _t()
    vals = [0.0, -0.0]
    for v in (1e-38, 1e-20, 1e-3, 0.5, 1.0, 5.0, 20.0, 90.0, 100.0, 1e4, 1e10, 1e19, 2e19, 1e20, 1e30, 3e38):
        vals += [v, -v]
    N, K = len(vals), 8
    g = torch.tensor([vals], dtype=torch.bfloat16, device="cuda")
    one = torch.ones(1, N, dtype=torch.bfloat16, device="cuda")
    x = torch.ones(1, K, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(N, K, dtype=torch.bfloat16, device="cuda")
    dx, dwg, dwu = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    with spg.Gated(1, N, K, "bf16", "nk", act) as plan:
        ws = _workspace(plan.workspace_bytes())
        plan.backward(one, x, w, w, g, one, dx, dwg, dwu, workspace=ws)
        d = g[0].double()
        e, tiny = _half_ulp("bf16"), _tiny("bf16")
        A, S = _act(d, act), _slope(d, act)
        # fp32 in between: the smallest results may be flushed
        _within(dwg[:, 0], S, 2 * e * S.abs() + 2.0 ** -19 * (1 + d.abs().clamp(max=100)) + tiny, "dG")
        _within(dwu[:, 0], A, 2 * e * A.abs() + 2.0 ** -20 * d.abs().clamp(max=100) + 2.0 ** -126, "dU")
        assert bool((dx == 0).all())
        g[0, 3] = float("nan")
        plan.backward(one, x, w, w, g, one, dx, dwg, dwu, workspace=ws)
        assert bool(torch.isnan(dwu[3]).all()) and bool(torch.isfinite(dwu[:3]).all())


@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "relu"])
def test_nan_gates_give_nan(act):
    torch = _t()
    for layout in ("nk", "kn"):
        for M, N, K in ((1, 40, 64), (40, 72, 64), (40, 72, 4), (30, 264, 2048)):
            x, wg, wu = (b.t for b in _gated_case(M, N, K, "f16", layout, 81))
            (wg if layout == "nk" else wg.t())[5] = float("nan")
            h = torch.empty(M, N, dtype=torch.float16, device="cuda")
            with spg.Gated(M, N, K, "f16", layout, act) as plan:
                plan(x, wg, wu, h, workspace=_workspace(plan.workspace_bytes()))
            nan = torch.isnan(h)
            assert bool(nan[:, 5].all()) and int(nan.sum()) == M, (layout, M, N, K)
    for M, N, K in ((1, 40, 64), (40, 72, 64), (40, 72, 4), (30, 264, 4096)):
        a, b = _ints(_gen(82), (M, K)), _ints(_gen(83), (N, K))
        sa, sb, sn = torch.ones(M, device="cuda"), torch.full((N,), 1e-6, device="cuda"), torch.full((N,), 1e-6, device="cuda")
        sn[5] = float("nan")
        c = torch.empty(M, N, device="cuda")
        with spg.QuantizedGemm(M, N, K, "f32", act) as plan:
            plan(a, sa, b, sn, c, B2=b, scale_b2=sb, workspace=_workspace(plan.workspace_bytes()))
        nan = torch.isnan(c)
        assert bool(nan[:, 5].all()) and int(nan.sum()) == M, (M, N, K)


def test_small_scales_whose_product_leaves_the_range():
    # 1e-30 * 1e-12 is subnormal in fp32, times sums of about 10^6 the results are not
    torch = _t()
    for M, N, K in ((3, 40, 640), (40, 72, 640), (40, 72, 12), (30, 264, 8192)):
        a, b = _ints(_gen(84), (M, K)), _ints(_gen(85), (N, K))
        sa, sb = torch.full((M,), 1e-30, device="cuda"), torch.full((N,), 1e-12, device="cuda")
        c = torch.empty(M, N, device="cuda")
        with spg.QuantizedGemm(M, N, K, "f32") as plan:
            plan(a, sa, b, sb, c, workspace=_workspace(plan.workspace_bytes()))
        p = (a.double() @ b.double().t()) * sa.double()[:, None] * sb.double()
        _within(c, p, 3.01 * U32 * p.abs() + 2.0 ** -149, "C")


@pytest.mark.parametrize("layout", ["nk", "kn"])
def test_gated_sizes_without_a_chunk(layout):
    # reductions and rows shorter than 16 bytes, and empty ones
    torch = _t()
    for M, N, K in ((5, 7, 3), (130, 5, 40), (4, 9, 0), (0, 5, 9), (6, 0, 9), (1, 1, 1), (9, 3, 17)):
        x, wg, wu = _gated_case(M, N, max(K, 0), "f16", layout, 31) if K else (
            Buf((M, 0), torch.float16), Buf((N, 0) if layout == "nk" else (0, N), torch.float16),
            Buf((N, 0) if layout == "nk" else (0, N), torch.float16))
        h, g, u = (Buf((M, N), torch.float16) for _ in range(3))
        dh = Buf((M, N), torch.float16, 0, _normal(_gen(5), (M, N), 0.3).half())
        dx, dwg, dwu = (Buf(b.t.shape, torch.float16) for b in (x, wg, wu))
        with spg.Gated(M, N, K, "f16", layout, "silu") as plan:
            ws = _workspace(plan.workspace_bytes())
            plan(x.t, wg.t, wu.t, h.t, G=g.t, U=u.t, workspace=ws)
            plan.backward(dh.t, x.t, wg.t, wu.t, g.t, u.t, dx.t, dwg.t, dwu.t, workspace=ws)
        torch.cuda.synchronize()
        _check_forward(x.t, wg.t, wu.t, h.t, g.t, u.t, "f16", layout, "silu")
        _check_backward(dh.t, x.t, wg.t, wu.t, g.t, u.t, dx.t, dwg.t, dwu.t, "f16", layout, "silu")
        assert all(b.intact() for b in (h, g, u, dx, dwg, dwu))


def _ints(gen, shape):
    torch = _t()
    return torch.randint(-128, 128, shape, generator=gen, device="cuda", dtype=torch.int32).to(torch.int8)


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("size", SIZES + [(1, 5, 7), (3, 4, 0), (90, 300, 5000), (1024, 768, 1280)], ids=str)
def test_quantized_product(size, out):
    torch = _t()
    M, N, K = size
    for i, (act, off) in enumerate((("none", 0), ("none", 3), ("silu", 0), ("gelu_tanh", 1), ("relu", 0),
                                    ("silu", 4))):
        gen = _gen(400 + i)
        a = Buf((M, K), torch.int8, off, _ints(gen, (M, K)))
        b = [Buf((N, K), torch.int8, off, _ints(gen, (N, K))) for _ in range(2 if act != "none" else 1)]
        std = 1.0 / (74.0 * 74.0 * max(K, 1) ** 0.5)          # products of uniform int8: about unit results
        sa = torch.empty(M, device="cuda").uniform_(0.5, 1.5, generator=gen)
        sb = [torch.empty(N, device="cuda").uniform_(0.5, 1.5, generator=gen) * std for _ in b]
        c = Buf((M, N), _dt(out), off)
        with spg.QuantizedGemm(M, N, K, out, act) as plan:
            ws = _workspace(plan.workspace_bytes())
            plan(a.t, sa, b[0].t, sb[0], c.t, B2=b[1].t if len(b) > 1 else None,
                 scale_b2=sb[1] if len(b) > 1 else None, workspace=ws)
        torch.cuda.synchronize()
        # |acc| < 2^31 is exact in 64 bits; its conversion, the product of the scales and
        # their product round once each in fp32
        p = [(a.t.double() @ w.t.double().t()) * sa.double()[:, None] * s.double() for w, s in zip(b, sb)]
        e, tiny = _half_ulp(out), _tiny(out)
        if act == "none":
            want, tol = p[0], (e + 3.01 * U32) * p[0].abs() + tiny
        else:
            A = _act(p[0], act)
            want = A * p[1]
            tol = (e * want.abs() + SLOPE * 3.01 * U32 * p[0].abs() * p[1].abs() * 1.01
                   + 4.02 * U32 * want.abs() + 2.0 ** -20 * p[0].abs() * p[1].abs() + tiny)
        _within(c.t, want, tol, f"C {act}")
        assert c.intact() and a.intact() and all(w.intact() for w in b)


def test_quantized_extremes():
    # the largest sums: every operand -128, the longest reduction
    torch = _t()
    for M, K in ((2, 131071), (70, 131056), (70, 131071)):
        a = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
        b = torch.full((40, K), -128, dtype=torch.int8, device="cuda")
        one, c = torch.ones(M, device="cuda"), torch.empty(M, 40, device="cuda")
        with spg.QuantizedGemm(M, 40, K, "f32") as plan:
            plan(a, one, b, torch.ones(40, device="cuda"), c, workspace=_workspace(plan.workspace_bytes()))
        assert bool((c == torch.tensor(16384.0 * K, dtype=torch.float64).float().item()).all())


def _rounded_rows(x):
    """The definition in 64 bits: 127 x / amax is off by less than 2^-46, and no quotient of
    two fp32 values that is not a half lies closer to one than 2^-33."""
    torch = _t()
    d = x.double()
    amax = d.abs().amax(dim=1, keepdim=True) if d.shape[1] else torch.zeros(d.shape[0], 1, dtype=torch.float64, device=d.device)
    q = torch.round(d * 127.0 / torch.where(amax > 0, amax, torch.ones_like(amax)))
    return q.to(torch.int8), (amax / 127.0).float().flatten()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_quantize_rows(dtype):
    torch = _t()
    dt = _dt(dtype)
    for K in (1, 7, 8, 40, 129, 1001, 4096, 5000, 16384, 20011):
        for off in (0, 1):
            gen = _gen(500 + K)
            M = 37
            x = _normal(gen, (M, K), 1.0)
            x[3] = 0.0
            x[4] *= 1e-3
            x[5] = 1.0
            x[6] *= 1e4
            if dtype != "f16":
                x[7] *= 1e-30
                x[8] *= 1e30
                x[9] *= 1e-42          # subnormal in fp32
            x[10] = -x[10].abs()
            # quotients on and next to halves: amax = 254, values k + 1/2
            r = torch.arange(K, device="cuda")
            x[11] = (r % 254 - 127).float() + 0.5
            x[11, K - 1] = 127.0
            x[12] = x[11] * 2
            xb = Buf((M, K), dt, off, x.to(dt))
            a, s = Buf((M, K), torch.int8, off), Buf((M,), torch.float32)
            spg.gemm_quantize_rows(xb.t, a.t, s.t)
            torch.cuda.synchronize()
            qa, qs = _rounded_rows(xb.t)
            assert bool((a.t == qa).all()), (K, off, int((a.t != qa).sum()))
            assert bool((s.t == qs).all()), (K, off)
            assert a.intact() and s.intact() and xb.intact()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_quantize_rows_of_every_length(dtype):
    # many short rows (a wave each, the last workgroup not full), and lengths on both sides of
    # what 2, 4, 8 and 16 vectors of 16 bytes a thread hold
    torch = _t()
    dt = _dt(dtype)
    e = 4 if dtype == "f32" else 8
    sizes = [(M, K) for M in (2047, 2048, 2049, 2051) for K in (1, 9, 64 * e + 3, 128 * e, 128 * e + 1)]
    sizes += [(3, v * 256 * e + d) for v in (2, 4, 8, 16) for d in (-1, 0, 1)]
    for M, K in sizes:
        for off in (0, 1):
            gen = _gen(700 + K)
            x = _normal(gen, (M, K), 1.0)
            x[1] = 0.0
            x[M - 1] *= 30.0
            xb = Buf((M, K), dt, off, x.to(dt))
            a, s = Buf((M, K), torch.int8, off), Buf((M,), torch.float32)
            spg.gemm_quantize_rows(xb.t, a.t, s.t)
            torch.cuda.synchronize()
            qa, qs = _rounded_rows(xb.t)
            assert bool((a.t == qa).all()), (M, K, off, int((a.t != qa).sum()))
            assert bool((s.t == qs).all()), (M, K, off)
            assert a.intact() and s.intact() and xb.intact()


def test_quantize_rows_past_one_grid_dimension():
    # four rows a workgroup and 2^23 workgroups in the grid's first dimension: the last five rows
    # are in the next
    torch = _t()
    M, K = (1 << 25) + 5, 2
    x = _normal(_gen(71), (M, K), 1.0).bfloat16()
    a = torch.full((M, K), 77, dtype=torch.int8, device="cuda")
    s = torch.full((M,), -1.0, device="cuda")
    spg.gemm_quantize_rows(x, a, s)
    for i in range(0, M, 1 << 23):
        qa, qs = _rounded_rows(x[i:i + (1 << 23)])
        assert bool((a[i:i + (1 << 23)] == qa).all()) and bool((s[i:i + (1 << 23)] == qs).all()), i


def test_quantize_rows_halves_of_fp32():
    # fp32 neighbours of every half: the rounding side is decided exactly
    torch = _t()
    for amax in (1.0, 3.3, 0.7531):
        top = torch.tensor(amax, dtype=torch.float32)
        half = torch.arange(-127, 127, dtype=torch.float64) + 0.5
        x = (half * top.double() / 127.0).float()
        rows = [x]
        for _ in range(3):
            rows.append(torch.nextafter(rows[-1], torch.tensor(float("inf"))))
        x = torch.cat(rows + [top[None]]).cuda()[None].repeat(2, 1).contiguous()
        a = torch.empty(x.shape, dtype=torch.int8, device="cuda")
        s = torch.empty(2, device="cuda")
        spg.gemm_quantize_rows(x, a, s)
        qa, qs = _rounded_rows(x)
        assert bool((a == qa).all()) and bool((s == qs).all())


def test_quantized_rows_that_are_not_finite():
    torch = _t()
    x = _normal(_gen(1), (6, 300), 1.0).bfloat16()
    x[1, 5] = float("inf")
    x[4, 299] = float("nan")
    a, s = torch.empty(6, 300, dtype=torch.int8, device="cuda"), torch.empty(6, device="cuda")
    spg.gemm_quantize_rows(x, a, s)
    b, sb, c = _ints(_gen(2), (50, 300)), torch.ones(50, device="cuda"), torch.empty(6, 50, device="cuda")
    with spg.QuantizedGemm(6, 50, 300, "f32") as plan:
        plan(a, s, b, sb, c, workspace=_workspace(plan.workspace_bytes()))
    for m in range(6):
        assert bool(torch.isnan(c[m]).all()) if m in (1, 4) else bool(torch.isfinite(c[m]).all())


def _big(shape, dtype, seed):
    torch = _t()
    t = torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, 1.0, generator=_gen(seed))
    assert bool((t[-1] != 0).any()) and bool((t[shape[0] // 2] != 0).any())
    return t


def _some(n):
    """The first and last indices of n, and some in between on both sides of its middle."""
    torch = _t()
    i = list(range(3)) + [n // 3, n // 2 - 1, n // 2, 2 * n // 3] + list(range(n - 70, n))
    return torch.tensor(sorted({j for j in i if 0 <= j < n}), device="cuda")


def test_rows_past_32_bits():
    # operands of more than 2^32 bytes: many rows of X, many rows of [N,K] weights (streamed
    # and tiled), long rows of [K,N] weights
    torch = _t()
    for M, N, K, layout in ((540000, 40, 4096, "nk"), (9, 1100000, 2048, "nk"), (70, 1100000, 2048, "nk"),
                            (70, 1100000, 2048, "kn"), (540001, 24, 4097, "nk")):
        x = _big((M, K), torch.bfloat16, 91)
        wg, wu = (_big((N, K) if layout == "nk" else (K, N), torch.bfloat16, s) for s in (92, 93))
        wg *= K ** -0.5
        wu *= K ** -0.5
        h = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        with spg.Gated(M, N, K, "bf16", layout, "silu") as plan:
            plan(x, wg, wu, h, workspace=_workspace(plan.workspace_bytes()))
        r, c = _some(M), _some(N)
        if layout == "nk":
            _check_forward(x[r], wg[c], wu[c], h[r][:, c], None, None, "bf16", "nk", "silu")
        else:
            _check_forward(x[r], wg[:, c], wu[:, c], h[r][:, c], None, None, "bf16", "kn", "silu")
        del x, wg, wu, h
        torch.cuda.empty_cache()


@pytest.mark.parametrize("layout", ["nk", "kn"])
def test_results_past_32_bits(layout):
    # H, G, U, dH of more than 2^31 elements, dG and dU of more than 2^32
    torch = _t()
    M, N, K = 50000, 45000, 64
    x, wg, wu = (b.t for b in _gated_case(M, N, K, "bf16", layout, 94))
    h, g, u = (torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    dx, dwg, dwu = torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)
    with spg.Gated(M, N, K, "bf16", layout, "silu") as plan:
        ws = torch.empty(plan.workspace_bytes(), dtype=torch.uint8, device="cuda")
        plan(x, wg, wu, h, G=g, U=u, workspace=ws)
        r, c = _some(M), _some(N)
        pick = (lambda w: w[c]) if layout == "nk" else (lambda w: w[:, c])
        _check_forward(x[r], pick(wg), pick(wu), h[r][:, c], g[r][:, c], u[r][:, c], "bf16", layout, "silu")
        dh = _big((M, N), torch.bfloat16, 95)
        plan.backward(dh, x, wg, wu, g, u, dx, dwg, dwu, workspace=ws)
    # dX of some rows, and the weights' gradients of some columns
    _check_dx(dh[r], wg, wu, g[r], u[r], dx[r], "bf16", layout, "silu")
    _check_dw(dh[:, c], x, g[:, c], u[:, c], pick(dwg), pick(dwu), "bf16", layout, "silu")


def test_int8_rows_past_32_bits():
    torch = _t()
    for M, N, K in ((70000, 40, 65537), (40, 70000, 65540), (9, 70000, 65540)):
        x = _big((M, K), torch.bfloat16, 96)
        a, sa = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
        spg.gemm_quantize_rows(x, a, sa)
        r, c = _some(M), _some(N)
        qa, qs = _rounded_rows(x[r])
        assert bool((a[r] == qa).all()) and bool((sa[r] == qs).all())
        del x
        b = torch.randint(-128, 128, (N, K), generator=_gen(97), device="cuda", dtype=torch.int8)
        sb = torch.full((N,), 1e-4, device="cuda")
        y = torch.empty(M, N, device="cuda")
        with spg.QuantizedGemm(M, N, K, "f32") as plan:
            plan(a, sa, b, sb, y, workspace=_workspace(plan.workspace_bytes()))
        p = (a[r].double() @ b[c].double().t()) * sa[r].double()[:, None] * sb[c].double()
        _within(y[r][:, c], p, 3.01 * U32 * p.abs(), "C")
        del a, b, y
        torch.cuda.empty_cache()


def test_other_stream_and_graph_replays():
    torch = _t()
    M, N, K = 200, 1024, 512
    x, wg, wu = (b.t for b in _gated_case(M, N, K, "bf16", "nk", 61))
    h, g, u, dh = (torch.zeros(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    dh.copy_(_normal(_gen(62), (M, N), 0.3))
    grads = [torch.empty_like(t) for t in (x, wg, wu)]
    a8, sa = torch.empty(M, N, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    b8, sb = _ints(_gen(63), (K, N)), torch.full((K,), 1e-3, device="cuda")
    y = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    plan, down = spg.Gated(M, N, K, "bf16", "nk", "silu"), spg.QuantizedGemm(M, K, N, "bf16")
    ws = _workspace(max(plan.workspace_bytes(), down.workspace_bytes()))

    def once():
        plan(x, wg, wu, h, G=g, U=u, workspace=ws)
        plan.backward(dh, x, wg, wu, g, u, *grads, workspace=ws)
        spg.gemm_quantize_rows(h, a8, sa)
        down(a8, sa, b8, sb, y, workspace=ws)
        return [h, g, u, *grads, y]

    want = [t.clone() for t in once()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for t in once():
            t.zero_()
        got = once()
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        once()
    for r in range(4):
        for t in (h, g, u, *grads, y):
            t.fill_(r)
        ws.fill_(0xFF)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(want, (h, g, u, *grads, y))), r


def test_repeated_passes_are_bitwise_equal():
    # split reductions are added in a fixed order
    torch = _t()
    M, N, K = 96, 1536, 4096
    for layout in ("nk", "kn"):
        x, wg, wu = (b.t for b in _gated_case(M, N, K, "f16", layout, 71))
        outs = []
        for _ in range(3):
            h, g, u = (torch.empty(M, N, dtype=torch.float16, device="cuda") for _ in range(3))
            grads = [torch.empty_like(t) for t in (x, wg, wu)]
            with spg.Gated(M, N, K, "f16", layout, "relu") as plan:
                ws = _workspace(plan.workspace_bytes())
                plan(x, wg, wu, h, G=g, U=u, workspace=ws)
                plan.backward(h, x, wg, wu, g, u, *grads, workspace=ws)
            outs.append([h, *grads])
        for o in outs[1:]:
            assert all(torch.equal(p, q) for p, q in zip(outs[0], o))


def test_wrappers_on_device_tensors(monkeypatch):
    # both call paths (compiled and Python) make the same calls and the same refusals
    torch = _t()
    M, N, K = 20, 72, 64
    x, wg, wu = (b.t for b in _gated_case(M, N, K, "bf16", "nk", 91))
    a8, sa = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    b8, sb = _ints(_gen(92), (N, K)), torch.full((N,), 1e-2, device="cuda")
    results = []
    for compiled in (True, False):
        if compiled:
            assert spg._calls_module() is not None, "the compiled call path is not built"
        else:
            monkeypatch.setattr(spg, "_calls", None)
        h, c = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda"), torch.zeros(M, N, device="cuda")
        side = torch.cuda.Stream()
        with spg.Gated(M, N, K, "bf16", "nk", "silu") as plan, spg.QuantizedGemm(M, N, K, "f32") as q:
            ws = _workspace(max(plan.workspace_bytes(), q.workspace_bytes()))
            side.wait_stream(torch.cuda.current_stream())
            plan(x, torch.nn.Parameter(wg), wu.detach().requires_grad_(True), h, workspace=ws, stream=side)
            side.synchronize()
            spg.gemm_quantize_rows(x.view(4, 5, K), a8.view(4, 5, K), sa.view(4, 5))
            q(a8, sa, b8, sb, c, workspace=ws)
            raw = torch.zeros_like(h)
            plan(x.data_ptr(), wg.data_ptr(), wu.data_ptr(), raw.data_ptr(), workspace=ws.data_ptr(),
                 stream=torch.cuda.current_stream().cuda_stream)
            torch.cuda.synchronize()
            results.append([h, c, raw, a8.clone(), sa.clone()])
            wide = torch.zeros(M, 2 * N, dtype=torch.bfloat16, device="cuda")
            for args in ((x.half(), wg, wu, h), (x, wg[:-1], wu, h), (x, wg, wu, wide[:, :N]), (x, wg, wu.cpu(), h),
                         (x[None], wg, wu, h)):
                with pytest.raises(spg.GemmError) as e:
                    plan(*args, workspace=ws)
                assert e.value.status == 1
            with pytest.raises(spg.GemmError):
                plan(x, wg, wu, None, workspace=ws)
            with pytest.raises(spg.GemmError):
                plan(x, wg, wu, h, G=torch.zeros_like(h), workspace=ws)
            for args in ((a8, sa, b8, sb.double(), c), (a8, sa[:-1], b8, sb, c), (a8.float(), sa, b8, sb, c)):
                with pytest.raises(spg.GemmError):
                    q(*args, workspace=ws)
            for args in ((x, a8[:-1], sa), (x, a8, sa.double()), (x.double(), a8, sa), (x, a8.t(), sa)):
                with pytest.raises(spg.GemmError):
                    spg.gemm_quantize_rows(*args)
    assert torch.equal(results[0][0], results[0][2])
    assert all(torch.equal(p, q) for p, q in zip(*results))


def test_example_block_trains_and_serves():
    # the example as a user runs it, on a small block: the loss falls every step (plain
    # gradient descent at a small rate on a smooth loss), and the int8 block differs by the
    # rounding of its operands: three quantisations a layer with steps of amax / 127, about
    # 4 standard deviations / 127, uniform errors of step / sqrt(12), give below 1% each of
    # the row's norm and together below 5%
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    try:
        import feed_forward
    finally:
        sys.path.pop(0)
    losses, err = feed_forward.main(tokens=96, model=136, hidden=264, steps=6, rate=0.2)
    assert all(b < a for a, b in zip(losses, losses[1:])), losses
    assert 0.0 < err < 0.05, err


def test_workspaces_are_checked_on_both_call_paths(monkeypatch):
    # refusals before any launch; only the workspace is wrong
    torch = _t()
    M, N, K = 96, 256, 8192
    x, wg, wu = (b.t for b in _gated_case(M, N, K, "bf16", "nk", 101))
    h = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    a8, sa = _ints(_gen(102), (M, K)), torch.ones(M, device="cuda")
    b8, sb, c = _ints(_gen(103), (N, K)), torch.ones(N, device="cuda"), torch.zeros(M, N, device="cuda")
    for compiled in (True, False):
        if not compiled:
            monkeypatch.setattr(spg, "_calls", None)
        with spg.Gated(M, N, K, "bf16", "nk", "silu") as plan, spg.QuantizedGemm(M, N, K, "f32") as q:
            n = max(plan.workspace_bytes(), q.workspace_bytes())
            for bad in (torch.empty(n, dtype=torch.uint8), torch.empty(1, dtype=torch.uint8, device="cuda").expand(n),
                        torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2],
                        torch.empty(16, dtype=torch.uint8, device="cuda"), None):
                for call in (lambda: plan(x, wg, wu, h, workspace=bad),
                             lambda: plan.backward(h, x, wg, wu, h, h, x, wg, wu, workspace=bad),
                             lambda: q(a8, sa, b8, sb, c, workspace=bad)):
                    with pytest.raises(spg.GemmError) as e:
                        call()
                    assert e.value.status == 1
    torch.cuda.synchronize()
    assert not bool(h.any()) and not bool(c.any())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "relu"])
def test_slopes_of_infinite_preactivations(act, dtype):
    # a stored infinity is a sum beyond the type's range: it counts as the largest finite
    # value.  One row and X = 1: dWg and dWu are dG and dU, rounded to the type twice.
    torch = _t()
    inf, dt = float("inf"), _dt(dtype)
    big = torch.finfo(dt).max
    # (bf16: dH U has to stay inside fp32)
    gates = [(g, u, d) for g in (inf, -inf, 2.0, -2.0, 0.0) for u in (inf, -inf, 1.0, -0.5, 0.0) for d in (0.0, 0.01, -1.0)]
    G, U, D = (torch.tensor([[t[i] for t in gates]], dtype=dt, device="cuda") for i in range(3))
    N, K = len(gates), 8
    x, w = torch.ones(1, K, dtype=dt, device="cuda"), torch.zeros(N, K, dtype=dt, device="cuda")
    dx, dwg, dwu = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    with spg.Gated(1, N, K, dtype, "nk", act) as plan:
        ws = _workspace(plan.workspace_bytes())
        plan.backward(D, x, w, w, G, U, dx, dwg, dwu, workspace=ws)
        g, u, d = G[0].double().clamp(-big, big), U[0].double().clamp(-big, big), D[0].double()
        e, tiny = _half_ulp(dtype), _tiny(dtype)
        A, S = _act(g, act), _slope(g, act)
        small = g.abs().clamp(max=100)
        want = d * u * S
        # slopes pass 1: where a result leaves the type's range, its rounding is infinite
        over = torch.isinf(want.to(dt))
        assert torch.equal(dwg[over, 0], want[over].to(dt))
        tol = 2.01 * e * want.abs() + 2.0 ** -19 * (d * u).abs() * (1 + small) + 2 * tiny
        _within(dwg[~over, 0], want[~over], tol[~over], "dG")
        _within(dwu[:, 0], d * A, 2.01 * e * (d * A).abs() + 2.0 ** -20 * d.abs() * small + 2.0 ** -126 + 2 * tiny, "dU")
        assert bool(over.any()) or bool((dx == 0).all())      # inf * 0 in the products
        # what is not a number stays so
        G[0, 0], U[0, 20] = float("nan"), float("nan")
        plan.backward(D, x, w, w, G, U, dx, dwg, dwu, workspace=ws)
        assert bool(torch.isnan(dwu[0]).all()) and bool(torch.isfinite(dwu[1:]).all())
        assert bool(torch.isnan(dwg[20]).all()) and not bool(torch.isnan(dwg[21:]).any())


@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "relu"])
def test_gates_beyond_fp16_train(act):
    # gates of +-70000 are infinite in fp16; H and every gradient of the formula in fp32 are not
    torch = _t()
    M, N, K = 3, 24, 16
    for layout in ("nk", "kn"):
        x = torch.full((M, K), 1.0, dtype=torch.float16, device="cuda")
        wg, wu = torch.full((N, K), 0.01, device="cuda"), torch.full((N, K), 1e-5, device="cuda")
        wg[3], wg[7] = 70000.0 / K, -70000.0 / K
        wg, wu = (w.half() if layout == "nk" else w.half().t().contiguous() for w in (wg, wu))
        h, g, u = (torch.empty(M, N, dtype=torch.float16, device="cuda") for _ in range(3))
        dh = torch.full_like(h, 0.125)
        dh[1] = 0.0
        grads = [torch.empty_like(t) for t in (x, wg, wu)]
        with spg.Gated(M, N, K, "f16", layout, act) as plan:
            ws = _workspace(plan.workspace_bytes())
            plan(x, wg, wu, h, G=g, U=u, workspace=ws)
            assert bool((g[:, 3] == float("inf")).all()) and bool((g[:, 7] == -float("inf")).all())
            plan.backward(dh, x, wg, wu, g, u, *grads, workspace=ws)
        assert all(bool(torch.isfinite(t).all()) for t in (h, *grads)), layout


def test_raw_pointers_with_a_workspace():
    # operands and workspace as raw pointers, where the reduction is split, against tensors
    torch = _t()
    M, N, K = 96, 256, 8192
    x, wg, wu = (b.t for b in _gated_case(M, N, K, "bf16", "nk", 105))
    out = []
    with spg.Gated(M, N, K, "bf16", "nk", "silu") as plan:
        ws = _workspace(plan.workspace_bytes())
        stream = torch.cuda.current_stream().cuda_stream
        for raw in (False, True):
            h, g, u = (torch.zeros(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(3))
            grads = [torch.zeros_like(t) for t in (x, wg, wu)]
            p = (lambda t: t.data_ptr()) if raw else (lambda t: t)
            plan(p(x), p(wg), p(wu), p(h), G=p(g), U=p(u), workspace=p(ws), stream=stream)
            plan.backward(*(p(t) for t in (h, x, wg, wu, g, u, *grads)), workspace=p(ws), stream=stream)
            torch.cuda.synchronize()
            out.append([h, g, u, *grads])
    assert all(torch.equal(a, b) and bool(a.any()) for a, b in zip(*out))


@pytest.mark.parametrize("layout", ["nk", "kn"])
def test_serving_in_its_own_workspace(layout):
    # split reductions and operands laid out again, in exactly what the projection asks for
    torch = _t()
    for M, N, K in ((96, 256, 8192), (1300, 2051, 1003), (300, 1024, 448)):
        x, wg, wu = (b.t for b in _gated_case(M, N, K, "bf16", layout, 107))
        h = Buf((M, N), torch.bfloat16)
        with spg.Gated(M, N, K, "bf16", layout, "silu") as plan:
            n = plan.workspace_bytes(backward=False)
            assert n <= plan.workspace_bytes()
            ws = Buf((max(n, 16),), torch.uint8, 0)
            plan(x, wg, wu, h.t, workspace=ws.t)
        torch.cuda.synchronize()
        _check_forward(x, wg, wu, h.t, None, None, "bf16", layout, "silu")
        assert h.intact() and ws.intact()


@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "relu"])
def test_slopes_where_dh_times_u_leaves_the_range(act):
    # bf16 holds values whose product fp32 does not; with the slope it does.  One row and X = 1:
    # dWg is dG, rounded to the type twice
    torch = _t()
    vals = [(g, u, d) for g in (-200.0, -20.0, -3.0, 0.5, 30.0) for u in (1e20, -3e38, 1e-3) for d in (1e20, -1e25, 2.0)]
    G, U, D = (torch.tensor([[t[i] for t in vals]], dtype=torch.bfloat16, device="cuda") for i in range(3))
    N, K = len(vals), 8
    x = torch.ones(1, K, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(N, K, dtype=torch.bfloat16, device="cuda")
    dx, dwg, dwu = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    with spg.Gated(1, N, K, "bf16", "nk", act) as plan:
        plan.backward(D, x, w, w, G, U, dx, dwg, dwu, workspace=_workspace(plan.workspace_bytes()))
    g, u, d = (t[0].double() for t in (G, U, D))
    want = d * u * _slope(g, act)
    tol = 2.01 * _half_ulp("bf16") * want.abs() + 2.0 ** -19 * (d * u).abs() * (1 + g.abs()) + 2 * _tiny("bf16")
    got = dwg[:, 0]
    assert not bool(torch.isnan(got).any())
    # clear of the range's end on either side: finite, or the infinity
    inside, outside = want.abs() + tol < 3e38, want.abs() - tol > 3.5e38
    _within(got[inside], want[inside], tol[inside], "dG")
    assert torch.equal(got[outside].double(), torch.sign(want[outside]) * float("inf"))
    assert bool(inside.any()) and bool(outside.any())
