"""GPU tests of the layer norm on rows of very large finite values: squares of deviations above 2^64
and sums above 2^128 pass fp32's range, the results do not.  Against the formulas in 64 bits, with
the tolerances of test_gpu_norm.py: they are relative to the rows' own sizes, and a power of two
that a row is multiplied by changes none of them."""

import pytest

import software_pipelined_tiled_gemm_amd as spg
from tests.test_gpu_feed_forward import U32, Buf, _dt, _gen, _half_ulp, _normal, _t, _tiny, _within, _workspace
from tests.test_gpu_norm import EPS, _backward_of, _check_forward, _forward

pytestmark = pytest.mark.gpu

# (rows, K): rows of any length, and every team that keeps them in registers, whole vectors and tails
SIZES = [(9, 5), (9, 24), (2100, 40), (2100, 999), (9, 520), (9, 1001), (9, 4096), (18, 5000), (9, 12345), (9, 16384), (9, 20000)]
TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]
# deviations of the rows in turn; those above 1e36 have a reciprocal below fp32's normal numbers
SIZE_OF_ROW = [1.0, 1e15, 1.5e19, 4e19, 1e24, 1e30, 3e33, 1e36, 1e-3]


def _rows(M, K, dtype, shift, seed):
    torch = _t()
    size = torch.tensor([SIZE_OF_ROW[i % len(SIZE_OF_ROW)] for i in range(M)], device="cuda")[:, None]
    x = (_normal(_gen(seed), (M, K), 1.0).clamp(-20, 20) + shift * _normal(_gen(seed + 1), (M, 1), 1.0).clamp(-4, 4)) * size
    x = x.to(_dt(dtype))
    assert bool(torch.isfinite(x).all())
    return x


@pytest.mark.parametrize("types", TYPES, ids="-".join)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward_and_backward(size, types):
    torch = _t()
    M, K = size
    dtype, params = types
    D = K / 64 + 16
    e, ep = _half_ulp(dtype), _half_ulp(params)
    for off, shift in ((0, 0.0), (1, 3.0)):
        x = Buf((M, K), _dt(dtype), off, _rows(M, K, dtype, shift, 5))
        dy = Buf((M, K), _dt(dtype), off, _normal(_gen(7), (M, K), 0.3).to(_dt(dtype)))
        w = Buf((K,), _dt(params), off, (1 + _normal(_gen(8), (K,), 0.3)).to(_dt(params)))
        b = Buf((K,), _dt(params), off, _normal(_gen(9), (K,), 0.3).to(_dt(params)))
        y, dx, mean, rstd = Buf((M, K), _dt(dtype), off), Buf((M, K), _dt(dtype), off), Buf((M,), torch.float32), Buf((M,), torch.float32)
        dw, db = Buf((K,), _dt(params), off), Buf((K,), _dt(params), off)
        _, m, r, n, *_, wd, _ = _forward(x.t, w.t, b.t)
        m32, r32 = m[:, 0].float(), r[:, 0].float()
        with spg.LayerNorm(M, K, dtype, params, eps=EPS) as plan:
            plan(x.t, w.t, b.t, y.t, mean=mean.t, rstd=rstd.t)
            plan.backward(dy.t, x.t, w.t, m32, r32, dx.t, dw.t, db.t, workspace=_workspace(plan.workspace_bytes()))
        torch.cuda.synchronize()
        _check_forward(x.t, w.t, b.t, y.t, mean.t, rstd.t, dtype)
        d = dy.t.double()
        c = x.t.double() - m
        en = r * 1.01 * (U32 * m.abs() + U32 * c.abs()) + 3 * U32 * n.abs()
        g = d * wd
        s, t = g.mean(1, keepdim=True), (g * n).mean(1, keepdim=True)
        es = (D + 3) * U32 * g.abs().mean(1, keepdim=True)
        et = (D + 5) * U32 * (g * n).abs().mean(1, keepdim=True) + 1.01 * (g.abs() * en).mean(1, keepdim=True)
        want, ww, wb = _backward_of(x.t, w.t, dy.t)
        inner = r * (6 * U32 * (g.abs() + s.abs() + (n * t).abs()) + es + n.abs() * et + en * (t.abs() + et))
        _within(dx.t, want, 1.02 * inner + e * (want.abs() + inner) + _tiny(dtype), "dX")
        inner = (M + 3) * U32 * (d * n).abs().sum(0) + 1.01 * (d.abs() * en).sum(0)
        _within(dw.t, ww, 1.01 * inner + ep * (ww.abs() + inner) + _tiny(params), "dweight")
        inner = (M + 1) * U32 * d.abs().sum(0)
        _within(db.t, wb, 1.01 * inner + ep * (wb.abs() + inner) + _tiny(params), "dbias")
        assert all(v.intact() for v in (x, w, b, dy, y, dx, mean, rstd, dw, db))


@pytest.mark.parametrize("types", TYPES, ids="-".join)
@pytest.mark.parametrize("K", [6, 24, 40, 1000, 5000, 12345, 20000])
def test_one_value_throughout(K, types):
    # n is 0 exactly: powers of two, of which sums are exact; 2^122 sqrt(1 / eps) and larger sums than
    # 2^128 are past fp32's range
    torch = _t()
    dtype, params = types
    M = 2100 if K == 40 else 5
    x = torch.full((M, K), 2.0 ** 122, dtype=_dt(dtype), device="cuda")
    x[1], x[2] = -2.0 ** 127, 1.0
    dy = _normal(_gen(3), (M, K), 0.5).to(_dt(dtype))
    w = (1 + _normal(_gen(4), (K,), 0.3)).to(_dt(params))
    b = _normal(_gen(5), (K,), 0.3).to(_dt(params))
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = (torch.empty(M, device="cuda") for _ in range(2))
    dw, db = torch.empty_like(w), torch.empty_like(b)
    with spg.LayerNorm(M, K, dtype, params, eps=EPS) as plan:
        plan(x, w, b, y, mean=mean, rstd=rstd)
        plan.backward(dy, x, w, mean, rstd, dx, dw, db, workspace=_workspace(plan.workspace_bytes()))
    assert torch.equal(mean, x[:, 0].float())
    assert torch.equal(y, b.to(y.dtype).expand(M, K))
    # rstd: 4 roundings of the root and the quotient, as in test_gpu_norm.py
    _within(rstd, torch.full((M,), EPS, dtype=torch.double, device="cuda").float().double().rsqrt(),
            torch.full((M,), 5 * U32 * EPS ** -0.5, dtype=torch.double, device="cuda"), "rstd")
    g = dy.double() * w.double()
    r, D, e = rstd.double()[:, None], K / 64 + 16, _half_ulp(dtype)
    want = r * (g - g.mean(1, keepdim=True))
    inner = r * (6 * U32 * (g.abs() + g.mean(1, keepdim=True).abs()) + (D + 3) * U32 * g.abs().mean(1, keepdim=True))
    _within(dx, want, 1.02 * inner + e * (want.abs() + inner), "dX")
    assert bool((dw == 0).all())


@pytest.mark.parametrize("K", [6, 24, 4096, 12346, 20000])
def test_the_largest_values(K):
    # +-the largest fp32 value in turn: n is +-1; rstd is 2^-128, a number of 22 bits, so that it and
    # what it is multiplied with are off by 2^-21 more
    torch = _t()
    M, most = 3, torch.finfo(torch.float32).max
    x = torch.full((M, K), most, device="cuda")
    x[:, 1::2] = -most
    w, b = 1 + _normal(_gen(4), (K,), 0.3), _normal(_gen(5), (K,), 0.3)
    dy = _normal(_gen(3), (M, K), 0.5)
    y, dx, mean, rstd, dw, db = (torch.empty_like(t) for t in (x, x, x[:, 0], x[:, 0], w, b))
    with spg.LayerNorm(M, K, "f32", eps=EPS) as plan:
        plan(x, w, b, y, mean=mean, rstd=rstd)
        plan.backward(dy, x, w, mean, rstd, dx, dw, db, workspace=_workspace(plan.workspace_bytes()))
    n = torch.sign(x).double()
    near = 2.0 ** -20 + (K / 64 + 40) * U32
    _within(y, n * w.double() + b.double(), near * (w.double().abs() + b.double().abs()).expand(M, K), "Y")
    assert bool((mean == 0).all())
    _within(rstd, torch.full_like(mean, most).double().reciprocal(), torch.full_like(mean, near * 2.0 ** -128).double(), "rstd")
    g = dy.double() * w.double()
    size = g.abs() + g.mean(1, keepdim=True).abs() + (g * n).abs().mean(1, keepdim=True)
    want = (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True)) / most
    _within(dx, want, near * size / most + 2.0 ** -149, "dX")
    _within(dw, (dy.double() * n).sum(0), near * dy.double().abs().sum(0), "dweight")


def test_infinities_and_nan_stay():
    torch = _t()
    for K in (5, 24, 4096, 20000):
        for dtype in ("bf16", "f32", "f16"):
            x = torch.full((4, K), 60000.0 if dtype == "f16" else 1e30, device="cuda", dtype=_dt(dtype))
            x[1, K // 2], x[2, 0], x[3, K - 1] = float("inf"), float("nan"), float("-inf")
            y = torch.zeros_like(x)
            with spg.LayerNorm(4, K, dtype) as plan:
                plan(x, None, None, y)
            assert not bool(torch.isnan(y[0]).any()) and bool(torch.isnan(y[1:]).all()), (K, dtype)
