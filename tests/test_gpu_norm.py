"""GPU tests of the layer norm and its backward pass against the formulas in 64 bits.

Tolerances, derived from the arithmetic and applied to every element.  u = 2^-24 is fp32's
rounding, e the output type's.  A sum of K values is accumulated in chains of at most
D = K / 64 + 16 additions (64 lanes at least share a row; the rest joins their sums): off by
D u S, S the sum of the magnitudes.  With c = x - mean:
  mean   em = (D + 2) u sum|x| / K
  var    sum (c - em)^2 / K = var + em^2 (c sums to 0), every term and the sum rounded:
         (D + 6) u var + em^2
  rstd   relative: half of var's error over var + eps, and 4 u for the root and the quotient
  n      rstd (em + u |c|) + |n| (rstd's + 2 u)
The backward pass is given the exact mean and rstd rounded to fp32: em = u |mean|, rstd's is u.
"""

import pytest

import software_pipelined_tiled_gemm_amd as spg
from tests.test_gpu_feed_forward import U32, Buf, _dt, _gen, _half_ulp, _normal, _t, _tiny, _within, _workspace

pytestmark = pytest.mark.gpu

EPS = 1e-5
# (rows, K): single rows, rows shorter than a vector, odd ones, rows that fill one to many vectors
# of a thread, more than any registers hold, many short rows, more rows than workgroups
SIZES = [(1, 4096), (1, 1), (3, 2), (5, 7), (4, 24), (2, 63), (9, 64), (33, 129), (70, 520), (511, 1001), (300, 2048),
         (7, 4095), (40, 5000), (12, 8192), (5, 12345), (3, 16384), (4, 20000), (2, 70001), (5000, 40), (3001, 512),
         (2500, 1025), (1, 16), (2049, 255)]
TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32"), ("f32", "f32")]


def _case(M, K, dtype, params, seed, off=0):
    gen = _gen(seed)
    x = _normal(gen, (M, K), 1.0) * _normal(gen, (M, 1), 1.0).exp_() + _normal(gen, (M, 1), 3.0)
    x = Buf((M, K), _dt(dtype), off, x.to(_dt(dtype)))
    w = Buf((K,), _dt(params), off, (1 + _normal(gen, (K,), 0.3)).to(_dt(params)))
    b = Buf((K,), _dt(params), off, _normal(gen, (K,), 0.3).to(_dt(params)))
    return x, w, b


def _forward(x, w, b):
    """y, mean, rstd, n in 64 bits, and how far mean, rstd (relative) and n may be off."""
    x = x.double()
    M, K = x.shape
    D = K / 64 + 16
    mean = x.mean(1, keepdim=True)
    c = x - mean
    var = (c * c).mean(1, keepdim=True)
    rstd = (var + EPS).rsqrt()
    n = c * rstd
    em = (D + 2) * U32 * x.abs().mean(1, keepdim=True)
    er = 0.51 * ((D + 6) * U32 * var + em * em) / (var + EPS) + 4 * U32
    en = rstd * (1 + er) * (em + U32 * c.abs()) + n.abs() * (er + 2 * U32)
    w = w.double() if w is not None else 1.0
    b = b.double() if b is not None else 0.0
    return n * w + b, mean, rstd, n, em, er, en, w, b


def _check_forward(x, w, b, y, mean, rstd, dtype):
    want, m, r, n, em, er, en, wd, bd = _forward(x, w, b)
    e, tiny = _half_ulp(dtype), _tiny(dtype)
    inner = en * abs(wd) + 2 * U32 * ((n * wd).abs() + abs(bd))
    _within(y, want, 1.01 * inner + e * (want.abs() + inner) + tiny, "Y")
    if mean is not None:
        _within(mean, m[:, 0], 1.01 * em[:, 0] + U32 * m[:, 0].abs() + 2.0 ** -140, "mean")
        _within(rstd, r[:, 0], 1.01 * er[:, 0] * r[:, 0], "rstd")


@pytest.mark.parametrize("types", TYPES, ids="-".join)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward(size, types):
    torch = _t()
    M, K = size
    dtype, params = types
    for i, (off, weight, bias, keep) in enumerate(((0, True, True, True), (1, True, False, False), (0, False, True, True),
                                                   (3, False, False, False))):
        x, w, b = _case(M, K, dtype, params, 10 + i, off)
        y, mean, rstd = Buf((M, K), _dt(dtype), off), Buf((M,), torch.float32), Buf((M,), torch.float32)
        with spg.LayerNorm(M, K, dtype, params, eps=EPS) as plan:
            plan(x.t, w.t if weight else None, b.t if bias else None, y.t, mean=mean.t if keep else None,
                 rstd=rstd.t if keep else None)
        torch.cuda.synchronize()
        _check_forward(x.t, w.t if weight else None, b.t if bias else None, y.t, mean.t if keep else None, rstd.t, dtype)
        assert all(v.intact() for v in (x, w, b, y, mean, rstd))


def _backward_of(x, w, dy):
    """dX, dweight, dbias in 64 bits."""
    y, mean, rstd, n, *_, wd, _ = _forward(x, w, None)
    g = dy.double() * wd
    dx = rstd * (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True))
    return dx, (dy.double() * n).sum(0), dy.double().sum(0)


@pytest.mark.parametrize("types", TYPES, ids="-".join)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_backward(size, types):
    torch = _t()
    M, K = size
    dtype, params = types
    D = K / 64 + 16
    e, ep = _half_ulp(dtype), _half_ulp(params)
    for i, (off, weight, want_w, want_b) in enumerate(((0, True, True, True), (1, True, True, False),
                                                       (0, False, False, True), (3, True, False, False))):
        x, w, _ = _case(M, K, dtype, params, 20 + i, off)
        dy = Buf((M, K), _dt(dtype), off, _normal(_gen(30 + i), (M, K), 0.3).to(_dt(dtype)))
        _, m, r, n, *_, wd, _ = _forward(x.t, w.t if weight else None, None)
        mean, rstd = m[:, 0].float(), r[:, 0].float()
        dx, dw, db = Buf((M, K), _dt(dtype), off), Buf((K,), _dt(params), off), Buf((K,), _dt(params), off)
        with spg.LayerNorm(M, K, dtype, params, eps=EPS) as plan:
            ws = _workspace(plan.workspace_bytes())
            plan.backward(dy.t, x.t, w.t if weight else None, mean, rstd, dx.t, dw.t if want_w else None,
                          db.t if want_b else None, workspace=ws)
        torch.cuda.synchronize()
        d = dy.t.double()
        c = x.t.double() - m
        en = r * 1.01 * (U32 * m.abs() + U32 * c.abs()) + 3 * U32 * n.abs()
        g = d * wd
        s, t = g.mean(1, keepdim=True), (g * n).mean(1, keepdim=True)
        es = (D + 3) * U32 * g.abs().mean(1, keepdim=True)
        et = (D + 5) * U32 * (g * n).abs().mean(1, keepdim=True) + 1.01 * (g.abs() * en).mean(1, keepdim=True)
        want, ww, wb = _backward_of(x.t, w.t if weight else None, dy.t)
        inner = r * (6 * U32 * (g.abs() + s.abs() + (n * t).abs()) + es + n.abs() * et + en * (t.abs() + et))
        _within(dx.t, want, 1.02 * inner + e * (want.abs() + inner) + _tiny(dtype), "dX")
        # sums over the rows: M - 1 additions at most, in whatever order
        if want_w:
            inner = (M + 3) * U32 * (d * n).abs().sum(0) + 1.01 * (d.abs() * en).sum(0)
            _within(dw.t, ww, 1.01 * inner + ep * (ww.abs() + inner) + _tiny(params), "dweight")
        if want_b:
            inner = (M + 1) * U32 * d.abs().sum(0)
            _within(db.t, wb, 1.01 * inner + ep * (wb.abs() + inner) + _tiny(params), "dbias")
        assert all(v.intact() for v in (x, w, dy, dx, dw, db))


def test_gradients_against_differences():
    # the 64-bit forward formula at x +- h d: the central difference is off by h^2 / 6 of the third
    # derivative (below 100 of the direction's size here) and by 64-bit rounding over h
    torch = _t()
    M, K, h = 6, 200, 1e-4
    gen = _gen(5)
    x, w, b = (v.t for v in _case(M, K, "f32", "f32", 6))
    dy = _normal(gen, (M, K), 0.5)
    y, mean, rstd = torch.empty_like(x), torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    with spg.LayerNorm(M, K, "f32", eps=EPS) as plan:
        plan(x, w, b, y, mean=mean, rstd=rstd)
        plan.backward(dy, x, w, mean, rstd, dx, dw, db, workspace=_workspace(plan.workspace_bytes()))

    def loss(x, w, b):
        return (_forward(x, w, b)[0] * dy.double()).sum()

    for grad, which in ((dx, 0), (dw, 1), (db, 2)):
        for _ in range(4):
            d = _normal(gen, grad.shape, 1.0).double()
            hi, lo = [v.double() for v in (x, w, b)], [v.double() for v in (x, w, b)]
            hi[which], lo[which] = hi[which] + h * d, lo[which] - h * d
            want = float((loss(*hi) - loss(*lo)) / (2 * h))
            got = float((grad.double() * d).sum())
            # fp32's share: the element tolerances of the tests above are below 2^-18 of the gradients' sizes
            tol = 2.0 ** -18 * float((grad.double().abs() * d.abs()).sum()) + 100 * h * h * float(d.norm()) ** 3 + 1e-9
            assert abs(got - want) <= tol, (which, got, want, tol)


def test_rows_far_from_zero_keep_their_variance():
    # mean 1000, deviation 1: sum x^2 - mean^2 would lose 20 of fp32's 24 bits
    torch = _t()
    for M, K in ((3, 4096), (2, 33000), (2100, 300)):
        gen = _gen(7)
        x = 1000 + _normal(gen, (M, K), 1.0)
        y = torch.empty_like(x)
        with spg.LayerNorm(M, K, "f32", eps=EPS) as plan:
            plan(x, None, None, y)
        _check_forward(x, None, None, y, None, None, "f32")


def test_constant_rows_infinities_and_nan():
    torch = _t()
    for K in (8, 1024, 5000, 40000):
        for M in (5, 3000 if K == 8 else 6):
            x = torch.full((M, K), 3.0, device="cuda", dtype=torch.bfloat16)
            x[1, K // 2], x[2, 0], x[3, K - 1] = float("inf"), float("nan"), float("-inf")
            w = torch.ones(K, device="cuda", dtype=torch.bfloat16)
            b = torch.full((K,), 0.25, device="cuda", dtype=torch.bfloat16)
            y = torch.empty_like(x)
            with spg.LayerNorm(M, K, "bf16") as plan:
                plan(x, w, b, y)
            # sums of threes are exact up to 2^24 / 3 of them: the deviation is zero
            assert bool((y[0] == 0.25).all()) and bool((y[4:] == 0.25).all()), K
            assert bool(torch.isnan(y[1:4]).all()), K


def test_nothing_to_do_and_sums_over_nothing():
    torch = _t()
    for params in ("bf16", "f32"):
        with spg.LayerNorm(0, 100, "bf16", params) as plan:
            e = torch.empty(0, 100, device="cuda", dtype=torch.bfloat16)
            r = torch.empty(0, device="cuda")
            plan(e, None, None, e, mean=r, rstd=r)
            dw = torch.full((100,), 7.0, device="cuda", dtype=_dt(params))
            db = dw.clone()
            plan.backward(e, e, None, r, r, e, dw, db, workspace=_workspace(plan.workspace_bytes()))
            assert bool((dw == 0).all()) and bool((db == 0).all())
    with spg.LayerNorm(4, 0, "f32") as plan:
        e = torch.empty(4, 0, device="cuda")
        plan(e, None, None, e)


@pytest.mark.parametrize("size", [(511, 1001), (9000, 300), (4000, 4096), (70, 40000)], ids=str)
def test_results_repeat(size):
    torch = _t()
    M, K = size
    x, w, b = (v.t for v in _case(M, K, "bf16", "f32", 8))
    dy = _normal(_gen(9), (M, K), 0.3).bfloat16()
    seen = []
    with spg.LayerNorm(M, K, "bf16", "f32") as plan:
        for _ in range(3):
            y, dx = torch.empty_like(x), torch.empty_like(x)
            mean, rstd, dw, db = (torch.empty(n, device="cuda") for n in (M, M, K, K))
            plan(x, w, b, y, mean=mean, rstd=rstd)
            plan.backward(dy, x, w, mean, rstd, dx, dw, db, workspace=_workspace(plan.workspace_bytes()))
            seen.append((y, mean, rstd, dx, dw, db))
    for other in seen[1:]:
        assert all(torch.equal(p, q) for p, q in zip(seen[0], other))
