"""GPU tests of the parameters' gradients of the layer norm over rows that no registers hold (K < 8
and K > 16384): many rows, whose sums are taken in parts.  Against sums in 64 bits, with tolerances
that a single chain of additions over all rows does not meet.

A sum over M rows is a chain of at most C additions: a thread's own rows (M / (parts R) of them,
R = 32 threads of a workgroup share its rows for K < 8, 4 for long rows), R of the workgroup, and the
parts' sums (an eighth of a sixteenth of them, rounded up, times 8, and 16).  With S the sum of the
magnitudes it is off by (C + 3) 2^-24 S, 3 for n and its product, and n by what it is off itself
(en as in test_gpu_norm.py)."""

import pytest

import software_pipelined_tiled_gemm_amd as spg
from tests.test_gpu_feed_forward import U32, Buf, _dt, _gen, _half_ulp, _normal, _t, _tiny, _within, _workspace

pytestmark = pytest.mark.gpu


def _chain(M, K):
    r, blocks = (32, 1) if K < 8 else (4, -(-K // 64))
    parts = max(1, min(-(-M // 256), 2048 // blocks))
    return -(-M // parts) // r + 1 + r + parts // 16 + 8 + 16


def _check(got, want, inner, params, what):
    """got is want, off by `inner` before its rounding to the parameters' type.  fp16 ends at 65504, and
    what is 65520 or more (half a step of 32 beyond) rounds to infinity: 300007 values of 0.24 on
    average, fp16's half-normal ones here, sum to 71900."""
    torch = _t()
    if params == "f16":
        past = want.abs() - inner >= 65520.0
        assert torch.equal(got.double()[past], torch.sign(want[past]) * float("inf")), what
        got, want, inner = got[~past], want[~past], inner[~past]
    _within(got, want, 1.01 * inner + _half_ulp(params) * (want.abs() + inner) + _tiny(params), what)


# one part, two, a part that ends early, as many as there are
@pytest.mark.parametrize("types", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f32", "f32")], ids="-".join)
@pytest.mark.parametrize("size", [(256, 4), (257, 3), (513, 7), (40001, 1), (300007, 5), (1 << 20, 6), (200, 20000), (257, 16385),
                                  (1025, 20001), (2100, 16500), (300, 70001)], ids=str)
def test_many_rows(size, types):
    torch = _t()
    M, K = size
    dtype, params = types
    C = _chain(M, K)
    for off, want_w, want_b in ((0, True, True), (1, True, False), (0, False, True)):
        x = Buf((M, K), _dt(dtype), off, (_normal(_gen(1), (M, K), 1.0) + _normal(_gen(2), (M, 1), 2.0)).to(_dt(dtype)))
        # gradients of one sign, so that the sums are as large as their magnitudes
        dy = Buf((M, K), _dt(dtype), off, _normal(_gen(3), (M, K), 0.3).abs().to(_dt(dtype)))
        mean, rstd = x.t.float().mean(1), 0.5 + torch.rand(M, generator=_gen(4), device="cuda")
        dx, dw, db = Buf((M, K), _dt(dtype), off), Buf((K,), _dt(params), off), Buf((K,), _dt(params), off)
        with spg.LayerNorm(M, K, dtype, params) as plan:
            ws = Buf((max(1, plan.workspace_bytes()),), torch.uint8)
            plan.backward(dy.t, x.t, None, mean, rstd, dx.t, dw.t if want_w else None, db.t if want_b else None, workspace=ws.t)
        torch.cuda.synchronize()
        sw, aw, ew, sb = (torch.zeros(K, dtype=torch.double, device="cuda") for _ in range(4))
        for i in range(0, M, 1 << 18):
            j = slice(i, i + (1 << 18))
            d, m, r = dy.t[j].double(), mean[j].double()[:, None], rstd[j].double()[:, None]
            c = x.t[j].double() - m
            n = c * r
            sw += (d * n).sum(0)
            aw += (d * n).abs().sum(0)
            ew += (d.abs() * (r * U32 * c.abs() + 2 * U32 * n.abs())).sum(0)
            sb += d.sum(0)
        if want_w:
            _check(dw.t, sw, (C + 3) * U32 * aw + 1.01 * ew, params, "dweight")
        if want_b:
            _check(db.t, sb, C * U32 * sb, params, "dbias")
        assert (want_w or bool((dw.raw == 0x5A).all())) and (want_b or bool((db.raw == 0x5A).all()))
        assert all(v.intact() for v in (x, dy, dx, dw, db, ws))


def test_a_hundred_million_rows():
    # sums of ones, which a thread's single chain would end at 2^24.  A thread's own and a workgroup's
    # are exact (below 2^24), the parts' join has at most 8 + 16 roundings after them
    torch = _t()
    M, K = 100_000_000, 4
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    x[:, ::2] = 1.0
    dy = torch.ones_like(x)
    mean, rstd = torch.full((M,), 0.5, device="cuda"), torch.full((M,), 2.0, device="cuda")
    dx, dw, db = torch.empty_like(x), torch.empty(K, device="cuda"), torch.empty(K, device="cuda")
    with spg.LayerNorm(M, K, "bf16", "f32") as plan:
        plan.backward(dy, x, None, mean, rstd, dx, dw, db, workspace=_workspace(plan.workspace_bytes()))
    want = torch.full((K,), float(M), dtype=torch.double, device="cuda")
    _within(db, want, 152 * U32 * want, "dbias")         # 128 parts a wave, 8 at a time, and 16 waves
    sign = torch.tensor([1.0, -1.0, 1.0, -1.0], dtype=torch.double, device="cuda")
    _within(dw, sign * want, 152 * U32 * want, "dweight")


@pytest.mark.parametrize("K", [5, 20000])
def test_repeats_and_captures(K):
    torch = _t()
    M = 3000
    x, dy = (_normal(_gen(i), (M, K), 1.0).bfloat16() for i in (1, 2))
    mean, rstd = x.float().mean(1), torch.ones(M, device="cuda")
    dx, dw, db = torch.empty_like(x), torch.empty(K, device="cuda"), torch.empty(K, device="cuda")
    with spg.LayerNorm(M, K, "bf16", "f32") as plan:
        ws = _workspace(plan.workspace_bytes())

        def go():
            plan.backward(dy, x, None, mean, rstd, dx, dw, db, workspace=ws)
        go()
        want = [t.clone() for t in (dx, dw, db)]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            go()
        for _ in range(4):
            for t in (dx, dw, db):
                t.zero_()
            ws.fill_(0xFF)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), want))
            go()
            assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), want))
