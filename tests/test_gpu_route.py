"""GPU tests of the routing and of the combination of the experts' rows.

Choices, places and offsets are whole numbers and have to be exact.  Gates: with u = 2^-24 and
z = |x - max| over the logits, the subtraction is off by u z, expf by 2 u of its result at most
(its documented 1 ulp), a sum of E terms in chains of D = E / 64 + 8 additions by D u of it,
the quotient by u: relative (z + mean of z over the softmax + D + 6) u.  The logits' gradient
multiplies a gate with d - sum p d, whose sum has the same relative error on its magnitudes.
"""

import pytest

import software_pipelined_tiled_gemm_amd as spg
from tests.test_gpu_feed_forward import U32, Buf, _dt, _gen, _half_ulp, _normal, _t, _tiny, _within, _workspace

pytestmark = pytest.mark.gpu

NINF = float("-inf")


def _want(x, k, renorm):
    """What the routing of logits x (64 bits, on the CPU) has to give; gates where no NaN is."""
    torch = _t()
    T, E = x.shape
    key = torch.where(torch.isnan(x), torch.full_like(x, NINF), x)
    order = key.sort(dim=1, descending=True, stable=True).indices[:, :k]
    value = key.gather(1, order)
    live = value > NINF
    expert = torch.where(live, order, -1)
    group = torch.where(live, order, E).reshape(-1)
    by = group.sort(stable=True).indices
    slot = torch.empty(T * k, dtype=torch.long)
    slot[by] = torch.arange(T * k)
    slot = torch.where(live, slot.view(T, k), -1)
    count = torch.bincount(group, minlength=E + 1)[:E]
    offsets = torch.cat((torch.zeros(1, dtype=torch.long), count.cumsum(0)))
    n = int(offsets[-1])
    source = by[:n] // k
    part = torch.zeros_like(x, dtype=torch.bool)
    if k and T:
        part.scatter_(1, order, live)
    share = torch.where(part, x, torch.full_like(x, NINF)) if renorm else x
    some = live.any(1, keepdim=True)
    p = torch.softmax(torch.where(some, share, torch.zeros_like(share)), 1)
    p = torch.where(some, p, torch.zeros_like(p))
    gate = torch.where(live, p.gather(1, order), torch.zeros_like(value))
    return expert, slot, source, offsets, gate, p, part, order, live


def _logits(T, E, dtype, seed, ties=True):
    torch = _t()
    x = _normal(_gen(seed), (T, E), 2.0)
    if ties and E > 1:
        x = (x * 4).round() / 4             # many equal ones
    return x.to(_dt(dtype))


def _call(x, k, dtype, renorm, off=0):
    torch = _t()
    T, E = x.shape
    xb = Buf((T, E), _dt(dtype), off, x)
    gate = Buf((T, k), torch.float32)
    expert, slot = Buf((T, k), torch.int32), Buf((T, k), torch.int32)
    source, offsets = Buf((T * k,), torch.int32), Buf((E + 1,), torch.int32)
    with spg.Router(T, E, k, dtype, renormalise=renorm) as plan:
        plan(xb.t, gate.t, expert.t, slot.t, source.t, offsets.t, workspace=_workspace(plan.workspace_bytes()))
    torch.cuda.synchronize()
    assert all(b.intact() for b in (xb, gate, expert, slot, source, offsets))
    return xb.t, gate.t, expert.t, slot.t, source.t, offsets.t


def _tolerance(x, p, E):
    """Relative error of the softmax p of x [T,E], per element."""
    torch = _t()
    D = E / 64 + 8
    z = torch.where(p > 0, (x - x.amax(1, keepdim=True)).abs(), torch.zeros_like(x))
    return (z + (p * z).sum(1, keepdim=True) + D + 6) * U32 * 1.01


def _check(x, k, renorm, got):
    torch = _t()
    _, gate, expert, slot, source, offsets = got
    xd = x.double().cpu()
    w_expert, w_slot, w_source, w_offsets, w_gate, p, part, order, live = _want(xd, k, renorm)
    assert torch.equal(offsets.long().cpu(), w_offsets)
    assert torch.equal(expert.long().cpu(), w_expert)
    assert torch.equal(slot.long().cpu(), w_slot)
    n = w_source.numel()
    assert torch.equal(source[:n].long().cpu(), w_source)
    assert bool((source[n:] == 0x5A).all())              # behind the last group: as they were
    whole = torch.where(part, xd, torch.full_like(xd, NINF)) if renorm else xd
    rel = _tolerance(torch.where(torch.isfinite(whole), whole, torch.full_like(whole, -1e4)), p, x.shape[1]).gather(1, order)
    _within(gate.cpu(), w_gate, rel * w_gate + 2.0 ** -126, "gate")


SIZES = [(0, 4, 2), (1, 1, 1), (1, 8, 2), (3, 5, 5), (4, 64, 8), (63, 63, 3), (64, 65, 6), (65, 64, 1), (200, 128, 8), (130, 200, 7),
         (1000, 256, 4), (300, 300, 10), (77, 1024, 64), (5000, 8, 2), (16384, 64, 8), (16385, 16, 3), (40000, 7, 2),
         (129, 33, 33)]


@pytest.mark.parametrize("renorm", [False, True], ids=["all", "chosen"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_routing(size, dtype, renorm):
    T, E, k = size
    for off, ties in ((0, True), (1, False)):
        x = _logits(T, E, dtype, 40 + off, ties)
        _check(x, k, renorm, _call(x, k, dtype, renorm, off))


@pytest.mark.parametrize("renorm", [False, True], ids=["all", "chosen"])
@pytest.mark.parametrize("size", [(70, 64, 8), (300, 130, 4), (6, 5, 3), (20000, 64, 2)], ids=str)
def test_masked_logits(size, renorm):
    # experts that a token may not use, tokens left with fewer than k, and with none
    torch = _t()
    T, E, k = size
    x = _logits(T, E, "f32", 44)
    x[torch.empty(T, E, device="cuda").uniform_(generator=_gen(45)) < 0.3] = NINF
    x[1::3, k // 2:] = NINF
    x[2::5] = NINF
    x[T // 2:T // 2 + T // 8] = NINF
    _check(x, k, renorm, _call(x, k, "f32", renorm))


@pytest.mark.parametrize("renorm", [False, True], ids=["all", "chosen"])
def test_nan_and_infinite_logits(renorm):
    torch = _t()
    T, E, k = 8, 70, 4
    x = _logits(T, E, "f32", 46, ties=False)
    x[1, 5], x[2, 66], x[3] = float("nan"), float("inf"), float("nan")
    x[4, 3], x[4, 7] = float("inf"), NINF
    x[5] = torch.finfo(torch.float32).min                # a mask of the lowest value: equal logits
    x[6, 1] = torch.finfo(torch.float32).max
    _, gate, expert, slot, source, offsets = _call(x, k, "f32", renorm)
    w_expert, w_slot, w_source, w_offsets, *_ = _want(x.double().cpu(), k, renorm)
    assert torch.equal(expert.long().cpu(), w_expert) and torch.equal(slot.long().cpu(), w_slot)
    assert torch.equal(offsets.long().cpu(), w_offsets)
    assert 5 not in expert[1].tolist() and expert[2, 0] == 66 and bool((expert[3] == -1).all())
    nan = torch.isnan(gate)
    assert bool(nan[[1, 2, 4]].all()) and not bool(nan[[0, 3, 5, 6, 7]].any())
    assert bool((gate[3] == 0).all())
    assert expert[5].tolist() == [0, 1, 2, 3]
    assert bool((gate[5] == (1 / k if renorm else torch.tensor(1.0) / E)).all())
    assert gate[6].tolist() == [1.0, 0.0, 0.0, 0.0]
    # and the gradients of exactly these rows
    d = torch.empty_like(x)
    with spg.Router(T, E, k, "f32", renormalise=renorm) as plan:
        plan.backward(x, expert, torch.ones_like(gate), d)
    nan = torch.isnan(d)
    chosen = torch.zeros(T, E, dtype=torch.bool, device="cuda").scatter_(1, expert.clamp(min=0).long(), expert >= 0)
    assert bool(nan[[1, 2, 4]][chosen[[1, 2, 4]]].all())
    assert not bool(nan[[0, 3, 5, 6, 7]].any()) and bool((d[3] == 0).all())


def _want_back(x, expert, dgate, renorm):
    torch = _t()
    x, dgate = x.double(), dgate.double()
    live = expert >= 0
    index = expert.clamp(min=0).long()
    part = torch.zeros_like(x).scatter_add_(1, index, live.double()) > 0      # -1 shares column 0
    d = torch.zeros_like(x)
    d.scatter_add_(1, index, torch.where(live, dgate, torch.zeros_like(dgate)))
    some = live.any(1, keepdim=True)
    share = torch.where(part, x, torch.full_like(x, NINF)) if renorm else x
    p = torch.where(some, torch.softmax(torch.where(some, share, torch.zeros_like(x)), 1), torch.zeros_like(x))
    inner = (p * d).sum(1, keepdim=True)
    return p * (d - inner), p, d, share


@pytest.mark.parametrize("renorm", [False, True], ids=["all", "chosen"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_backward(size, dtype, renorm):
    torch = _t()
    T, E, k = size
    x = _logits(T, E, dtype, 47)
    if T > 8 and E > k:
        x[T // 2:T // 2 + 3] = NINF
        x[T - 2, 1:] = NINF
    _, _, expert, _, _, _ = _call(x, k, dtype, renorm)
    dgate = _normal(_gen(48), (T, k), 1.0)
    dgate[expert < 0] = float("nan")                     # not read
    out = Buf((T, E), _dt(dtype), 1)
    with spg.Router(T, E, k, dtype, renormalise=renorm) as plan:
        plan.backward(x, expert, dgate, out.t)
    torch.cuda.synchronize()
    want, p, d, share = _want_back(x, expert, torch.nan_to_num(dgate), renorm)
    rel = _tolerance(torch.where(torch.isfinite(share), share, torch.full_like(share, -1e4)), p, E)
    # d - inner, inner a sum of p d
    inner = (p * d).abs().sum(1, keepdim=True)
    tol = p * ((rel + 3 * U32) * (d.abs() + inner) + ((p * d).abs() * (rel + U32)).sum(1, keepdim=True) + (E / 64 + 9) * U32 * inner)
    _within(out.t, want, 1.01 * tol + _half_ulp(dtype) * want.abs() + _tiny(dtype) + 2.0 ** -126, "dlogits")
    assert out.intact()


@pytest.mark.parametrize("renorm", [False, True], ids=["all", "chosen"])
def test_gradient_against_differences(renorm):
    # of the 64-bit gates with the choice held fixed, as between two steps that choose alike
    torch = _t()
    T, E, k, h = 20, 40, 5, 1e-4
    x = _logits(T, E, "f32", 49, ties=False)
    _, gate, expert, *_ = _call(x, k, "f32", renorm)
    dgate = _normal(_gen(50), (T, k), 1.0)
    d = torch.empty_like(x)
    with spg.Router(T, E, k, "f32", renormalise=renorm) as plan:
        plan.backward(x, expert, dgate, d)

    def loss(v):
        part = torch.zeros_like(v, dtype=torch.bool).scatter_(1, expert.long(), True)
        p = torch.softmax(torch.where(part, v, torch.full_like(v, NINF)) if renorm else v, 1)
        return (p.gather(1, expert.long()) * dgate.double()).sum()

    for i in range(4):
        step = _normal(_gen(51 + i), (T, E), 1.0).double()
        want = float((loss(x.double() + h * step) - loss(x.double() - h * step)) / (2 * h))
        got = float((d.double() * step).sum())
        # the third derivative of a softmax along a step is below its size to the third power
        tol = 2.0 ** -17 * float((d.double().abs() * step.abs()).sum()) + h * h * float(step.abs().max()) ** 3 * float(dgate.abs().sum()) + 1e-9
        assert abs(got - want) <= tol, (i, got, want, tol)


def _slots(T, k, rows, seed, empty=0.2):
    """Different rows in random order, some places empty, some out of range."""
    torch = _t()
    g = _gen(seed)
    slot = torch.randperm(max(rows, T * k), generator=g, device="cuda")[: T * k].view(T, k)
    slot = torch.where(slot < rows, slot, -1)
    slot[torch.empty(T, k, device="cuda").uniform_(generator=g) < empty] = -1
    if T > 2:
        slot[1] = -1
        slot[2, 0] = rows
        slot[0, k - 1] = -7
    return slot.int()


COMBINE = [(1, 1, 1, 1), (1, 2, 2, 40), (4, 8, 32, 2048), (5, 3, 20, 7), (3, 64, 192, 9), (33, 2, 66, 129), (70, 6, 500, 1001),
           (300, 2, 600, 4096), (9, 4, 30, 20000), (2000, 5, 9000, 24), (8, 1, 4, 260)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("size", COMBINE, ids=str)
def test_combine(size, dtype):
    torch = _t()
    T, k, rows, N = size
    e, tiny = _half_ulp(dtype), _tiny(dtype)
    for i, (off, gated) in enumerate(((0, True), (1, False), (2, True))):
        y = Buf((rows, N), _dt(dtype), off, _normal(_gen(60 + i), (rows, N), 1.0).to(_dt(dtype)))
        do = Buf((T, N), _dt(dtype), off, _normal(_gen(70 + i), (T, N), 0.3).to(_dt(dtype)))
        slot = _slots(T, k, rows, 80 + i)
        bad = (slot < 0) | (slot >= rows)
        gate = _normal(_gen(90 + i), (T, k), 1.0) if gated else None
        if gated:
            gate[bad] = float("nan")                     # contributes nothing, whatever it is
        out, dy = Buf((T, N), _dt(dtype), off), Buf((rows, N), _dt(dtype), off)
        dgate = Buf((T, k), torch.float32)
        with spg.Combine(T, k, rows, N, dtype) as plan:
            plan(y.t, slot, gate, out.t)
            plan.backward(do.t, y.t, slot, gate, dy.t, dgate.t)
        torch.cuda.synchronize()
        g = torch.where(bad, torch.zeros(T, k, device="cuda"), gate if gated else torch.ones(T, k, device="cuda")).double()
        at = torch.where(bad, torch.zeros_like(slot), slot).long()
        rowsd = y.t.double()[at] * (~bad)[:, :, None]
        want = (g[:, :, None] * rowsd).sum(1)
        mag = (g[:, :, None] * rowsd).abs().sum(1)
        _within(out.t, want, k * U32 * mag + e * (want.abs() + k * U32 * mag) + tiny, "out")
        # each element: one product rounded to fp32, then to the type
        named = torch.zeros(rows, dtype=torch.bool, device="cuda")
        named[at[~bad]] = True
        wdy = torch.zeros(rows, N, dtype=torch.double, device="cuda")
        wdy[at[~bad]] = (g[:, :, None] * do.t.double()[:, None, :])[~bad]
        _within(dy.t[named], wdy[named], (e + 1.01 * U32) * wdy[named].abs() + tiny, "dY")
        untouched = dy.t[~named].view(torch.int16 if dtype != "f32" else torch.int32)
        assert bool((untouched == 0x5A).all())
        wdg = (rowsd * do.t.double()[:, None, :]).sum(2)
        mag = (rowsd * do.t.double()[:, None, :]).abs().sum(2)
        # chains of N / 64 + 16 additions at most
        _within(dgate.t, wdg, (N / 64 + 16) * U32 * mag + 2.0 ** -140, "dgate")
        assert all(b.intact() for b in (y, do, out, dy, dgate))


def test_combine_without_gate_gradients_and_empty():
    torch = _t()
    T, k, rows, N = 40, 2, 80, 136
    do = _normal(_gen(1), (T, N), 1.0).bfloat16()
    slot = torch.randperm(80, generator=_gen(2), device="cuda").view(T, k).int()
    gate = _normal(_gen(3), (T, k), 1.0)
    dy, again = torch.zeros(rows, N, device="cuda", dtype=torch.bfloat16), torch.zeros(rows, N, device="cuda", dtype=torch.bfloat16)
    dg = torch.empty(T, k, device="cuda")
    with spg.Combine(T, k, rows, N, "bf16") as plan:
        plan.backward(do, None, slot, gate, dy)
        plan.backward(do, dy, slot, gate, again, dg)
    assert torch.equal(dy, again)
    with spg.Combine(T, k, 0, N, "bf16") as plan:        # no rows at all
        out = torch.full((T, N), 3.0, device="cuda", dtype=torch.bfloat16)
        none = torch.empty(0, N, device="cuda", dtype=torch.bfloat16)
        plan(none, slot, gate, out)
        plan.backward(do, none, slot, gate, none, dg)
    assert bool((out == 0).all()) and bool((dg == 0).all())
    with spg.Combine(0, k, rows, N, "bf16") as plan:
        e = torch.empty(0, N, device="cuda", dtype=torch.bfloat16)
        i = torch.empty(0, k, device="cuda", dtype=torch.int32)
        plan(dy, i, None, e)


def test_infinite_rows_stay_where_they_are():
    # a row that no slot names may hold anything; a named infinity reaches its token alone
    torch = _t()
    T, k, rows, N = 6, 2, 14, 72
    y = _normal(_gen(4), (rows, N), 1.0).half()
    y[12] = float("nan")
    y[3] = float("inf")
    slot = torch.arange(12, device="cuda", dtype=torch.int32).view(T, k)
    out = torch.empty(T, N, device="cuda", dtype=torch.float16)
    with spg.Combine(T, k, rows, N, "f16") as plan:
        plan(y, slot, None, out)
    assert bool(torch.isinf(out[1]).all()) and bool(torch.isfinite(out[[0, 2, 3, 4, 5]]).all())
