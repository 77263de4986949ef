"""GPU tests of the operators around experts at sizes whose byte offsets pass 32 bits: matrices of
more than 4 GiB, groups that start behind them, tokens gathered from more than 2 GiB, logits of
4 GiB.  The formulas in 64 bits are checked at rows from the start, the middle and the end (all
of a row); tolerances as in test_gpu_norm.py, test_gpu_route.py and test_gpu_grouped.py."""

import pytest

import software_pipelined_tiled_gemm_amd as spg
from tests.test_gpu_feed_forward import U32, _gen, _half_ulp, _t, _tiny, _within, _workspace
from tests.test_gpu_grouped import _as_kn, _check_rows, _check_weight
from tests.test_gpu_norm import _check_forward

pytestmark = pytest.mark.gpu


def _rand(shape, std, seed, dtype):
    torch = _t()
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=_gen(seed))


def _some(rows, n=64):
    torch = _t()
    return torch.tensor(sorted({0, 1, rows // 2, rows - 2, rows - 1} | {rows * i // n for i in range(n)}), device="cuda")


def test_norm():
    torch = _t()
    M, K = 530000, 4100                                  # 4.3 GB
    x, dy = _rand((M, K), 1.0, 1, torch.bfloat16), _rand((M, K), 0.3, 2, torch.bfloat16)
    w, b = _rand((K,), 1.0, 3, torch.float32), _rand((K,), 1.0, 4, torch.float32)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = (torch.empty(M, device="cuda") for _ in range(2))
    dw, db = torch.empty_like(w), torch.empty_like(b)
    at = _some(M)
    with spg.LayerNorm(M, K, "bf16", "f32") as plan:
        plan(x, w, b, y, mean, rstd)
        plan.backward(dy, x, w, mean, rstd, dx, dw, db, workspace=_workspace(plan.workspace_bytes()))
    torch.cuda.synchronize()
    _check_forward(x[at], w, b, y[at], mean[at], rstd[at], "bf16")
    m, r = mean[at].double()[:, None], rstd[at].double()[:, None]
    n = (x[at].double() - m) * r
    g = dy[at].double() * w.double()
    s1, s2 = g.mean(1, keepdim=True), (g * n).mean(1, keepdim=True)
    want = r * (g - s1 - n * s2)
    # n is off by 3 u |n| and the subtraction, each sum by D + 3 roundings of its magnitudes, the rest by 4
    D = K / 64 + 16
    en = 3 * U32 * n.abs() + r * U32 * (x[at].double() - m).abs()
    e1 = (D + 3) * U32 * g.abs().mean(1, keepdim=True)
    e2 = ((D + 4) * U32 * (g * n).abs() + g.abs() * en).mean(1, keepdim=True)
    inner = r * (e1 + n.abs() * e2 + s2.abs() * en + 5 * U32 * (g.abs() + s1.abs() + (n * s2).abs()))
    _within(dx[at], want, 1.01 * inner + _half_ulp("bf16") * (want.abs() + inner) + _tiny("bf16"), "dX")
    sw, sb, mw, mb = (torch.zeros(K, dtype=torch.double, device="cuda") for _ in range(4))
    for i in range(0, M, 50000):
        d = dy[i:i + 50000].double()
        t = d * ((x[i:i + 50000].double() - mean[i:i + 50000].double()[:, None]) * rstd[i:i + 50000].double()[:, None])
        sw += t.sum(0)
        mw += t.abs().sum(0)
        sb += d.sum(0)
        mb += d.abs().sum(0)
    # chains of at most all rows of a workgroup's waves (M / 256) and the sums of them
    _within(dw, sw, (M / 256 + 1024) * U32 * mw, "dweight")
    _within(db, sb, (M / 256 + 1024) * U32 * mb, "dbias")


def test_routing():
    torch = _t()
    T, E, k = 1 << 24, 64, 8
    x = _rand((T, E), 2.0, 5, torch.float32)
    gate = torch.empty(T, k, device="cuda")
    expert, slot = (torch.empty(T, k, dtype=torch.int32, device="cuda") for _ in range(2))
    source, offsets = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (T * k, E + 1))
    dl = torch.empty_like(x)
    dgate = _rand((T, k), 1.0, 6, torch.float32)
    with spg.Router(T, E, k, "f32") as plan:
        plan(x, gate, expert, slot, source, offsets, workspace=_workspace(plan.workspace_bytes()))
        plan.backward(x, expert, dgate, dl)
    torch.cuda.synchronize()
    # a choice in its place, each place once, the groups in order
    flat = expert.view(-1)
    count = torch.bincount(flat, minlength=E)
    assert torch.equal(offsets[1:].long(), count.cumsum(0)) and int(offsets[0]) == 0
    place = slot.view(-1).long()
    by = torch.full((T * k,), -1, dtype=torch.int32, device="cuda")
    by[place] = torch.arange(T * k, dtype=torch.int32, device="cuda")
    assert bool((by >= 0).all())
    assert torch.equal(source, by // k)
    sorted_experts = flat[by.long()]
    assert bool((sorted_experts[1:] >= sorted_experts[:-1]).all())
    same = sorted_experts[1:] == sorted_experts[:-1]
    assert bool((by[1:] > by[:-1])[same].all())
    at = _some(T, 4096)
    xd = x[at].double()
    order = xd.sort(dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(expert[at].long(), order)
    p = torch.softmax(xd, 1)
    z = (xd - xd.amax(1, keepdim=True)).abs()
    rel = (z + (p * z).sum(1, keepdim=True) + E / 64 + 8 + 6) * U32 * 1.01
    _within(gate[at], p.gather(1, order), (rel * p).gather(1, order) + 2.0 ** -126, "gate")
    d = torch.zeros_like(p).scatter_(1, order, dgate[at].double())
    s, ms = (p * d).sum(1, keepdim=True), (p * d).abs().sum(1, keepdim=True)
    es = (rel * (p * d).abs()).sum(1, keepdim=True) + (E / 64 + 10) * U32 * ms
    want = p * (d - s)
    _within(dl[at], want, 1.01 * (rel * want.abs() + p * es + 3 * U32 * p * (d.abs() + s.abs())) + 2.0 ** -126, "dlogits")


def test_combine():
    torch = _t()
    T, k, N = 300000, 2, 4100
    rows = T * k                                         # Y: 4.9 GB
    y = _rand((rows, N), 1.0, 7, torch.bfloat16)
    do = _rand((T, N), 0.3, 8, torch.bfloat16)
    slot = torch.randperm(rows, generator=_gen(9), device="cuda").int().view(T, k)
    gate = _rand((T, k), 1.0, 10, torch.float32)
    out, dy, dgate = torch.empty_like(do), torch.empty_like(y), torch.empty_like(gate)
    with spg.Combine(T, k, rows, N, "bf16") as plan:
        plan(y, slot, gate, out)
        plan.backward(do, y, slot, gate, dy, dgate)
    torch.cuda.synchronize()
    at = _some(T, 1024)
    e, tiny = _half_ulp("bf16"), _tiny("bf16")
    g, rowsd = gate[at].double(), y[slot[at].long()].double()
    parts = g[:, :, None] * rowsd
    want, mag = parts.sum(1), parts.abs().sum(1)
    _within(out[at], want, k * U32 * mag + e * (want.abs() + k * U32 * mag) + tiny, "out")
    dd = do[at].double()[:, None, :]
    want = g[:, :, None] * dd
    _within(dy[slot[at].long()], want, (e + 1.01 * U32) * want.abs() + tiny, "dY")
    _within(dgate[at], (rowsd * dd).sum(2), (N / 64 + 16) * U32 * (rowsd * dd).abs().sum(2), "dgate")


# (rows, N, K, tokens): X, then Y beyond 4 GiB; tokens whose matrix is more than 2 GiB, which rows
# cannot address in place
ROWS = [(330000, 136, 6664, None), (270000, 8200, 72, None), (3000, 264, 2056, 560000), (270000, 8200, 72, 500)]


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("size", ROWS, ids=str)
def test_many_rows(size, layout):
    torch = _t()
    rows, N, K, tokens = size
    dt = torch.bfloat16
    o = [2, rows // 3, rows // 3, rows - 700, rows - 3]
    E = len(o) - 1
    offsets = torch.tensor(o, dtype=torch.int32, device="cuda")
    x = _rand((rows if tokens is None else tokens, K), 1.0, 11, dt)
    shape = (E, N, K) if layout == "nk" else (E, K, N)
    w = _rand(shape, K ** -0.5, 12, dt)
    dy = _rand((rows, N), 0.3, 13, dt)
    source = None if tokens is None else torch.randint(0, tokens, (rows,), generator=_gen(14), device="cuda").int()
    y, dx, dw = torch.zeros_like(dy), torch.zeros(rows, K, dtype=dt, device="cuda"), torch.zeros_like(w)
    with spg.GroupedGemm(rows, N, K, E, "bf16", layout, tokens=tokens) as plan:
        plan(x, w, offsets, y, source=source, workspace=_workspace(plan.workspace_bytes(backward=False)))
        plan.backward(dy, x, w, offsets, dx, dw, source=source, workspace=_workspace(plan.workspace_bytes()))
    torch.cuda.synchronize()
    for e in (0, 2, 3):
        n = o[e + 1] - o[e]
        r = _some(n) + o[e]
        xs = x[r] if source is None else x[source[r].long()]
        wd = _as_kn(w[e], layout)
        _check_rows(xs, wd, y[r], "bf16", f"Y of group {e}")
        _check_rows(dy[r], wd.t().contiguous(), dx[r], "bf16", f"dX of group {e}")
    r = slice(o[3], o[4])                                # the last rows of all
    xs = x[r] if source is None else x[source[r].long()]
    _check_weight(xs, dy[r], dw[3], "bf16", layout, "dW of the last group")
    assert bool((dw[1] == 0).all())
    assert bool((y[:2] == 0).all()) and bool((y[-3:] == 0).all()) and bool((dx[-3:] == 0).all())


@pytest.mark.parametrize("layout", ["nk", "kn"])
def test_many_matrices(layout):
    # 5 GB of each matrix: groups of few rows, the last ones' matrices behind 4 GiB
    torch = _t()
    N, K, E = 4104, 2048, 300
    dt = torch.bfloat16
    counts = [(7 * i) % 5 for i in range(E - 2)] + [70, 3]
    o = [sum(counts[:i]) for i in range(E + 1)]
    rows = o[-1]
    offsets = torch.tensor(o, dtype=torch.int32, device="cuda")
    shape = (E, N, K) if layout == "nk" else (E, K, N)
    x, w, dy = _rand((rows, K), 1.0, 15, dt), _rand(shape, K ** -0.5, 16, dt), _rand((rows, N), 0.3, 17, dt)
    y, dx, dw = torch.zeros_like(dy), torch.zeros_like(x), torch.full_like(w, float("nan"))
    with spg.GroupedGemm(rows, N, K, E, "bf16", layout) as plan:
        plan(x, w, offsets, y, workspace=_workspace(plan.workspace_bytes(backward=False)))
        plan.backward(dy, x, w, offsets, dx, dw, workspace=_workspace(plan.workspace_bytes()))
    torch.cuda.synchronize()
    for e in (1, 150, E - 4, E - 3, E - 2, E - 1):
        r = slice(o[e], o[e + 1])
        wd = _as_kn(w[e], layout)
        _check_rows(x[r], wd, y[r], "bf16", f"Y of group {e}")
        _check_rows(dy[r], wd.t().contiguous(), dx[r], "bf16", f"dX of group {e}")
        _check_weight(x[r], dy[r], dw[e], "bf16", layout, f"dW of group {e}")
    assert bool((dw[0] == 0).all()) and bool(torch.isfinite(dw[-6:]).all())


@pytest.mark.parametrize("layout", ["nk", "kn"])
def test_more_rows_than_small_tiles_launch(layout):
    # row tiles of 64 rows would be more workgroups than a launch holds
    torch = _t()
    rows, N, K = 600_000_000, 8, 8
    o = [1, rows // 2 + 3, rows // 2 + 3, rows - 2]
    offsets = torch.tensor(o, dtype=torch.int32, device="cuda")
    x = _rand((rows, K), 1.0, 18, torch.bfloat16)
    w = _rand((3, N, K) if layout == "nk" else (3, K, N), 0.3, 19, torch.bfloat16)
    y, dx = torch.zeros_like(x), torch.zeros_like(x)
    with spg.GroupedGemm(rows, N, K, 3, "bf16", layout) as plan:
        plan(x, w, offsets, y, workspace=_workspace(plan.workspace_bytes(backward=False)))
        plan.backward(x, None, w, offsets, dx, None, workspace=_workspace(plan.workspace_bytes()))
    torch.cuda.synchronize()
    for e in (0, 2):
        n = o[e + 1] - o[e]
        r = _some(n, 4096) + o[e]
        wd = _as_kn(w[e], layout)
        _check_rows(x[r], wd, y[r], "bf16", f"Y of group {e}")
        _check_rows(x[r], wd.t().contiguous(), dx[r], "bf16", f"dX of group {e}")
    assert bool((y[0] == 0).all()) and bool((y[-2:] == 0).all()) and bool((dx[-2:] == 0).all())
