"""GPU tests of calls on the products by group that their documentation allows and that are far
from the ordinary: no tokens, one token for every row, source places nobody wrote, one plan on
two streams at once, and a captured call whose groups change from replay to replay (the
last round's parts among them)."""

import pytest

import software_pipelined_tiled_gemm_amd as spg
from tests.test_gpu_feed_forward import _gen, _normal, _t, _workspace
from tests.test_gpu_grouped import _as_kn, _check_rows, _check_weight, _weights

pytestmark = pytest.mark.gpu


def _i32(values):
    torch = _t()
    return torch.tensor(values, dtype=torch.int32, device="cuda")


# streamed, tiled, register-staged, without MFMAs
SIZES = [(3, 48, 64), (300, 264, 512), (300, 131, 77), (70, 6, 5)]


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_no_tokens(size, layout):
    torch = _t()
    rows, N, K = size
    o = [0, rows // 3, rows // 3, rows]
    E, offsets, source = 3, _i32([0, rows // 3, rows // 3, rows]), torch.zeros(rows, dtype=torch.int32, device="cuda")
    x = torch.empty(0, K, dtype=torch.bfloat16, device="cuda")
    w = [_weights(E, N, K, "bf16", layout, 1 + i, 0).t for i in (0, 1)]
    dy = _normal(_gen(4), (rows, N), 0.3).bfloat16()
    y, h, g, u = (torch.full_like(dy, 7) for _ in range(4))
    dx = torch.full((rows, K), 7.0, dtype=torch.bfloat16, device="cuda")
    dw, dwg, dwu = (torch.full_like(w[0], 7) for _ in range(3))
    with spg.GroupedGemm(rows, N, K, E, "bf16", layout, tokens=0) as plan:
        ws = _workspace(plan.workspace_bytes())
        plan(x, w[0], offsets, y, source=source, workspace=ws)
        plan.backward(dy, x, w[0], offsets, dx, dw, source=source, workspace=ws)
    with spg.GroupedGated(rows, N, K, E, "bf16", layout, "silu", tokens=0) as plan:
        ws = _workspace(plan.workspace_bytes())
        plan(x, *w, offsets, h, source=source, G=g, U=u, workspace=ws)
        plan.backward(dy, x, *w, g, u, offsets, torch.empty_like(dx), dwg, dwu, source=source, workspace=ws)
    for t in (y, h, g, u, dw, dwg, dwu):
        assert bool((t == 0).all())
    for e in range(E):                                   # the rows' own gradients do not ask for tokens
        r = slice(o[e], o[e + 1])
        if o[e] < o[e + 1]:
            _check_rows(dy[r], _as_kn(w[0][e], layout).t().contiguous(), dx[r], "bf16", "dX")


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("size", SIZES + [(700, 1024, 264)], ids=str)
def test_one_token_for_every_row(size, layout):
    torch = _t()
    rows, N, K = size
    o = [0, rows // 2, rows - 1]                         # the last row belongs to no group, its source is anything
    offsets = _i32(o)
    source = torch.full((rows,), 5, dtype=torch.int32, device="cuda")
    source[-1] = -2 ** 31
    x = _normal(_gen(1), (9, K), 1.0).bfloat16()
    w = _weights(2, N, K, "bf16", layout, 2, 0).t
    dy = _normal(_gen(4), (rows, N), 0.3).bfloat16()
    y, dw = torch.full_like(dy, 7), torch.zeros_like(w)
    dx = torch.full((rows, K), 7.0, dtype=torch.bfloat16, device="cuda")
    with spg.GroupedGemm(rows, N, K, 2, "bf16", layout, tokens=9) as plan:
        plan(x, w, offsets, y, source=source, workspace=_workspace(plan.workspace_bytes(backward=False)))
        plan.backward(dy, x, w, offsets, dx, dw, source=source, workspace=_workspace(plan.workspace_bytes()))
    xs = x[5:6].expand(rows, K)
    for e in range(2):
        r = slice(o[e], o[e + 1])
        _check_rows(xs[r], _as_kn(w[e], layout), y[r], "bf16", "Y")
        _check_weight(xs[r], dy[r], dw[e], "bf16", layout, "dW")
    assert bool((y[-1] == 7).all()) and bool((dx[-1] == 7).all())


def _calls(plan, x, w, offsets, source, dh, ws, stream=None):
    """A gated pass forward and back, into fresh outputs (made before the call, on the current stream)."""
    torch = _t()
    h, g, u = (torch.zeros_like(dh) for _ in range(3))
    dx = torch.zeros(dh.shape[0], x.shape[1], dtype=dh.dtype, device="cuda")
    dwg, dwu = (torch.zeros_like(t) for t in w)

    def go(stream=None):
        plan(x, *w, offsets, h, source=source, G=g, U=u, workspace=ws, stream=stream)
        plan.backward(dh, x, *w, g, u, offsets, dx, dwg, dwu, source=source, workspace=ws, stream=stream)
    return go, (h, g, u, dx, dwg, dwu)


@pytest.mark.parametrize("size", [(300, 264, 136), (2600, 2304, 4160)], ids=str)
def test_one_plan_on_two_streams(size):
    torch = _t()
    rows, N, K = size
    E, tokens = 3, 500
    inputs = []
    with spg.GroupedGated(rows, N, K, E, "bf16", "nk", "silu", tokens=tokens) as plan:
        for i in range(2):
            x = _normal(_gen(10 * i + 1), (tokens, K), 1.0).bfloat16()
            w = [_weights(E, N, K, "bf16", "nk", 10 * i + 2 + j, 0).t for j in (0, 1)]
            dh = _normal(_gen(10 * i + 4), (rows, N), 0.3).bfloat16()
            offsets = _i32([0, rows // (i + 2), rows // 2 + 7, rows])
            source = torch.randint(0, tokens, (rows,), generator=_gen(10 * i + 5), device="cuda").int()
            inputs.append((x, w, offsets, source, dh))
        want = []
        for a in inputs:
            go, out = _calls(plan, *a, _workspace(plan.workspace_bytes()))
            go()
            want.append(out)
        streams = [torch.cuda.Stream() for _ in inputs]
        runs = [_calls(plan, *a, _workspace(plan.workspace_bytes())) for a in inputs]
        torch.cuda.synchronize()
        for _ in range(3):
            for (go, _), s in zip(runs, streams):
                go(s)
        torch.cuda.synchronize()
    for (_, got), exp in zip(runs, want):
        assert all(torch.equal(p, q) for p, q in zip(got, exp))


@pytest.mark.parametrize("size", [(300, 264, 136), (40, 520, 320), (3300, 2304, 4160)], ids=str)
def test_groups_change_between_replays(size):
    torch = _t()
    rows, N, K = size
    E, tokens = 4, 600
    x = _normal(_gen(1), (tokens, K), 1.0).bfloat16()
    w = [_weights(E, N, K, "bf16", "nk", 2 + j, 0).t for j in (0, 1)]
    dh = _normal(_gen(4), (rows, N), 0.3).bfloat16()
    cuts = [[0, rows, rows, rows, rows], [0, 1, rows // 2, rows // 2, rows], [3, 3, 3, 3, 3], [0, rows // 4, rows // 2, rows - 9, rows],
            [5, rows // 3, rows // 3 + 1, rows - 1, rows - 1]]
    sources = [torch.randint(-1, tokens + 1, (rows,), generator=_gen(20 + i), device="cuda").int() for i in range(len(cuts))]
    offsets, source = _i32(cuts[0]), sources[0].clone()
    with spg.GroupedGated(rows, N, K, E, "bf16", "nk", "silu", tokens=tokens) as plan:
        ws = _workspace(plan.workspace_bytes())
        go, out = _calls(plan, x, w, offsets, source, dh, ws)

        def fresh(i):
            offsets.copy_(_i32(cuts[i])), source.copy_(sources[i])
            for t in out:
                t.zero_()
            ws.fill_(0xFF)

        want = []
        for i in range(len(cuts)):
            fresh(i)
            go()
            want.append([t.clone() for t in out])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            go(torch.cuda.current_stream())
        for i in (2, 0, 3, 1, 4, 4, 0):
            fresh(i)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(out, want[i])), i
            fresh((i + 1) % len(cuts))
            go()                                         # the program's own call between the replays
            assert all(torch.equal(p, q) for p, q in zip(out, want[(i + 1) % len(cuts)])), i
