"""The operators of a mixture of experts together, as a block calls them: forward and backward
against the formulas in 64 bits, captured into a graph, on another stream, through the example."""

import pytest

import software_pipelined_tiled_gemm_amd as spg
from examples import mixture_of_experts as example
from tests.test_gpu_feed_forward import _gen, _normal, _t

pytestmark = pytest.mark.gpu


def _block(tokens=300, model=264, hidden=328, experts=7, choices=3, seed=4):
    return example.ExpertsBlock(tokens, model, hidden, experts, choices, seed=seed)


def _reference(block, x, expert):
    """The block in 64 bits with the choice of experts held fixed; x and the weights get gradients."""
    torch = _t()
    w = {k: v.double().requires_grad_() for k, v in block.w.items()}
    xd = x.double().requires_grad_()
    c = xd - xd.mean(1, keepdim=True)
    n = c * ((c * c).mean(1, keepdim=True) + 1e-5).rsqrt() * w["norm_w"] + w["norm_b"]
    logits = n @ w["router"].t()
    gate = torch.softmax(logits.gather(1, expert.long()), 1)
    rows = []
    for j in range(expert.shape[1]):
        out = torch.zeros_like(n)
        for e in range(w["gate"].shape[0]):
            at = (expert[:, j] == e).nonzero()[:, 0]
            v = n[at]
            g, u = v @ w["gate"][e].t(), v @ w["up"][e].t()
            out = out.index_copy(0, at, (g * torch.sigmoid(g) * u) @ w["down"][e].t())
        rows.append(out)
    return xd, w, xd + (gate[:, :, None] * torch.stack(rows, 1)).sum(1)


def _relative(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("sizes", [dict(), dict(tokens=1, choices=2), dict(tokens=64, model=200, hidden=130, experts=40, choices=8)],
                         ids=["batch", "token", "many"])
def test_block_against_its_formulas(sizes):
    # Every tensor on a path from x to a gradient is stored in bf16, each time off by at most 2^-8
    # of its values: n, G, U, H, Y, out forward; dY, dH, dG and dU, dX, their sum, dlogits and what
    # comes back from them, the gradient itself backward.  At most 12 lie on one path.
    torch = _t()
    block = _block(**sizes)
    T, D = block.shape[:2]
    x = _normal(_gen(5), (T, D), 1.0).bfloat16()
    dout = _normal(_gen(6), (T, D), 0.2).bfloat16()
    out = block.forward(x).clone()
    dx = block.backward(x, dout)
    xd, w, want = _reference(block, x, block.expert)
    assert _relative(out, want.detach()) <= 7 * 2.0 ** -8
    want.backward(dout.double())
    assert _relative(dx, xd.grad) <= 12 * 2.0 ** -8
    for k in block.NAMES:
        if float(w[k].grad.norm()) > 0:
            assert _relative(block.grad[k], w[k].grad) <= 12 * 2.0 ** -8, k


def test_captured_and_replayed():
    # forward and backward in one graph; between the replays other inputs, the program's own eager
    # work on the same plans and workspace, and synchronizations
    torch = _t()
    block = _block()
    T, D = block.shape[:2]
    x, dout = torch.zeros(T, D, device="cuda", dtype=torch.bfloat16), torch.zeros(T, D, device="cuda", dtype=torch.bfloat16)
    inputs = [(_normal(_gen(10 + i), (T, D), 1.0).bfloat16(), _normal(_gen(20 + i), (T, D), 0.2).bfloat16()) for i in range(4)]

    def step():
        return block.forward(x), block.backward(x, dout)

    def state(dx):
        return [t.clone() for t in (block.out, dx, block.g, block.expert, block.slot, block.offsets,
                                    *(block.grad[k] for k in block.NAMES))]

    eager = []
    for a, b in inputs:
        x.copy_(a), dout.copy_(b)
        _, dx = step()
        eager.append(state(dx))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, dx = step()
    for i in (1, 3, 0, 2, 2):
        x.copy_(inputs[i][0]), dout.copy_(inputs[i][1])
        graph.replay()
        got = state(dx)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, eager[i])), i
        x.copy_(inputs[0][0]), dout.copy_(inputs[0][1])
        _, other = step()
        assert all(torch.equal(p, q) for p, q in zip(state(other), eager[0])), i


def test_two_graphs_share_a_workspace():
    torch = _t()
    block, serve = _block(), _block()
    serve.ws = block.ws if block.ws.numel() >= serve.ws.numel() else serve.ws
    T, D = block.shape[:2]
    x = _normal(_gen(5), (T, D), 1.0).bfloat16()
    dout = _normal(_gen(6), (T, D), 0.2).bfloat16()
    want = block.forward(x).clone(), block.backward(x, dout).clone()
    torch.cuda.synchronize()
    a, b = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(a):
        block.forward(x)
        dx = block.backward(x, dout)
    with torch.cuda.graph(b):
        serve.forward(x)
    for _ in range(3):
        block.out.zero_(), serve.out.zero_()
        b.replay()
        a.replay()
        b.replay()
        torch.cuda.synchronize()
        assert torch.equal(block.out, want[0]) and torch.equal(serve.out, want[0]) and torch.equal(dx, want[1])


def test_on_another_stream():
    torch = _t()
    block = _block()
    T, D = block.shape[:2]
    x = _normal(_gen(5), (T, D), 1.0).bfloat16()
    want = block.forward(x).clone()
    block.out.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = block.forward(x).clone()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    # and named, as an object and as a raw handle
    y = torch.zeros_like(block.n)
    side.wait_stream(torch.cuda.current_stream())
    block.norm(x, None, None, y, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    z = torch.zeros_like(y)
    side.wait_stream(torch.cuda.current_stream())
    block.norm(x, None, None, z, stream=side.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, z) and bool(y.any())


def test_padding_changes_nothing():
    # the same tokens with padding behind them: masked logits, no rows, equal bits
    torch = _t()
    T, E, k, D, N, pad = 90, 6, 2, 136, 72, 38
    logits = _normal(_gen(1), (T + pad, E), 1.0)
    logits[T:] = float("-inf")
    x = _normal(_gen(2), (T + pad, D), 1.0).bfloat16()
    x[T:] = float("nan")
    w = _normal(_gen(3), (E, N, D), 0.1).bfloat16()

    def run(n):
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
        gate, expert, slot, source, offsets = torch.zeros(n, k, device="cuda"), i32(n, k), i32(n, k), i32(n * k), i32(E + 1)
        h, out = (torch.zeros(m, N, dtype=torch.bfloat16, device="cuda") for m in (n * k, n))
        ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
        with spg.Router(n, E, k, "f32") as r, spg.GroupedGated(n * k, N, D, E, tokens=n) as g, spg.Combine(n, k, n * k, N) as c:
            r(logits[:n].contiguous(), gate, expert, slot, source, offsets, workspace=ws)
            g(x[:n].contiguous(), w, w, offsets, h, source=source, workspace=ws)
            c(h, slot, gate, out)
        return out

    full, padded = run(T), run(T + pad)
    assert torch.equal(full, padded[:T]) and bool((padded[T:] == 0).all())


def test_example_runs():
    losses, worst = example.main(tokens=96, model=128, hidden=192, experts=6, choices=2, steps=2)
    assert len(losses) == 2 and all(v == v for v in losses)
    # a served token differs by the roundings alone, unless one flips its choice of experts
    assert worst == worst
