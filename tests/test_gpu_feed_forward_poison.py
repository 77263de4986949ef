"""The feed-forward operators on the poisoned library: in it every ring slot starts as NaN
patterns and becomes NaN again the moment its release barrier has passed, so a fragment read
that the barriers do not cover gives NaN (int8: -1) in the result.  Results have to be finite
and bitwise those of the production library, over both copy modes, split and merged launches,
and k-tile counts around the rings' depths; test_gpu_feed_forward_forms.py does the same for
every kernel that the choice of tiles launches."""

import pytest

import software_pipelined_tiled_gemm_amd as spg

pytestmark = pytest.mark.gpu

# (M, N, K): 64x64 .. 256x256 tiles, one to many k-tiles, split reductions, ragged rows
SIZES = [(64, 64, 64), (40, 200, 128), (65, 264, 192), (96, 512, 2048), (300, 1024, 448), (300, 2731, 1001),
         (511, 1365, 500), (512, 4096, 320), (1024, 2048, 1024), (2048, 4096, 832), (1300, 2051, 1003),
         (150, 262, 1002), (2100, 2050, 334)]


def _both(fn, monkeypatch):
    """fn() with the production library, then with the poisoned one."""
    want = fn()
    poison = spg.poison_lib()
    with monkeypatch.context() as m:
        m.setattr(spg, "_lib", poison)
        got = fn()
    return want, got


def _same(want, got):
    import torch
    for i, (p, q) in enumerate(zip(want, got)):
        assert bool(torch.isfinite(q.float()).all()), i
        assert torch.equal(p, q), i


def _rand(gen, shape, std, dtype):
    import torch
    return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=gen).to(dtype)


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_gated_pass(size, layout, monkeypatch):
    import torch
    M, N, K = size
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    dt = torch.bfloat16
    w = (N, K) if layout == "nk" else (K, N)
    x, dh = _rand(gen, (M, K), 1.0, dt), _rand(gen, (M, N), 0.3, dt)
    wg, wu = _rand(gen, w, K ** -0.5, dt), _rand(gen, w, K ** -0.5, dt)

    def step():
        h, g, u = (torch.zeros(M, N, dtype=dt, device="cuda") for _ in range(3))
        grads = [torch.zeros_like(t) for t in (x, wg, wu)]
        with spg.Gated(M, N, K, "bf16", layout, "silu") as plan:
            ws = torch.zeros(max(1, plan.workspace_bytes()), dtype=torch.uint8, device="cuda")
            plan(x, wg, wu, h, G=g, U=u, workspace=ws)
            plan.backward(dh, x, wg, wu, g, u, *grads, workspace=ws)
        torch.cuda.synchronize()
        return [h, g, u, *grads]

    _same(*_both(step, monkeypatch))


@pytest.mark.parametrize("act", ["none", "gelu_tanh"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_quantized_product(size, act, monkeypatch):
    import torch
    M, N, K = size
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    a, b, b2 = (torch.randint(-128, 128, s, generator=gen, device="cuda", dtype=torch.int32).to(torch.int8)
                for s in ((M, K), (N, K), (N, K)))
    sa, sb = torch.ones(M, device="cuda"), torch.full((N,), 2e-4 * K ** -0.5, device="cuda")

    def step():
        c = torch.zeros(M, N, device="cuda")
        with spg.QuantizedGemm(M, N, K, "f32", act) as plan:
            ws = torch.zeros(max(1, plan.workspace_bytes()), dtype=torch.uint8, device="cuda")
            plan(a, sa, b, sb, c, B2=b2 if act != "none" else None, scale_b2=sb if act != "none" else None, workspace=ws)
        torch.cuda.synchronize()
        return [c]

    _same(*_both(step, monkeypatch))
