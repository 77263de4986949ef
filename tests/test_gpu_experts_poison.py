"""The products by group on the poisoned library (test_gpu_feed_forward_poison.py has its terms):
results have to be finite and bitwise those of the production library, over both layouts and copy
modes, rows in place and by source, groups that end inside tiles, few rows, one to many k-tiles,
and grids whose last tiles are split along the sum."""

import pytest

import software_pipelined_tiled_gemm_amd as spg
from tests.test_gpu_feed_forward_poison import _both, _rand, _same

pytestmark = pytest.mark.gpu

# rows of the groups, N, K, tokens (None: rows in their groups' order)
CASES = {
    "few": ([1, 0, 5, 17], 264, 512, None),
    "thin": ([30, 20, 0, 31, 9] * 4, 520, 320, 41),
    "small": ([70, 64, 129, 3] * 3, 200, 448, None),
    "odd": ([70, 64, 129, 3, 257], 257, 1001, 300),
    "cut": ([130, 200, 0, 300], 262, 1002, 512),
    "mid": ([128, 300, 77, 250], 1024, 832, 600),
    "tall": ([600, 1000, 0, 515], 2050, 1024, None),
    "big": ([1024, 1300, 700, 1111], 2048, 2304, 1500),
    "parts": ([1300, 1100, 0, 900], 2304, 4160, None),
    "long": ([30, 1, 0, 64], 136, 5000, 70),                        # few tiles, split along the sum
    "longer": ([9, 100, 33], 6000, 72, None),                       # the input gradient's
    "odd and long": ([9, 100, 33], 77, 4001, None),
    "rows": ([3000, 0, 1700, 5], 72, 136, 300),                     # few matrices, split along the rows
    "odd rows": ([9000, 100], 33, 65, None),
    "short": ([40, 1, 64, 65, 100, 129, 256] * 6, 2048, 2048, None),   # gradients: reductions of one to four k-tiles
}


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("kind", list(CASES))
def test_gated_pass(kind, layout, monkeypatch):
    import torch
    counts, N, K, tokens = CASES[kind]
    o = [sum(counts[:i]) for i in range(len(counts) + 1)]
    rows, E = o[-1], len(counts)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    offsets = torch.tensor(o, dtype=torch.int32, device="cuda")
    source = None if tokens is None else torch.randint(0, tokens, (rows,), generator=gen, device="cuda").int()
    dt = torch.bfloat16
    w = (E, N, K) if layout == "nk" else (E, K, N)
    x, dh = _rand(gen, (rows if tokens is None else tokens, K), 1.0, dt), _rand(gen, (rows, N), 0.3, dt)
    wg, wu = _rand(gen, w, K ** -0.5, dt), _rand(gen, w, K ** -0.5, dt)

    def step():
        h, g, u, y = (torch.zeros(rows, N, dtype=dt, device="cuda") for _ in range(4))
        dx, dx1 = (torch.zeros(rows, K, dtype=dt, device="cuda") for _ in range(2))
        dwg, dwu, dw = (torch.full_like(wg, float("nan")) for _ in range(3))
        with spg.GroupedGated(rows, N, K, E, "bf16", layout, "silu", tokens=tokens) as plan:
            ws = torch.zeros(max(1, plan.workspace_bytes()), dtype=torch.uint8, device="cuda")
            plan(x, wg, wu, offsets, h, source=source, G=g, U=u, workspace=ws)
            plan.backward(dh, x, wg, wu, g, u, offsets, dx, dwg, dwu, source=source, workspace=ws)
        with spg.GroupedGemm(rows, N, K, E, "bf16", layout, tokens=tokens) as plan:
            ws = torch.zeros(max(1, plan.workspace_bytes()), dtype=torch.uint8, device="cuda")
            plan(x, wg, offsets, y, source=source, workspace=ws)
            plan.backward(dh, x, wg, offsets, dx1, dw, source=source, workspace=ws)
        torch.cuda.synchronize()
        return [h, g, u, y, dx, dx1, dwg, dwu, dw]

    _same(*_both(step, monkeypatch))
