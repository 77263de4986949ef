"""GPU tests of the products by group on few tiles with long reductions, which are split over the
CUs and joined: every small tile, both layouts and alignments, reductions that end inside a k-tile
and inside a 16-byte chunk, rows by their source, forward and input gradients.  Formulas and
tolerances of test_gpu_grouped.py; parts are sums in fp32 like any other order of them."""

import pytest

from tests.test_gpu_grouped import run_gated, run_plain

pytestmark = pytest.mark.gpu

# (N, K): the forward pass's reduction is K, the input gradient's N
SIZES = [(96, 4200), (89, 3001), (40, 6000), (520, 2056), (4200, 96), (3001, 89), (8, 12288), (2056, 2050)]


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("kind", ["one", "single", "few", "tile", "ragged", "skewed", "empty"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_plain(size, kind, layout):
    run_plain(kind, *size, "bf16", layout, 0, None, 200)
    run_plain(kind, *size, "f16", layout, 1, 37, 210)


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("kind", ["one", "few", "tile", "skewed"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_gated(size, kind, layout):
    run_gated(kind, *size, "bf16", layout, "silu", 0, 50, True, 220)
    run_gated(kind, *size, "f16", layout, "gelu_tanh", 1, None, True, 230)
