"""GPU tests of the example's block of experts where it serves single tokens with a batch's weights,
and of its update of the weights.

Served and in a batch, a token takes other kernels, whose fp32 sums have other orders: the values
that are stored in bf16 on its way (the norm, H, the experts' rows, their combination) differ by
roundings, 2^-8 of their size each.  The norm is in both factors of H, and silu passes on up to 1.28
of a relative change of what it is taken of: 2.3 for the norm and 3 for the rest, for either of the
two ways, so that they differ by at most 2 * 5.3 * 2^-8 of the token's size."""

import pytest

from examples import mixture_of_experts as example
from tests.test_gpu_feed_forward import _gen, _normal, _t

pytestmark = pytest.mark.gpu

LIMIT = 2 * 5.3 * 2.0 ** -8


@pytest.mark.parametrize("sizes", [dict(tokens=96, model=128, hidden=192, experts=6, choices=2),
                                   dict(tokens=70, model=264, hidden=328, experts=7, choices=3),
                                   dict(tokens=40, model=200, hidden=130, experts=40, choices=8)], ids=["example", "odd", "many"])
def test_served_tokens_are_the_batchs(sizes):
    torch = _t()
    T, D, k = sizes["tokens"], sizes["model"], sizes["choices"]
    batch = example.ExpertsBlock(**sizes, seed=2)
    one = example.ExpertsBlock(**dict(sizes, tokens=1), weights=batch.master)
    x = _normal(_gen(3), (T, D), 1.0).bfloat16()
    batch.forward(x)
    experts, y = batch.expert.clone(), batch.y.float()
    top = batch.logits.sort(dim=1, descending=True).values
    alike = 0
    for t in range(T):
        one.forward(x[t:t + 1])
        if not torch.equal(one.expert[0], experts[t]):
            # two logits next to each other in the order of the first k + 1: sums of D products of n
            # and bf16 weights, with n off by one rounding of its own
            gap = float((top[t, :k] - top[t, 1:k + 1]).min())
            assert gap <= 2.0 ** -7 * float(batch.logits[t].abs().max()), t
            continue
        alike += 1
        off = float((one.y[0].float() - y[t]).norm() / y[t].norm())
        assert off <= LIMIT, (t, off)
        # the residual is added in either, and rounded once
        assert float((one.out[0].float() - batch.out[t].float()).norm()) <= LIMIT * float(y[t].norm()) + 2.0 ** -8 * float(batch.out[t].float().norm())
    assert alike >= 0.9 * T
    # another token's output is not within the limit
    assert float((one.y[0].float() - y[0]).norm() / y[0].norm()) > 10 * LIMIT


def test_update_takes_the_gradients_off():
    torch = _t()
    sizes = dict(tokens=64, model=128, hidden=192, experts=6, choices=2)
    block = example.ExpertsBlock(**sizes, seed=2)
    x = _normal(_gen(3), (64, 128), 1.0).bfloat16()
    block.forward(x)
    block.backward(x, _normal(_gen(4), (64, 128), 0.2).bfloat16())
    before = {k: v.clone() for k, v in block.master.items()}
    block.update(0.25)
    for k in block.NAMES:
        step = 0.25 * block.grad[k].float()
        assert bool((step != 0).any()), k
        assert torch.equal(block.master[k], before[k] - step), k
        # what the products read are the new weights
        assert torch.equal(block.w[k], block.master[k] if k.startswith("norm") else block.master[k].bfloat16()), k
    # norms' weights are read in place, the others are copies: the next pass takes both
    first = block.forward(x).clone()
    again = example.ExpertsBlock(**sizes, weights={k: v.clone() for k, v in block.master.items()})
    assert torch.equal(first, again.forward(x))
