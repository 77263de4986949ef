"""The check of the gated gradients by group (tests/grouped_gradients.py) on the CPU: it accepts
gradients with the roundings that it allows, and rejects planted mistakes."""

import pytest

torch = pytest.importorskip("torch")

from tests.grouped_gradients import act_of, check, gradients, loss   # noqa: E402

OFFSETS = [2, 2, 5, 21, 38, 38, 39]
N, K = 40, 48


def _case(dtype, seed=1):
    gen = torch.Generator()
    gen.manual_seed(seed)
    draw = lambda *s, std=1.0: (std * torch.randn(*s, generator=gen)).to(dtype).double()
    E = len(OFFSETS) - 1
    return draw(OFFSETS[-1] + 5, K), draw(E, K, N, std=K ** -0.5), draw(E, K, N, std=K ** -0.5), draw(OFFSETS[-1] + 5, N, std=0.3)


def _rounded(x, wg, wu, dh, act, dtype):
    """The backward formula with G, U, dG, dU and the gradients rounded to the 16-bit type."""
    q = lambda t: t.to(dtype).double()
    dx, dwg, dwu = torch.zeros_like(x), torch.zeros_like(wg), torch.zeros_like(wu)
    parts = []
    for e in range(len(OFFSETS) - 1):
        r = slice(OFFSETS[e], OFFSETS[e + 1])
        g, u = q(x[r] @ wg[e]).requires_grad_(), q(x[r] @ wu[e])
        a = act_of(g, act)
        slope, = torch.autograd.grad(a.sum(), g)
        dg, du = q(dh[r] * u * slope), q(dh[r] * a.detach())
        dx[r] = q(dg @ wg[e].t() + du @ wu[e].t())
        dwg[e], dwu[e] = q(x[r].t() @ dg), q(x[r].t() @ du)
        parts.append((r, dg, du))
    return [dx, dwg, dwu], parts


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
def test_roundings_pass_and_mistakes_do_not(dtype, act):
    half = torch.finfo(dtype).eps / 2
    x, wg, wu, dh = _case(dtype)
    good, parts = _rounded(x, wg, wu, dh, act, dtype)
    check(good, x, wg, wu, dh, OFFSETS, act, half)
    check(gradients(x, wg, wu, dh, OFFSETS, act), x, wg, wu, dh, OFFSETS, act, half)

    def without(path):
        """dX of the gate or of the up projection alone."""
        dx = torch.zeros_like(x)
        for e, (r, dg, du) in enumerate(parts):
            dx[r] = dg @ wg[e].t() if path == "gate" else du @ wu[e].t()
        return dx

    first = OFFSETS.index(5)                             # the group of three rows' end
    swapped = good[1].clone()
    swapped[first - 1], swapped[first] = good[1][first], good[1][first - 1]
    last = good[0].clone()
    last[OFFSETS[-1] - 1] = 0                            # one row of 37 left out
    linear = [torch.zeros_like(wg), torch.zeros_like(wu)]
    for e, (r, dg, du) in enumerate(parts):              # act' taken as 1
        u = x[r] @ wu[e]
        linear[0][e] = x[r].t() @ (dh[r] * u)
    bad = {"halved": [0.5 * g for g in good], "and a half": [1.5 * g for g in good], "negated": [-g for g in good],
           "5% more": [1.05 * g for g in good] if dtype is torch.float16 else None,
           "gate alone": [without("gate"), good[1], good[2]], "up alone": [without("up"), good[1], good[2]],
           "groups swapped": [good[0], swapped, good[2]], "a row left out": [last, good[1], good[2]],
           "no slope": [good[0], linear[0], good[2]], "gate for up": [good[0], good[2], good[1]]}
    for name, grads in bad.items():
        if grads is None:
            continue
        for i in range(3):
            if torch.equal(grads[i], good[i]):
                continue
            one = list(good)
            one[i] = grads[i]
            with pytest.raises(AssertionError):
                check(one, x, wg, wu, dh, OFFSETS, act, half)
                pytest.fail(f"{name}, gradient {i}, passes", pytrace=False)


def test_the_loss_is_the_operators():
    # H = act(X Wg) * (X Wu) by group, rows outside the groups not in it
    x, wg, wu, dh = _case(torch.float16)
    want = 0.0
    for e in range(len(OFFSETS) - 1):
        for r in range(OFFSETS[e], OFFSETS[e + 1]):
            g, u = x[r] @ wg[e], x[r] @ wu[e]
            want += float((dh[r] * (g / (1 + torch.exp(-g))) * u).sum())
    assert abs(float(loss(x, wg, wu, dh, OFFSETS, "silu")) - want) <= 1e-10 * abs(want) + 1e-12
