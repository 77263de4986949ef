"""The gated projection by group and its loss in 64 bits, differentiated by central differences and
by autograd (not by the backward formula), and how far gradients from 16-bit G, U, dG and dU may be
off it.  On any device; used on the CPU with planted mistakes and on the GPU with the kernels' gradients.

With e half a step of the 16-bit type, relative: G and U are stored off by e, so that dG = dH U act'(G)
is off by e (|dH U G act''(G)| + |dG|), one e more for its own rounding, and dU = dH act(G) by
e (|dH G act'(G)| + |dU|).  A gradient is those times W or X^T, so a matrix norm more at most
(Frobenius for the factor, the largest singular value for the other), a rounding e of itself, and its
fp32 sum, K 2^-24 of the sum of magnitudes.  Projected on a unit direction no error is larger
than its norm.  1.1 covers the products of two of these."""

import torch

U32 = 2.0 ** -24
_C, _A = 0.7978845608, 0.044715


def act_of(g, act):
    z = g if act == "silu" else 2 * _C * (g + _A * g * g * g)
    return g * torch.sigmoid(z)


def loss(x, wg, wu, dh, offsets, act):
    """Sum of dh times H; x [rows,K], wg and wu [E,K,N], all in 64 bits."""
    s = x.new_zeros(())
    for e in range(len(offsets) - 1):
        r = slice(offsets[e], offsets[e + 1])
        s = s + (dh[r] * act_of(x[r] @ wg[e], act) * (x[r] @ wu[e])).sum()
    return s


def gradients(x, wg, wu, dh, offsets, act):
    leaves = [t.detach().clone().requires_grad_() for t in (x, wg, wu)]
    return torch.autograd.grad(loss(*leaves, dh, offsets, act), leaves)


def difference(args, which, d, h, dh, offsets, act):
    """The derivative of the loss along d by a central difference of fourth order."""
    def at(t):
        moved = list(args)
        moved[which] = args[which] + t * h * d
        return float(loss(*moved, dh, offsets, act))
    return (8 * (at(1) - at(-1)) - (at(2) - at(-2))) / (12 * h)


def error_norms(x, wg, wu, dh, offsets, act, half):
    """Bounds on the norms of the errors of dX, dWg and dWu."""
    x2 = g2 = u2 = 0.0
    for e in range(len(offsets) - 1):
        r = slice(offsets[e], offsets[e + 1])
        if offsets[e] == offsets[e + 1]:
            continue
        K, rows = x.shape[1], offsets[e + 1] - offsets[e]
        G = (x[r] @ wg[e]).requires_grad_()
        U, D = x[r] @ wu[e], dh[r]
        a = act_of(G, act)
        slope, = torch.autograd.grad(a.sum(), G, create_graph=True)
        bend, = torch.autograd.grad(slope.sum(), G)
        a, slope, G = a.detach(), slope.detach(), G.detach()
        dG, dU = D * U * slope, D * a
        eG = half * ((D * U * G * bend).abs() + 2 * dG.abs()) + 8 * U32 * (D * U).abs() + K * U32 * (D * U * bend).abs() * (x[r].abs() @ wg[e].abs())
        eU = half * ((D * G * slope).abs() + dU.abs()) + 8 * U32 * (D * G).abs()
        n = lambda t: float(t.norm())
        top = lambda t: float(torch.linalg.matrix_norm(t, 2))
        eG, eU = n(eG), n(eU)
        N = wg.shape[2]
        dX = dG @ wg[e].t() + dU @ wu[e].t()
        x2 += (eG * top(wg[e]) + eU * top(wu[e]) + half * n(dX) + 2 * N * U32 * n(dG.abs() @ wg[e].abs().t() + dU.abs() @ wu[e].abs().t())) ** 2
        g2 += (eG * top(x[r]) + half * n(x[r].t() @ dG) + rows * U32 * n(x[r].abs().t() @ dG.abs())) ** 2
        u2 += (eU * top(x[r]) + half * n(x[r].t() @ dU) + rows * U32 * n(x[r].abs().t() @ dU.abs())) ** 2
    return [1.1 * v ** 0.5 for v in (x2, g2, u2)]


def check(grads, x, wg, wu, dh, offsets, act, half):
    """Raises where dX, dWg or dWu (wg's and wu's layout, [E,K,N]) are not the loss's."""
    args = (x, wg, wu)
    exact = gradients(*args, dh, offsets, act)
    bounds = error_norms(*args, dh, offsets, act, half)
    for which, name in enumerate(("dX", "dWg", "dWu")):
        want, got, tol = exact[which], grads[which].double(), bounds[which]
        size = float(want.norm())
        off = float((got - want).norm())
        assert off <= tol, f"{name}: off by {off}, {off / size} of it, more than {tol}"
        # along the gradient itself, where a difference is the gradient's norm, and along a direction
        # that no symmetry of the formulas has
        gen = torch.Generator(device=x.device)
        gen.manual_seed(17 + which)
        other = torch.empty_like(want).normal_(generator=gen) * (want.abs() + size / want.numel() ** 0.5)
        for d in (want, other + 2 * want):
            d = d / d.norm()
            slope = difference(args, which, d, 1e-3, dh, offsets, act)
            along = float((exact[which] * d).sum())
            assert abs(slope - along) <= 1e-7 * size, f"{name}: a difference of {slope}, autograd {along}"
            seen = float((got * d).sum())
            assert abs(seen - slope) <= tol + 1e-7 * size, f"{name} along a direction: {seen}, difference {slope}, tolerance {tol}"
