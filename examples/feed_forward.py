"""A gated feed-forward block, trained for a few steps and then served in int8.

    Y = H Wd^T,  H = silu(X Wg^T) * (X Wu^T)

Training runs the gated projection with its pre-activations kept, the down projection
through the plain GEMM, and the backward pass; serving quantises the weights once and every
row of activations on the way, and runs both layers as int8 products.

    python examples/feed_forward.py [--tokens 512] [--model 1024] [--hidden 2816] [--steps 20]
"""

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import software_pipelined_tiled_gemm_amd as spg


class FeedForward:
    """One block's weights ([N,K] storage), plans and buffers for a fixed number of tokens."""

    def __init__(self, tokens, model, hidden, seed=0, dtype=torch.bfloat16):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)

        def weight(n, k):
            w = torch.empty(n, k, dtype=torch.float32, device="cuda")
            return w.normal_(0.0, k ** -0.5, generator=gen)

        # fp32 master weights, and the copies that the products read
        self.master = [weight(hidden, model), weight(hidden, model), weight(model, hidden)]
        self.w = [m.to(dtype) for m in self.master]
        new = lambda *s: torch.empty(*s, dtype=dtype, device="cuda")
        self.h, self.g, self.u, self.dh = (new(tokens, hidden) for _ in range(4))
        self.y, self.dx = new(tokens, model), new(tokens, model)
        self.dw = [torch.empty_like(w) for w in self.w]
        self.gated = spg.Gated(tokens, hidden, model, "bf16", "nk", "silu")
        self.down = spg.Gemm(tokens, model, hidden, "bf16", "bf16", "nk")
        self.down_dx = spg.Gemm(tokens, hidden, model, "bf16", "bf16", "kn")
        self.down_dw = spg.Gemm(model, hidden, tokens, "bf16", "bf16", "kn")
        self.ws = torch.empty(self.gated.workspace_bytes(), dtype=torch.uint8, device="cuda")

    def forward(self, x):
        wg, wu, wd = self.w
        self.gated(x, wg, wu, self.h, G=self.g, U=self.u, workspace=self.ws)
        return self.down(self.h, wd, self.y)

    def backward(self, x, dy):
        wg, wu, wd = self.w
        self.down_dx(dy, wd, self.dh)                            # dH = dY Wd
        self.down_dw(dy.t().contiguous(), self.h, self.dw[2])    # dWd = dY^T H
        self.gated.backward(self.dh, x, wg, wu, self.g, self.u, self.dx, self.dw[0], self.dw[1], workspace=self.ws)

    def update(self, rate):
        for m, w, d in zip(self.master, self.w, self.dw):
            m.sub_(d.float(), alpha=rate)
            w.copy_(m)


class Int8FeedForward:
    """The same block with int8 weights, one scale per output channel."""

    def __init__(self, weights, tokens):
        self.q = []
        for w in weights:
            a = torch.empty(w.shape, dtype=torch.int8, device="cuda")
            s = torch.empty(w.shape[0], dtype=torch.float32, device="cuda")
            spg.gemm_quantize_rows(w, a, s)
            self.q.append((a, s))
        hidden, model = weights[0].shape
        i8 = lambda *s: torch.empty(*s, dtype=torch.int8, device="cuda")
        self.x, self.sx = i8(tokens, model), torch.empty(tokens, device="cuda")
        self.h8, self.sh = i8(tokens, hidden), torch.empty(tokens, device="cuda")
        self.h = torch.empty(tokens, hidden, dtype=torch.bfloat16, device="cuda")
        self.y = torch.empty(tokens, model, dtype=torch.bfloat16, device="cuda")
        self.gated = spg.QuantizedGemm(tokens, hidden, model, "bf16", "silu")
        self.down = spg.QuantizedGemm(tokens, model, hidden, "bf16")
        self.ws = torch.empty(max(self.gated.workspace_bytes(), self.down.workspace_bytes()), dtype=torch.uint8,
                              device="cuda")

    def __call__(self, x):
        (wg, sg), (wu, su), (wd, sd) = self.q
        spg.gemm_quantize_rows(x, self.x, self.sx)
        self.gated(self.x, self.sx, wg, sg, self.h, B2=wu, scale_b2=su, workspace=self.ws)
        spg.gemm_quantize_rows(self.h, self.h8, self.sh)
        return self.down(self.h8, self.sh, wd, sd, self.y, workspace=self.ws)


def main(tokens=512, model=1024, hidden=2816, steps=20, rate=0.02):
    """Fit a block to another one's outputs, then serve it; returns the losses and the
    int8 block's relative error."""
    teacher, block = FeedForward(tokens, model, hidden, seed=1), FeedForward(tokens, model, hidden, seed=2)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    x = torch.empty(tokens, model, device="cuda").normal_(0.0, 1.0, generator=gen).bfloat16()
    target = teacher.forward(x).float()
    losses = []
    for _ in range(steps):
        diff = block.forward(x).float() - target
        losses.append(float(diff.square().mean()))
        block.backward(x, (diff * (2.0 / tokens)).bfloat16())
        block.update(rate)
    want = block.forward(x).float()
    got = Int8FeedForward(block.w, tokens)(x).float()
    return losses, float((got - want).norm() / want.norm())


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("tokens", 512), ("model", 1024), ("hidden", 2816), ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=default)
    ap.add_argument("--rate", type=float, default=0.02)
    losses, err = main(**vars(ap.parse_args()))
    print("mean squared error per step:", " ".join(f"{v:.4f}" for v in losses))
    print(f"int8 block: relative error {err:.4f} of the bf16 block's outputs")
