"""A mixture-of-experts feed-forward block, trained for a few steps and then served token by token.

    n = norm(x),  l = n Wr^T,  k experts e_j with gates g_j from l
    y = x + sum over j of g_j (silu(n Wg[e_j]^T) * (n Wu[e_j]^T)) Wd[e_j]^T

Every step is a call of this package: the layer norm, the router, the gated projection and the
down projection by group, the combination, and their backward passes; the router's logits come
from the plain GEMM.

    python examples/mixture_of_experts.py [--tokens 512] [--model 512] [--hidden 768] [--experts 8] [--choices 2] [--steps 10]
"""

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import software_pipelined_tiled_gemm_amd as spg


class ExpertsBlock:
    """One block's weights, and plans and buffers for a fixed number of tokens."""

    NAMES = ("norm_w", "norm_b", "router", "gate", "up", "down")

    def __init__(self, tokens, model, hidden, experts, choices, seed=0, weights=None):
        self.shape = tokens, model, hidden, experts, choices
        if weights is None:
            gen = torch.Generator(device="cuda")
            gen.manual_seed(seed)

            def weight(*s):
                return torch.empty(*s, device="cuda").normal_(0.0, s[-1] ** -0.5, generator=gen)

            weights = dict(norm_w=torch.ones(model, device="cuda"), norm_b=torch.zeros(model, device="cuda"),
                           router=weight(experts, model), gate=weight(experts, hidden, model),
                           up=weight(experts, hidden, model), down=weight(experts, model, hidden))
        self.master = weights                                    # fp32
        self.load()
        rows = tokens * choices

        def new(*s, dtype=torch.bfloat16):
            return torch.zeros(*s, dtype=dtype, device="cuda")

        self.n, self.y, self.out, self.dn = (new(tokens, model) for _ in range(4))
        self.mean, self.rstd = new(tokens, dtype=torch.float32), new(tokens, dtype=torch.float32)
        self.logits, self.dlogits = (new(tokens, experts, dtype=torch.float32) for _ in range(2))
        self.g, self.dg = (new(tokens, choices, dtype=torch.float32) for _ in range(2))
        self.expert, self.slot = (new(tokens, choices, dtype=torch.int32) for _ in range(2))
        self.source, self.offsets = new(rows, dtype=torch.int32), new(experts + 1, dtype=torch.int32)
        self.h, self.hg, self.hu, self.dh = (new(rows, hidden) for _ in range(4))
        self.yr, self.dyr, self.dxr = (new(rows, model) for _ in range(3))
        self.grad = {k: torch.zeros_like(v, dtype=torch.float32 if k.startswith("norm") else torch.bfloat16)
                     for k, v in weights.items()}
        self.norm = spg.LayerNorm(tokens, model, "bf16", "f32")
        self.to_logits = spg.Gemm(tokens, experts, model, "bf16", "f32", "nk")
        self.back_n = spg.Gemm(tokens, model, experts, "bf16", "bf16", "kn")
        self.back_router = spg.Gemm(experts, model, tokens, "bf16", "bf16", "kn")
        self.route = spg.Router(tokens, experts, choices, "f32", renormalise=True)
        self.gated = spg.GroupedGated(rows, hidden, model, experts, "bf16", "nk", "silu", tokens=tokens)
        self.down = spg.GroupedGemm(rows, model, hidden, experts, "bf16", "nk")
        self.combine = spg.Combine(tokens, choices, rows, model, "bf16")
        plans = self.norm, self.route, self.gated, self.down
        self.ws = torch.empty(max(1, *(p.workspace_bytes() for p in plans)), dtype=torch.uint8, device="cuda")

    def load(self):
        """The copies of the weights that the products read."""
        self.w = {k: v if k.startswith("norm") else v.bfloat16() for k, v in self.master.items()}

    def forward(self, x):
        w, ws = self.w, self.ws
        self.norm(x, w["norm_w"], w["norm_b"], self.n, mean=self.mean, rstd=self.rstd)
        self.to_logits(self.n, w["router"], self.logits)
        self.route(self.logits, self.g, self.expert, self.slot, self.source, self.offsets, workspace=ws)
        self.gated(self.n, w["gate"], w["up"], self.offsets, self.h, source=self.source, G=self.hg, U=self.hu, workspace=ws)
        self.down(self.h, w["down"], self.offsets, self.yr, workspace=ws)
        self.combine(self.yr, self.slot, self.g, self.y)
        return torch.add(x, self.y, out=self.out)

    def backward(self, x, dout):
        """Gradients of the weights into ``grad``; returns the input's."""
        w, d, ws = self.w, self.grad, self.ws
        self.combine.backward(dout, self.yr, self.slot, self.g, self.dyr, self.dg)
        self.down.backward(self.dyr, self.h, w["down"], self.offsets, self.dh, d["down"], workspace=ws)
        self.gated.backward(self.dh, self.n, w["gate"], w["up"], self.hg, self.hu, self.offsets, self.dxr, d["gate"],
                            d["up"], source=self.source, workspace=ws)
        self.route.backward(self.logits, self.expert, self.dg, self.dlogits)
        dl = self.dlogits.bfloat16()
        self.back_router(dl.t().contiguous(), self.n, d["router"])
        from_router, dn, dx = (torch.empty_like(x) for _ in range(3))
        self.back_n(dl, w["router"], from_router)
        self.combine(self.dxr, self.slot, None, dn)              # a token's rows, summed
        torch.add(dn, from_router, out=self.dn)
        self.norm.backward(self.dn, x, w["norm_w"], self.mean, self.rstd, dx, d["norm_w"], d["norm_b"], workspace=ws)
        return dx + dout

    def update(self, rate):
        for k, m in self.master.items():
            m.sub_(self.grad[k].float(), alpha=rate)
        self.load()


def main(tokens=512, model=512, hidden=768, experts=8, choices=2, steps=10, rate=0.05):
    """Fit a block to another one's outputs, then serve single tokens with it; returns the losses and
    the served tokens' largest difference from the batch's outputs, relative to the largest output."""
    teacher = ExpertsBlock(tokens, model, hidden, experts, choices, seed=1)
    block = ExpertsBlock(tokens, model, hidden, experts, choices, seed=2)
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
    one = ExpertsBlock(1, model, hidden, experts, choices, weights=block.master)
    worst = 0.0
    for t in range(min(tokens, 8)):
        got = one.forward(x[t:t + 1]).float()
        worst = max(worst, float((got - want[t:t + 1]).abs().max() / want.abs().max()))
    return losses, worst


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("tokens", 512), ("model", 512), ("hidden", 768), ("experts", 8), ("choices", 2), ("steps", 10)):
        ap.add_argument("--" + name, type=int, default=default)
    ap.add_argument("--rate", type=float, default=0.05)
    losses, worst = main(**vars(ap.parse_args()))
    print("mean squared error per step:", " ".join(f"{v:.4f}" for v in losses))
    print(f"served token by token: within {worst:.4f} of the batch's largest output")
