"""A transformer block around the mixture-of-experts layer, trained for a few
steps on one GPU: every operator of the package as a model would use it.

    python examples/train_block.py [--mode bf16|mxfp8|mxfp8_full] [--state fp32|mxfp8] [--steps N]

The block (token mixing left out): a dense feed-forward whose second
projection adds the residual stream, the norm that joins the experts' output
back into the stream, router logits in 32 bits from the same projection
operator, softmax and top-k routing, and the layer, which in the MXFP8 modes
takes its input as the norm quantised it.  The target is what a fixed random
map makes of the input.  One AdamW steps every tensor, with fp32 master copies
of the bf16 weights and the gradients clipped by a scale that stays on the GPU.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mixture_experts_layer_mok_gb300 as mok  # noqa: E402
from mixture_experts_layer_mok_gb300.autograd import MoKLayer, MoKLinear, MoKRMSNorm  # noqa: E402
from mixture_experts_layer_mok_gb300.inputs import route  # noqa: E402


class Block(torch.nn.Module):
    def __init__(self, H, I, E, k, I_s, mode, device, generator):
        super().__init__()
        kw = dict(device=device, generator=generator)
        self.k, self.mode = k, mode
        self.norm1 = MoKRMSNorm(H, device=device)
        self.up = MoKLinear(H, 4 * H, activation="gelu", **kw)
        self.down = MoKLinear(4 * H, H, **kw)
        self.norm2 = MoKRMSNorm(H, mxfp8=mode != "bf16", device=device)
        self.router = MoKLinear(H, E, out_dtype=torch.float32, **kw)
        self.experts = MoKLayer(E, H, I, I_s, mode=mode, **kw)
        self.norm3 = MoKRMSNorm(H, device=device)
        self.head = MoKLinear(H, H, **kw)

    def forward(self, x):
        y, stream = self.norm1(x)
        h = self.down(self.up(y), residual=stream)
        y, stream, *mx = self.norm2(h)
        weights, experts = route(self.router(y), self.k)
        out = self.experts(y, weights, experts, x_mx=mx[0] if mx else None)
        y, _ = self.norm3(out, stream)
        return self.head(y)


def train(steps=30, T=512, H=256, I=256, E=16, k=4, I_s=256, mode="bf16", state="fp32", lr=3e-3, seed=0, log=None):
    """Trains the block on one synthetic batch per step; returns the losses."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    block = Block(H, I, E, k, I_s, mode, "cuda", gen)
    target_map = torch.randn(H, H, generator=gen, device="cuda", dtype=torch.bfloat16) / H ** 0.5
    params = list(block.parameters())
    opt = mok.AdamW(params, lr=lr, betas=(0.9, 0.95), weight_decay=0.01, state=state, master=True, seed=seed)
    losses = []
    for step in range(steps):
        x = torch.randn(T, H, generator=gen, device="cuda", dtype=torch.bfloat16)
        loss = (block(x).float() - torch.tanh(x @ target_map).float()).square().mean()
        for p in params:
            p.grad = None
        loss.backward()
        norm = torch.stack([p.grad.float().square().sum() for p in params]).sum().sqrt()
        opt.step(grad_scale=(1.0 / norm.clamp(min=1.0)).reshape(1))
        losses.append(loss.detach())
        if log:
            log(f"step {step:3d}  loss {loss.item():.4f}  gradient norm {norm.item():.3f}")
    return [v.item() for v in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--mode", choices=sorted(mok.MODES), default="bf16", help="the experts' precision")
    ap.add_argument("--state", choices=("fp32", "mxfp8"), default="fp32", help="the optimiser's states")
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--hidden", type=int, default=256)
    a = ap.parse_args()
    losses = train(a.steps, T=a.tokens, H=a.hidden, mode=a.mode, state=a.state, log=print)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}")


if __name__ == "__main__":
    main()
