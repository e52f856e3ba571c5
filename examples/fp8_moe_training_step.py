"""A few training steps of one mixture-of-experts layer on 8-bit operands: group-limited routing
with a balance bias, experts quantised in blocks of 128, forward, backward and an update of the
weights, the router's projection and the bias.

    python examples/fp8_moe_training_step.py [--tokens 4096 --width 2048 --experts 64 ...]

Prints the loss (mean squared error to a fixed random target) and the spread of the experts'
loads at every step; needs a GPU of the kind that the library is built for.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import token_dispatch_expert_gb300 as tde  # noqa: E402


def train(tokens=4096, width=2048, ffn=768, experts=64, k=6, groups=8, top_groups=4, steps=8,
          lr=2.0, bias_step=0.002, seed=0, log=print):
    """Runs the steps; returns the losses."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = rand(tokens, width).bfloat16()
    target = rand(tokens, width).bfloat16()
    w1 = 0.02 * rand(experts, 2 * ffn, width)          # fp32 masters
    w2 = 0.02 * rand(experts, width, ffn)
    gate = 0.02 * rand(experts, width)
    bias = torch.zeros(experts, device="cuda")
    cfg = tde.make_config(tokens, width, experts, k, ffn, route_scale=1.0)
    router = tde.make_router("sigmoid", groups, top_groups, group_top=2, renorm=True, bias=bias)
    layer = tde.Fp8MoELayer(cfg, router, grad_dtype=torch.float32)
    losses = []
    for step in range(steps):
        logits = x.float() @ gate.t()
        wq = layer.quantize_weights(w1.bfloat16(), w2.bfloat16())
        y = layer.forward(logits, x, wq)
        diff = y.float() - target.float()
        losses.append(float(diff.square().mean()))
        grads = layer.backward(logits, x, diff.bfloat16(), wq)   # of half the summed square
        scale = lr / tokens
        w1 -= scale * grads["dW1"]
        w2 -= scale * grads["dW2"]
        gate -= scale * (grads["dlogits"].t() @ x.float())
        # the bias moves towards the experts that were chosen less than the average
        counts = layer.r["counts"].float()
        bias += bias_step * torch.sign(counts.mean() - counts)
        status, flags = layer.status()
        if status != 0:
            raise RuntimeError(f"{tde.moe_status_string(status)} flags={flags:#x}")
        log(f"step {step}: loss {losses[-1]:.5f}, rows per expert "
            f"{int(counts.min())} .. {int(counts.max())}")
    return losses


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    for name, value in (("tokens", 4096), ("width", 2048), ("ffn", 768), ("experts", 64), ("k", 6),
                        ("groups", 8), ("top-groups", 4), ("steps", 8)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    train(a.tokens, a.width, a.ffn, a.experts, a.k, a.groups, a.top_groups, a.steps)
