"""A few training steps of a stack of pre-norm mixture-of-experts blocks that keep their activations in
8 bits: each block adds its input to the stream, normalises it, routes and runs its experts.  Between
the passes a block holds the gate's logits, the routing, the statistics, 8-bit checkpoints and its
weights in bf16; the full-size buffers and the workspace are shared by all blocks.

    python examples/prenorm_moe_training_step.py [--tokens 2048 --width 1024 --blocks 4 ...]

Prints the loss (mean squared error to a fixed random target) and the bytes that a block keeps; needs a
GPU of the kind that the library is built for.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import token_dispatch_expert_gb300 as tde  # noqa: E402


class Block:
    def __init__(self, scratch, rand, kind, checkpoint):
        c = scratch.cfg
        self.norm = tde.MoENorm(c.T, c.d, kind=kind, checkpoint=checkpoint, ws=scratch.ws)
        self.moe = tde.CheckpointedMoELayer(scratch, checkpoint)
        self.p = {"gamma": torch.ones(c.d, device="cuda"), "beta": torch.zeros(c.d, device="cuda"),
                  "gate": 0.02 * rand(c.E, c.d), "W1": 0.03 * rand(c.E, 2 * c.ffn, c.d),
                  "W2": 0.03 * rand(c.E, c.d, c.ffn)}           # fp32 masters

    def kept_bytes(self):
        """(of activations, of weights in bf16): all that it holds from forward to backward but the
        masters."""
        n, m = self.norm, self.moe
        kept = [*n.kept, n.rstd, *([] if n.mean is None else [n.mean]), *m.ab, *m.yp, *m.r.values(), self.logits]
        return tuple(sum(t.numel() * t.element_size() for t in part) for part in (kept, self.w))

    def _beta(self):
        return self.p["beta"] if self.norm.kind == "layer" else None

    def forward(self, stream, branch):
        """(the stream with the branch added, this block's branch)"""
        n, stream = self.norm.forward(stream, self.p["gamma"], self._beta(), residual=branch)
        self.logits = n.float() @ self.p["gate"].t()
        self.w = self.p["W1"].bfloat16(), self.p["W2"].bfloat16()
        return stream, self.moe.forward(self.logits, n, *self.w)

    def backward(self, dstream, dbranch):
        """From the gradients of both results: (the gradient of both arguments, the parameters')."""
        n = self.norm.restore(self.p["gamma"], self._beta())
        g = self.moe.backward(self.logits, n, dbranch, *self.w)
        dn = (g["dx"].float() + g["dlogits"] @ self.p["gate"]).bfloat16()
        o = self.norm.backward(dn, self.p["gamma"], add=dstream, beta=self.norm.kind == "layer")
        grads = {"gate": g["dlogits"].t() @ n.float(), "W1": g["dW1"].float(), "W2": g["dW2"].float(),
                 "gamma": o["dgamma"]}
        if "dbeta" in o:
            grads["beta"] = o["dbeta"]
        return o["dx"], grads


def train(tokens=2048, width=1024, ffn=512, experts=16, k=2, blocks=4, steps=6, lr=0.1, kind="layer",
          checkpoint="int8", seed=0, log=print):
    """Runs the steps; returns the losses."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    cfg = tde.make_config(tokens, width, experts, k, ffn)
    scratch = tde.MoEScratch(cfg)
    stack = [Block(scratch, rand, kind, checkpoint) for _ in range(blocks)]
    x, target = rand(tokens, width).bfloat16(), rand(tokens, width).bfloat16()
    losses = []
    for step in range(steps):
        stream, branch = x, torch.zeros_like(x)
        for b in stack:
            stream, branch = b.forward(stream, branch)
        if step == 0:
            kept = [n / 2**20 for n in stack[0].kept_bytes()]
            log(f"kept by a block: {kept[0]:.1f} MiB of activations, {kept[1]:.1f} MiB of weights")
        diff = stream.float() + branch.float() - target.float()
        losses.append(float(diff.square().mean()))
        d = diff.bfloat16()                     # of half the summed square
        dstream = dbranch = d
        for b in reversed(stack):
            dstream, grads = b.backward(dstream, dbranch)
            dbranch = dstream                   # a block's arguments are summed
            for name, grad in grads.items():
                b.p[name] -= lr / tokens * grad
        status, flags = stack[0].moe.status()
        if status != 0:
            raise RuntimeError(f"{tde.moe_status_string(status)} flags={flags:#x}")
        log(f"step {step}: loss {losses[-1]:.5f}")
    return losses


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    for name, value in (("tokens", 2048), ("width", 1024), ("ffn", 512), ("experts", 16), ("k", 2),
                        ("blocks", 4), ("steps", 6)):
        p.add_argument("--" + name, type=int, default=value)
    p.add_argument("--kind", choices=sorted(tde.NORMS), default="layer")
    p.add_argument("--checkpoint", choices=tde.CKPT_FORMATS, default="int8")
    a = p.parse_args()
    train(a.tokens, a.width, a.ffn, a.experts, a.k, a.blocks, a.steps, kind=a.kind,
          checkpoint=a.checkpoint)
