"""A pre-norm block (norm, gate, layer that keeps checkpoints) and a stack of them, as the README and
the example program run them, against 64-bit numpy that rounds and quantises where the block does.

Each block is compared on the arguments that it was given, so a tolerance is that of the layers that
it is built from: within 2e-2 of rms + |o| and rel-L2 1e-2 (gpu_util); from E4M3 checkpoints within 0.1,
since a value that lies next to a border between two codes may be kept as either, a step of 2^-3
(test_gpu_fp8_layer).
"""

import os
import sys

import numpy as np
import pytest
import torch

import block_ref
import rows_ref as ref
import token_dispatch_expert_gb300 as tde
from gpu_util import assert_close
from rows_ref import f64
from test_gpu_ckpt_layer import bf, kept

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def block(p, stream, branch, dstream, dbranch, logits, r, kind, fmt):
    """Forward and backward of one block.  p: gamma, beta, gate, W1, W2; logits: the gate's, in 32 bits;
    r: the routing that the layer chose from them (checked by other tests)."""
    T, d = stream.shape
    E, f = p["W1"].shape[0], p["W1"].shape[1] // 2
    W1, W2 = (ref.typed(p[n], "bf16") for n in ("W1", "W2"))
    s = ref.typed(ref.f32(stream + branch), "bf16")
    beta = p["beta"] if kind == "layer" else 0.0
    n = ref.typed(ref.norm(s, p["gamma"], beta, kind, 1e-5), "bf16")
    m, rstd = ref.stats(s, kind, 1e-5)
    sk = kept(s, fmt)
    again = ref.typed((sk - m[:, None]) * rstd[:, None] * p["gamma"] + beta, "bf16")
    seg = [slice(r["offsets"][e], r["offsets"][e + 1]) for e in range(E)]
    rows = r["offsets"][-1]
    src = r["src_tok"][:rows]
    ab, yp = np.zeros((rows, 2 * f)), np.zeros((rows, d))
    for e in range(E):
        ab[seg[e]] = ref.typed(n[src[seg[e]]] @ W1[e].T, "bf16")
    h = ref.typed(ref.swiglu(ab[:, :f], ab[:, f:]), "bf16")
    for e in range(E):
        yp[seg[e]] = ref.typed(h[seg[e]] @ W2[e].T, "bf16")
    abk, ypk = kept(ab, fmt), kept(yp, fmt)
    hk, abk = ref.typed(ref.swiglu(abk[:, :f], abk[:, f:]), "bf16"), ref.typed(abk, "bf16")
    w = r["topk_w"].astype(np.float64)
    y, dw, dyp = np.zeros((T, d)), np.zeros(w.shape), np.zeros((rows, d))
    slots = [(t, j, r["dest_row"][t, j]) for t, j in np.ndindex(w.shape) if r["dest_row"][t, j] >= 0]
    for t, j, at in slots:
        y[t] += w[t, j] * yp[at]
        dw[t, j] = dbranch[t] @ ypk[at]
        dyp[at] = ref.typed(w[t, j] * dbranch[t], "bf16")
    dab, dxp, dx = np.zeros((rows, 2 * f)), np.zeros((rows, d)), np.zeros((T, d))
    dW1, dW2 = np.zeros(W1.shape), np.zeros(W2.shape)
    for e in range(E):
        g = seg[e]
        dab[g] = ref.typed(np.concatenate(ref.swiglu_bwd(dyp[g] @ W2[e], abk[g, :f], abk[g, f:]), 1), "bf16")
        dxp[g] = ref.typed(dab[g] @ W1[e], "bf16")
        dW1[e], dW2[e] = dab[g].T @ again[src[g]], dyp[g].T @ hk[g]
    for t, j, at in slots:
        dx[t] += dxp[at]
    dl = block_ref.route_grad(logits, r["topk_idx"], dw, score="softmax", renorm=True, scale=1.0)
    by_gate = dl @ p["gate"]
    dn = ref.typed(ref.f32(ref.typed(dx, "bf16") + by_gate), "bf16")
    dv, dgamma, dbeta = ref.norm_bwd(dn, sk, m, rstd, p["gamma"], dstream, kind)
    grads = {"gamma": dgamma, "gate": dl.T @ again, "W1": dW1, "W2": dW2}
    if kind == "layer":
        grads["beta"] = dbeta
    # what the gradient loses without the gate's share: far more than any tolerance here
    assert np.linalg.norm(by_gate) > 0.1 * np.linalg.norm(dn)
    return {"n": n, "stream": s, "branch": y, "dx": dv, "grads": grads}


def routing(layer):
    return {n: v.cpu().numpy() for n, v in layer.r.items()}


def inputs(rng, T, d, E, f):
    p = {"gamma": 1 + 0.3 * rng.normal(size=d), "beta": 0.2 * rng.normal(size=d),
         "gate": 0.3 * rng.normal(size=(E, d)), "W1": 0.2 * rng.normal(size=(E, 2 * f, d)),
         "W2": 0.2 * rng.normal(size=(E, d, f))}
    return {n: ref.f32(v) for n, v in p.items()}, [ref.typed(rng.normal(size=(T, d)), "bf16") for _ in range(4)]


def test_readme_block():
    """The README's lines for a pre-norm block, as they stand there."""
    text = open(os.path.join(ROOT, "README.md")).read()
    lines = text[text.index("# a pre-norm block"):]
    lines = lines[:lines.index("```")]
    T, d, E, k, f = 150, 128, 8, 2, 64
    p, (stream, branch, dstream, dbranch) = inputs(np.random.default_rng(4), T, d, E, f)
    put = lambda v: torch.from_numpy(v.astype(np.float32)).cuda()  # noqa: E731
    n = ref.typed(ref.norm(ref.typed(ref.f32(stream + branch), "bf16"), p["gamma"], p["beta"], "layer", 1e-5), "bf16")
    names = dict(tde=tde, torch=torch, cfg=tde.make_config(T, d, E, k, f), T=T, d=d, E=E, k=k, ffn=f,
                 stream=bf(stream), branch=bf(branch), dstream=bf(dstream), dbranch=bf(dbranch),
                 gamma=put(p["gamma"]), beta=put(p["beta"]), gate=put(p["gate"]), W1=bf(p["W1"]), W2=bf(p["W2"]),
                 logits=put(n) @ put(p["gate"]).t())
    exec(lines, names)
    o = block(p, stream, branch, dstream, dbranch, f64(names["logits"]), routing(names["moe"]), "layer", "int8")
    assert_close("logits", f64(names["logits"]), o["n"] @ p["gate"].T)
    assert_close("stream", f64(names["stream"]), o["stream"])
    assert_close("branch", f64(names["branch"]), o["branch"])
    assert_close("dx", f64(names["g2"]["dx"]), o["dx"])
    assert_close("dgamma", f64(names["g2"]["dgamma"]), o["grads"]["gamma"])
    assert_close("dbeta", f64(names["g2"]["dbeta"]), o["grads"]["beta"])
    for name in ("W1", "W2"):
        assert_close("d" + name, f64(names["g"]["d" + name]), o["grads"][name])


@pytest.mark.parametrize("kind,fmt", [("layer", "int8"), ("rms", "int8"), ("layer", "e4m3")])
def test_example_stack(kind, fmt, monkeypatch):
    """One step of the example's stack: what each block gives for what it was given, what it was given
    by the block before it or behind it, and the parameters after the step."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import prenorm_moe_training_step as ex
    blocks, T, d, E, k, f, lr = [], 130, 128, 8, 2, 64, 0.1

    class Recorded(ex.Block):
        def __init__(self, *a):
            super().__init__(*a)
            rng = np.random.default_rng(len(blocks))
            self.start, _ = inputs(rng, T, d, E, f)
            self.p = {n: torch.from_numpy(v.astype(np.float32)).cuda() for n, v in self.start.items()}
            blocks.append(self)

        def forward(self, *a):
            self.args, self.out = a, super().forward(*a)
            return self.out

        def backward(self, *a):
            self.dargs, self.dout = a, super().backward(*a)
            return self.dout

    monkeypatch.setattr(ex, "Block", Recorded)
    losses = ex.train(tokens=T, width=d, ffn=f, experts=E, k=k, blocks=3, steps=1, lr=lr, kind=kind,
                      checkpoint=fmt, log=lambda s: None)
    assert len(blocks) == 3 and np.isfinite(losses).all()
    tol = 0.1 if fmt == "e4m3" else 2e-2
    for i, b in enumerate(blocks):
        o = block(b.start, *(f64(t) for t in b.args + b.dargs), f64(b.logits), routing(b.moe), kind, fmt)
        assert_close("logits", f64(b.logits), o["n"] @ b.start["gate"].T)
        assert_close("stream", f64(b.out[0]), o["stream"])
        assert_close("branch", f64(b.out[1]), o["branch"])
        assert_close("dx", f64(b.dout[0]), o["dx"], max_tol=tol)
        assert set(b.dout[1]) == set(o["grads"])
        for n, want in o["grads"].items():
            assert_close("d" + n, f64(b.dout[1][n]), want, max_tol=tol)
            assert torch.equal(b.p[n], torch.from_numpy(b.start[n].astype(np.float32)).cuda() - lr / T * b.dout[1][n])
        if i:   # a block's arguments are what the one before it gave; both have one gradient
            assert all(a is g for a, g in zip(b.args, blocks[i - 1].out))
            assert all(a is b.dout[0] for a in blocks[i - 1].dargs)
    # the last block's results are added up: half the summed square's gradient is the difference
    last = blocks[-1]
    assert last.dargs[0] is last.dargs[1]
    want = float((f64(last.dargs[0]) ** 2).mean())     # (rounded to bf16: 2^-8 of each difference)
    assert abs(losses[0] - want) <= 1e-2 * want


@pytest.mark.parametrize("kind,fmt", [("layer", "int8"), ("rms", "e4m3")])
def test_kept_bytes(kind, fmt):
    """What the example says that a block keeps is every tensor that it, its norm and its layer hold
    between the passes, but the masters and what the blocks share."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import prenorm_moe_training_step as ex

    def tensors(o):
        if isinstance(o, torch.Tensor):
            return [o]
        o = list(o.values()) if isinstance(o, dict) else o if isinstance(o, (tuple, list)) else []
        return [t for v in o for t in tensors(v)]
    cfg = tde.make_config(100, 256, 8, 2, 64)
    scratch = tde.MoEScratch(cfg)
    b = ex.Block(scratch, lambda *s: torch.randn(*s, device="cuda"), kind, fmt)
    x = torch.randn((100, 256), device="cuda").bfloat16()
    b.forward(x, torch.zeros_like(x))
    own = {id(t): t for o in (b, b.norm, b.moe) for t in tensors(vars(o))}
    for t in tensors(vars(scratch)) + tensors(b.p):
        own.pop(id(t), None)
    assert sum(b.kept_bytes()) == sum(t.numel() * t.element_size() for t in own.values())
    assert b.kept_bytes()[1] == 2 * 8 * 3 * 64 * 256
