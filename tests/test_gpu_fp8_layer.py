"""Fp8MoELayer, the operators run together as a layer uses them, against the same path in 64-bit
numpy: the reference quantises at the same places (from values rounded to bf16 where the layer
stores bf16) and multiplies exactly.

Tolerances: with the layer's bf16 tensors (ab, yp, dh, dxp, dyp) both sides round the same value
to bf16 unless their fp32 and 64-bit sums straddle a border, so a stored value differs by at most
one bf16 step (2^-7 relative) at a few elements; there an E4M3 code may move by one step (2^-3 of
its value).  Outputs average over f or d such terms: rel-L2 within 1e-2 and every element within
0.1 of rms + |o|, the bound that the MXFP8 layer's tests derive from the same mechanism.
"""

import numpy as np
import pytest
import torch

import block_ref as ref
import token_dispatch_expert_gb300 as tde
from gpu_util import assert_close, dev

pytestmark = pytest.mark.gpu


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def deq_rows(x):
    q, s = ref.quantise_rows(x)
    return q * ref.spread(s, x.shape[1], 1)


def deq_cols(x):
    """One segment's rows quantised along the tokens."""
    return deq_rows(x.T).T


def deq_weights(w):
    q, s = ref.quantise_weights(w)
    return q * ref.spread(ref.spread(s, w.shape[0], 0), w.shape[1], 1)


def reference(logits, x, dy, W1, W2, k, kw):
    T, d = x.shape
    E, f2, _ = W1.shape
    f = f2 // 2
    r = ref.route(logits, k, **kw)
    w = r["topk_w"].astype(np.float32).astype(np.float64)
    n = r["offsets"][-1]
    xp = x[r["src_tok"][:n]]
    ab, yp = np.zeros((n, f2)), np.zeros((n, d))
    Wq = [[deq_weights(w_[e]) for e in range(E)] for w_ in (W1, W2)]
    seg = [slice(r["offsets"][e], r["offsets"][e + 1]) for e in range(E)]
    xq = deq_rows(xp)
    for e in range(E):
        ab[seg[e]] = ref.bf16(xq[seg[e]] @ Wq[0][e].T)
    h = ref.swiglu(ab)
    hq = deq_rows(h)
    for e in range(E):
        yp[seg[e]] = ref.bf16(hq[seg[e]] @ Wq[1][e].T)
    y, dw = np.zeros((T, d)), np.zeros((T, k))
    dyp, dxp, dh = np.zeros((n, d)), np.zeros((n, d)), np.zeros((n, f))
    for t in range(T):
        for j in range(k):
            p = r["dest_row"][t, j]
            if p >= 0:
                y[t] += w[t, j] * yp[p]
                dw[t, j] = dy[t] @ yp[p]
                dyp[p] = ref.bf16((w[t, j] * dy[t]).astype(np.float32))
    kg = {n_: kw[n_] for n_ in ("score", "renorm", "scale")}
    out = {"y": ref.bf16(y), "dlogits": ref.route_grad(logits, r["topk_idx"], dw, **kg)}
    dyq = deq_rows(dyp)
    for e in range(E):
        dh[seg[e]] = ref.bf16(dyq[seg[e]] @ Wq[1][e])
    dab = ref.swiglu_bwd(dh, ab)
    dabq = deq_rows(dab)
    dW1, dW2 = np.zeros(W1.shape), np.zeros(W2.shape)
    for e in range(E):
        s = seg[e]
        dxp[s] = ref.bf16(dabq[s] @ Wq[0][e])
        for lo in range(s.start, s.stop, 128):
            b = slice(lo, min(lo + 128, s.stop))
            dW2[e] += deq_cols(dyp[b]).T @ deq_cols(h[b])
            dW1[e] += deq_cols(dab[b]).T @ deq_cols(xp[b])
    dx = np.zeros((T, d))
    for t in range(T):
        for j in range(k):
            if r["dest_row"][t, j] >= 0:
                dx[t] += dxp[r["dest_row"][t, j]]
    return {**out, "dx": dx, "dW1": dW1, "dW2": dW2}, r


@pytest.mark.parametrize("T,d,E,k,f,kw,fp32", [
    (200, 128, 8, 2, 256, dict(score="softmax", renorm=True, scale=1.0), False),
    (150, 192, 16, 4, 64, dict(score="sigmoid", groups=4, top_groups=2, group_top=2, renorm=True,
                               scale=2.5, bias=True, capacity=40), True),
    (1, 256, 8, 3, 128, dict(score="softmax", renorm=False, scale=1.0), True),
])
def test_layer_forward_and_backward(T, d, E, k, f, kw, fp32):
    rng = np.random.default_rng(T)
    g = lambda *s: f64(dev(rng.normal(size=s).astype(np.float32)).bfloat16())  # noqa: E731
    x, dy = g(T, d), g(T, d)
    W1, W2 = 0.25 * g(E, 2 * f, d), 0.25 * g(E, d, f)     # exact in bf16
    logits = rng.normal(size=(T, E)).astype(np.float32)
    if T > 10:
        logits[5] = -np.inf                               # a padding token
    kw = dict(kw)
    if kw.get("bias"):
        kw["bias"] = (0.1 * rng.normal(size=E)).astype(np.float32)
    o, r = reference(logits, x, dy, W1, W2, k, kw)
    bias = dev(kw["bias"]) if kw.get("bias") is not None else None
    cfg = tde.make_config(T, d, E, k, f, route_scale=kw["scale"], capacity=kw.get("capacity", 0))
    router = tde.make_router(kw["score"], kw.get("groups", 1), kw.get("top_groups"),
                             kw.get("group_top", 1), kw["renorm"], bias)
    layer = tde.Fp8MoELayer(cfg, router, grad_dtype=torch.float32 if fp32 else None)
    b = lambda v: dev(v.astype(np.float32)).bfloat16()  # noqa: E731
    w = layer.quantize_weights(b(W1), b(W2))
    lg, xd, dyd = dev(logits), b(x), b(dy)
    for _ in range(2):      # the second pass overwrites every buffer of the first
        y = layer.forward(lg, xd, w)
        grads = layer.backward(lg, xd, dyd, w)
    assert layer.status()[1] == 0
    assert np.array_equal(layer.r["dest_row"].cpu().numpy(), r["dest_row"])
    assert_close("y", f64(y), o["y"], max_tol=0.1)
    for n in ("dx", "dW1", "dW2", "dlogits"):
        assert_close(n, f64(grads[n]), o[n], max_tol=0.1)
    assert (f64(grads["dW1"])[r["kept"] == 0] == 0).all()


def test_example_learns():
    """The example's update is plain gradient descent with a small step: the loss falls."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                    "examples"))
    import fp8_moe_training_step as ex
    losses = ex.train(tokens=300, width=256, ffn=128, experts=16, k=4, groups=4, top_groups=2,
                      steps=5, log=lambda s: None)
    assert losses == sorted(losses, reverse=True) and losses[-1] < 0.999 * losses[0]
