"""The layers that keep 8-bit checkpoints, as a training step uses them, against the same path in 64-bit
numpy (quantised and rounded where the layers quantise and round); the norm's module; blocks of both that
share their scratch (their numbers: test_gpu_prenorm_block.py).

Tolerances as in the tests of the layers that they are built from: bf16 products within 2e-2 of rms +
|o| (gpu_util), products of 8-bit operands within 0.1 (test_gpu_fp8_layer).
"""

import os
import sys

import numpy as np
import pytest
import torch

import block_ref
import rows_ref as ref
import test_gpu_fp8_layer as fp8
import token_dispatch_expert_gb300 as tde
from gpu_util import assert_close, dev
from rows_ref import f64

pytestmark = pytest.mark.gpu


def bf(a):
    return dev(np.asarray(a, np.float32)).bfloat16()


def inputs(rng, T, d, E, f):
    x, dy = (ref.typed(rng.normal(size=(T, d)), "bf16") for _ in range(2))
    W1 = ref.typed(0.2 * rng.normal(size=(E, 2 * f, d)), "bf16")
    W2 = ref.typed(0.2 * rng.normal(size=(E, d, f)), "bf16")
    return x, dy, W1, W2, rng.normal(size=(T, E)).astype(np.float32)


def kept(v, fmt):
    q, s = ref.quantise(v, fmt)
    return ref.restore(q, s)


def reference(logits, x, dy, W1, W2, k, r, gate, scale, fmt):
    """Forward and backward from the checkpoints; r: the routing (checked by other tests)."""
    T, d = x.shape
    E, f = W1.shape[0], W1.shape[1] // 2
    n = r["offsets"][-1]
    seg = [slice(r["offsets"][e], r["offsets"][e + 1]) for e in range(E)]
    xp = x[r["src_tok"][:n]]
    ab, yp = np.zeros((n, 2 * f)), np.zeros((n, d))
    for e in range(E):
        ab[seg[e]] = ref.typed(xp[seg[e]] @ W1[e].T, "bf16")
    h = ref.typed(ref.swiglu(ab[:, :f], ab[:, f:]), "bf16")
    for e in range(E):
        yp[seg[e]] = ref.typed(h[seg[e]] @ W2[e].T, "bf16")
    w, y, dw = r["topk_w"], np.zeros((T, d)), np.zeros((T, k))
    ypk, abk = kept(yp, fmt), kept(ab, fmt)
    hk, abk = ref.typed(ref.swiglu(abk[:, :f], abk[:, f:]), "bf16"), ref.typed(abk, "bf16")
    dyp, dxp, dab = np.zeros((n, d)), np.zeros((n, d)), np.zeros((n, 2 * f))
    for t in range(T):
        for j in range(k):
            p = r["dest_row"][t, j]
            if p >= 0:
                y[t] += w[t, j] * yp[p]
                dw[t, j] = dy[t] @ ypk[p]
                dyp[p] = ref.typed(w[t, j] * dy[t], "bf16")
    dW1, dW2 = np.zeros(W1.shape), np.zeros(W2.shape)
    for e in range(E):
        s = seg[e]
        da, db = ref.swiglu_bwd(dyp[s] @ W2[e], abk[s, :f], abk[s, f:])
        dab[s] = ref.typed(np.concatenate([da, db], 1), "bf16")
        dxp[s] = ref.typed(dab[s] @ W1[e], "bf16")
        dW1[e], dW2[e] = dab[s].T @ xp[s], dyp[s].T @ hk[s]
    dx = np.zeros((T, d))
    for t in range(T):
        for j in range(k):
            if r["dest_row"][t, j] >= 0:
                dx[t] += dxp[r["dest_row"][t, j]]
    dl = block_ref.route_grad(logits, r["topk_idx"], dw, score=gate, renorm=True, scale=scale)
    return {"y": y, "dx": dx, "dW1": dW1, "dW2": dW2, "dlogits": dl}


@pytest.mark.parametrize("T,d,E,k,f,gate,kw,fmt", [
    (150, 128, 8, 2, 64, "softmax", {}, "int8"),
    (90, 192, 16, 4, 128, "sigmoid", dict(route_scale=2.5, capacity=30), "e4m3"),
    (1, 64, 4, 1, 64, "softmax", {}, "int8"),
    (200, 256, 8, 3, 192, "softmax", dict(drop_negative=True), "int8")])
def test_checkpointed_layer(T, d, E, k, f, gate, kw, fmt):
    rng = np.random.default_rng(T)
    x, dy, W1, W2, logits = inputs(rng, T, d, E, f)
    cfg = tde.make_config(T, d, E, k, f, gate=gate, **kw)
    layer = tde.CheckpointedMoELayer(tde.MoEScratch(cfg), fmt)
    lg, xd, dyd, w1, w2 = dev(logits), bf(x), bf(dy), bf(W1), bf(W2)
    for _ in range(2):
        y = layer.forward(lg, xd, w1, w2)
        g = layer.backward(lg, xd, dyd, w1, w2)
    assert layer.status() == (0, 0)
    r = {n: v.cpu().numpy() for n, v in layer.r.items()}
    r["topk_w"] = r["topk_w"].astype(np.float64)
    o = reference(logits, x, dy, W1, W2, k, r, gate, kw.get("route_scale", 1.0), fmt)
    assert_close("y", f64(y), o["y"])
    for n in ("dx", "dW1", "dW2", "dlogits"):
        assert_close(n, f64(g[n]), o[n])
    # the layer without checkpoints: the same forward
    plain = tde.MoELayer(cfg)
    assert torch.equal(plain.forward(lg, xd, w1, w2), y)


def fp8_reference(logits, x, dy, W1, W2, k, fmt):
    """The 8-bit layer (softmax over the chosen) from its checkpoints: as test_gpu_fp8_layer's, but
    that the backward pass reads the kept tensors."""
    T, d = x.shape
    E, f = W1.shape[0], W1.shape[1] // 2
    r = block_ref.route(logits, k)
    w = ref.f32(r["topk_w"])
    n = r["offsets"][-1]
    seg = [slice(r["offsets"][e], r["offsets"][e + 1]) for e in range(E)]
    xp = x[r["src_tok"][:n]]
    ab, yp = np.zeros((n, 2 * f)), np.zeros((n, d))
    Wq = [[fp8.deq_weights(v[e]) for e in range(E)] for v in (W1, W2)]
    xq = fp8.deq_rows(xp)
    for e in range(E):
        ab[seg[e]] = block_ref.bf16(xq[seg[e]] @ Wq[0][e].T)
    hq = fp8.deq_rows(block_ref.swiglu(ab))
    for e in range(E):
        yp[seg[e]] = block_ref.bf16(hq[seg[e]] @ Wq[1][e].T)
    ypk, abk = kept(yp, fmt), kept(ab, fmt)
    h = ref.typed(ref.swiglu(abk[:, :f], abk[:, f:]), "bf16")
    y, dw, dyp, dxp = np.zeros((T, d)), np.zeros((T, k)), np.zeros((n, d)), np.zeros((n, d))
    slots = [(t, j, r["dest_row"][t, j]) for t in range(T) for j in range(k) if r["dest_row"][t, j] >= 0]
    for t, j, p in slots:
        y[t] += w[t, j] * yp[p]
        dw[t, j] = dy[t] @ ypk[p]
        dyp[p] = ref.typed(w[t, j] * dy[t], "bf16")
    dyq, dh = fp8.deq_rows(dyp), np.zeros((n, f))
    for e in range(E):
        dh[seg[e]] = block_ref.bf16(dyq[seg[e]] @ Wq[1][e])
    dab = ref.typed(np.concatenate(ref.swiglu_bwd(dh, abk[:, :f], abk[:, f:]), 1), "bf16")
    dabq = fp8.deq_rows(dab)
    dW1, dW2, dx = np.zeros(W1.shape), np.zeros(W2.shape), np.zeros((T, d))
    for e in range(E):
        s = seg[e]
        dxp[s] = block_ref.bf16(dabq[s] @ Wq[0][e])
        for lo in range(s.start, s.stop, 128):
            b = slice(lo, min(lo + 128, s.stop))
            dW2[e] += fp8.deq_cols(dyp[b]).T @ fp8.deq_cols(h[b])
            dW1[e] += fp8.deq_cols(dab[b]).T @ fp8.deq_cols(xp[b])
    for t, j, p in slots:
        dx[t] += dxp[p]
    dl = block_ref.route_grad(logits, r["topk_idx"], dw, score="softmax", renorm=True, scale=1.0)
    return {"y": y, "dx": dx, "dW1": dW1, "dW2": dW2, "dlogits": dl}


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_fp8_layer_with_checkpoints(fmt):
    T, d, E, k, f = 200, 128, 8, 2, 256
    rng = np.random.default_rng(1)
    x, dy, W1, W2, logits = inputs(rng, T, d, E, f)
    cfg, router = tde.make_config(T, d, E, k, f), tde.make_router("softmax")
    layer = tde.Fp8MoELayer(cfg, router, checkpoint=fmt)
    other = tde.Fp8MoELayer(cfg, router, checkpoint=fmt, scratch=layer)
    w = layer.quantize_weights(bf(W1), bf(W2))
    lg, xd, dyd = dev(logits), bf(x), bf(dy)
    y = layer.forward(lg, xd, w)
    other.forward(-lg, dyd, w)                 # the scratch holds something else
    g = layer.backward(lg, xd, dyd, w)
    assert layer.status() == (0, 0)
    o = fp8_reference(logits, x, dy, W1, W2, k, fmt)
    assert_close("y", f64(y), o["y"], max_tol=0.1)
    for n in ("dx", "dW1", "dW2", "dlogits"):
        assert_close(n, f64(g[n]), o[n], max_tol=0.1)


def test_blocks_share_their_scratch():
    """Two blocks, forward and backward in the order of a training step: each gives bit by bit what it
    gives alone."""
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import prenorm_moe_training_step as ex
    gen = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    cfg = tde.make_config(300, 256, 8, 2, 128)
    scratch = tde.MoEScratch(cfg)
    blocks = [ex.Block(scratch, rand, "layer", "int8") for _ in range(2)]
    x, br, d = (rand(300, 256).bfloat16() for _ in range(3))
    alone = []
    args = (x, br)
    for b in blocks:
        out = b.forward(*args)
        alone.append((out, b.backward(d, d)))
        args = out
    args = (x, br)
    outs = []
    for b in blocks:
        args = b.forward(*args)
        outs.append(args)
    for i in (1, 0):
        dx, grads = blocks[i].backward(d, d)
        assert torch.equal(dx, alone[i][1][0])
        for n, v in grads.items():
            assert torch.equal(v, alone[i][1][1][n]), n
        assert all(torch.equal(a, b) for a, b in zip(outs[i], alone[i][0]))


@pytest.mark.parametrize("kind,fmt", [("layer", "int8"), ("rms", "e4m3"), ("layer", None), ("rms", None)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_module(kind, fmt, dtype):
    """forward, restore and backward of MoENorm are the entry points' on its buffers."""
    T, d = 70, 384
    x, r = (torch.randn((T, d), device="cuda").to(dtype) for _ in range(2))
    gamma = torch.rand(d, device="cuda") + 0.5
    beta = torch.randn(d, device="cuda") if kind == "layer" else None
    dy, add = torch.randn((T, d), device="cuda").bfloat16(), torch.randn((T, d), device="cuda").to(dtype)
    m = tde.MoENorm(T, d, kind=kind, dtype=dtype, checkpoint=fmt)
    y, s = m.forward(x, gamma, beta, residual=r)
    assert torch.equal(s, (x.float() + r.float()).to(dtype))
    v = f64(s)
    off = 0.0 if beta is None else f64(beta)
    want = ref.norm(v, f64(gamma), off, kind, 1e-5)
    ref.check("y", y, want, 2.0 ** -18 * (np.abs(want) + 10) + 1.01 * ref.HALF["bf16"] * np.abs(want))
    back = m.restore(gamma, beta)
    if fmt is None:
        assert torch.equal(back, y)
    else:     # off by half a scale of int8 (1/254 of a block's largest) or 2^-4 of a value, through rstd
        step = np.abs(v).max(1, keepdims=True) / 254 if fmt == "int8" else np.abs(v) * 2.0 ** -4 + 2.0 ** -9
        _, rs = ref.stats(v, kind, 1e-5)
        ref.check("restored", back, want, 1.01 * step * rs[:, None] * f64(gamma) + 2 * ref.HALF["bf16"] * (np.abs(want) + 1))
    g = m.backward(dy, gamma, add=add, beta=beta is not None)
    assert set(g) == {"dx", "dgamma"} | ({"dbeta"} if beta is not None else set())
    dx = torch.empty_like(s)
    mean, rstd = m.mean, m.rstd
    codes, scales = m.kept or (s, None)
    tde.moe_norm_bwd(dy, codes, mean, rstd, dx, gamma=gamma, scales=scales, add=add, kind=kind, ws=m.ws)
    assert torch.equal(dx, g["dx"]) and g["dx"].dtype is dtype
    assert tde.moe_status(m.ws) == (0, 0)


def test_example_runs():
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import prenorm_moe_training_step as ex
    losses = ex.train(tokens=200, width=256, ffn=128, experts=8, k=2, blocks=2, steps=3, log=lambda s: None)
    assert len(losses) == 3 and np.isfinite(losses).all()
    for kind, fmt in (("rms", "e4m3"), ("layer", "e4m3"), ("rms", "int8")):
        assert np.isfinite(ex.train(tokens=64, width=128, ffn=64, experts=4, k=1, blocks=2, steps=2, kind=kind,
                                    checkpoint=fmt, log=lambda s: None)).all()


FIRST_CALLS_IN_A_CAPTURE = """
import torch
import token_dispatch_expert_gb300 as tde
T, C = 40, {C}
x, dy = (torch.randn((T, C), device="cuda").bfloat16() for _ in range(2))
gamma = torch.rand(C, device="cuda")
new = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device="cuda")
ws = torch.zeros(tde.moe_norm_ws_size(T, C), dtype=torch.uint8, device="cuda")
ld = (C + 15) // 16 * 16
def step(o):
    c = o["codes"], o["scales"]
    tde.moe_norm(x, o["y"], gamma, residual=dy, total=o["s"], mean=o["mean"], rstd=o["rstd"], codes=c[0], scales=c[1])
    tde.moe_norm_bwd(dy, c[0], o["mean"], o["rstd"], o["dx"], o["dg"], o["db"], gamma=gamma, scales=c[1], ws=ws)
    tde.moe_ckpt_norm(*c, o["mean"], o["rstd"], o["n"], gamma)
    tde.moe_ckpt_save(x, *c, ws=ws)
    tde.moe_ckpt_load(*c, o["x"], ws=ws)
    if C % 2 == 0:
        tde.moe_ckpt_swiglu(*c, o["ab"], o["h"], ws=ws)
        tde.moe_ckpt_swiglu_bwd(o["h"], *c, o["dab"], ws=ws)
def buffers():
    bf = torch.bfloat16
    return dict({{n: new(T, C, dt=bf) for n in ("y", "s", "dx", "n", "x", "ab", "dab")}}, h=new(T, C // 2, dt=bf),
                mean=new(T), rstd=new(T), dg=new(C), db=new(C), codes=new(T, ld, dt=torch.int8),
                scales=new(T, (C + 127) // 128))
a, b = buffers(), buffers()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    step(a)
g.replay()
step(b)
assert all(torch.equal(a[n], b[n]) for n in a), [n for n in a if not torch.equal(a[n], b[n])]
assert tde.moe_status(ws) == (0, 0) and bool(a["y"].any()) and bool(a["dg"].any())
print("same")
"""


@pytest.mark.parametrize("C", [4096, 1410, 7169])
def test_first_calls_of_a_process_in_a_capture(C):
    """Whatever the library looks up once (registers, shared memory) it can look up in a capture."""
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS_IN_A_CAPTURE.format(C=C)], cwd=root, capture_output=True,
                       text=True, timeout=120)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_refusals():
    cfg = tde.make_config(64, 128, 8, 2, 64)
    with pytest.raises(ValueError, match="^checkpoint: expected"):
        tde.CheckpointedMoELayer(tde.MoEScratch(cfg), "int4")
    with pytest.raises(ValueError, match="shared expert"):
        tde.CheckpointedMoELayer(tde.MoEScratch(tde.make_config(64, 128, 8, 2, 64, 64)))
    for kw in (dict(recompute=True), dict(mxfp8=1)):
        with pytest.raises(ValueError, match="must be unset"):
            tde.CheckpointedMoELayer(tde.MoEScratch(tde.make_config(64, 128, 8, 2, 128, **kw)))
    r = tde.make_router()
    plain = tde.Fp8MoELayer(cfg, r)
    with pytest.raises(ValueError, match="^scratch: only"):
        tde.Fp8MoELayer(cfg, r, checkpoint="int8", scratch=plain)
    with pytest.raises(ValueError, match="^scratch: expected a layer"):
        tde.Fp8MoELayer(tde.make_config(32, 128, 8, 2, 64), r, checkpoint="int8",
                        scratch=tde.Fp8MoELayer(cfg, r, checkpoint="int8"))
    with pytest.raises(ValueError, match="^kind: expected"):
        tde.MoENorm(4, 64, kind="batch")
    with pytest.raises(ValueError, match="^x: expected"):
        tde.MoENorm(4, 64).forward(torch.zeros((4, 32), dtype=torch.bfloat16, device="cuda"))
