"""Group-limited routing and its gradient against the plain 64-bit references.

Indices, counts, offsets and the side arrays are compared exactly.  Weights: every step in the
kernel is a correctly rounded fp32 operation (2^-24) or an expf (2^-23), at most about 24 of
them with the warp's sums, so 2^-19 relative; the argument of an exponential is a difference of
logits, whose rounding (2^-24 of it) passes into the result, so the bound grows with the
logits' range.  Gradients are sums of k differences of weights' gradients: the same bound
relative to the largest magnitude in the token's row.
"""

import numpy as np
import pytest
import torch

import block_ref as ref
import token_dispatch_expert_gb300 as tde
from gpu_util import dev, np_i

pytestmark = pytest.mark.gpu
KEYS = ["topk_idx", "topk_w", "counts", "kept", "offsets", "dest_row", "src_tok", "src_slot",
        "drop_mask"]


def call(logits, k, *, score="softmax", groups=1, top_groups=None, group_top=1, renorm=True,
         bias=None, scale=1.0, capacity=0, stream=None):
    T, E = logits.shape
    cfg = tde.make_config(T, 64, E, k, 64, route_scale=scale, capacity=capacity)
    b = None if bias is None else dev(bias.astype(np.float32))
    router = tde.make_router(score, groups, top_groups, group_top, renorm, b)
    ws = torch.empty(tde.moe_workspace_size(cfg)[0], dtype=torch.uint8, device="cuda")
    tde.moe_ws_init(ws)
    i32 = dict(dtype=torch.int32, device="cuda")
    r = {"topk_idx": torch.full((T, k), -9, **i32), "topk_w": torch.full((T, k), 9.0, device="cuda"),
         "counts": torch.full((E,), -9, **i32), "kept": torch.full((E,), -9, **i32),
         "offsets": torch.full((E + 1,), -9, **i32), "dest_row": torch.full((T, k), -9, **i32),
         "src_tok": torch.full((T * k,), -9, **i32), "src_slot": torch.full((T * k,), -9, **i32),
         "drop_mask": torch.full((T, k), 9, dtype=torch.uint8, device="cuda")}
    lg = dev(logits)
    tde.moe_route_groups(cfg, router, lg, *[r[n] for n in KEYS], ws, stream)
    return cfg, router, lg, ws, r


def weight_tol(logits):
    l = logits[np.isfinite(logits)]
    span = min(float(np.ptp(l)), 100.0) if l.size else 0.0
    return 2.0 ** -19 + 2.0 ** -23 * span


def check(logits, k, **kw):
    _, _, _, ws, r = call(logits, k, **kw)
    o = ref.route(logits, k, **kw)
    for n in KEYS:
        if n != "topk_w":
            assert np.array_equal(np_i(r[n]).astype(np.int64).reshape(-1), o[n].reshape(-1)), n
    w = np_i(r["topk_w"]).astype(np.float64)
    assert np.isfinite(w).all()
    # weights below fp32's normal numbers may lose their last bits
    assert (np.abs(w - o["topk_w"]) <= weight_tol(logits) * np.abs(o["topk_w"]) + 1e-37).all()
    return ws, o


def draw(T, E, seed, scale=1.0):
    return (np.random.default_rng(seed).normal(size=(T, E)) * scale).astype(np.float32)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,groups,top,group_top,k", [
    (256, 8, 4, 2, 8), (256, 8, 3, 1, 8), (64, 1, 1, 1, 6), (160, 8, 3, 2, 6), (10, 5, 2, 2, 3),
    (60, 4, 1, 2, 8), (32, 32, 8, 1, 8), (2, 1, 1, 1, 1), (128, 16, 16, 1, 8), (7, 1, 1, 1, 7)])
@pytest.mark.parametrize("T", [1, 32, 33, 257])
def test_choice_and_weights(score, renorm, E, groups, top, group_top, k, T):
    rng = np.random.default_rng(T * E)
    for bias in (None, 0.1 * rng.normal(size=E).astype(np.float32)):
        check(draw(T, E, T + E), k, score=score, renorm=renorm, groups=groups, top_groups=top,
              group_top=group_top, bias=bias, scale=2.5)


@pytest.mark.parametrize("T", [3, 100])
@pytest.mark.parametrize("capacity", [1, 5])
def test_capacity(T, capacity):
    check(draw(T, 16, 3) + np.linspace(3, 0, 16, dtype=np.float32), 4, capacity=capacity,
          score="sigmoid", groups=4, top_groups=2, group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("bias", [False, True])
def test_masks(score, renorm, bias):
    """Experts out of service, tokens with fewer than k in service and with none, masks of the
    type's lowest value, infinities."""
    l = draw(70, 24, 5)
    l[3] = -np.inf
    l[4, 5:] = -np.inf
    l[5, :23] = -np.inf
    l[6] = np.finfo(np.float32).min
    l[7, ::2] = np.finfo(np.float32).min
    l[8, 3] = np.inf
    l[9, [3, 20]] = np.inf
    l[10] = -200.0
    l[11] = np.arange(24) - 300.0
    l[12, ::3] = -np.inf
    l[13] = 50.0 + np.arange(24)
    b = np.linspace(-0.2, 0.2, 24).astype(np.float32) if bias else None
    for groups, top, gt in ((1, 1, 1), (4, 2, 1), (4, 2, 2)):
        _, o = check(l, 6, score=score, renorm=renorm, groups=groups, top_groups=top,
                     group_top=gt, bias=b)
        assert (o["topk_idx"][3] == -1).all() and (o["topk_idx"][5] >= 0).sum() == 1


@pytest.mark.parametrize("group_top", [1, 2])
def test_ties_go_to_the_lower_index(group_top):
    l = np.zeros((40, 64), np.float32)
    l[1] = -0.0
    l[2, 32:] = 1.0
    l[3] = np.tile([1, 0, 1, 0], 16)
    for bias in (None, np.zeros(64, np.float32), np.tile([0.5, 0.25], 32).astype(np.float32)):
        for score in ("softmax", "sigmoid"):
            _, o = check(l, 4, score=score, groups=8, top_groups=2, group_top=group_top, bias=bias)
    assert (o["topk_idx"][0] == [0, 2, 4, 6]).all()


def test_keys_closer_than_fp32_can_tell():
    """Biases that cancel the scores' differences to within 1e-9: the order of the sums in 64
    bits, which fp32 sums cannot give."""
    rng = np.random.default_rng(2)
    T, E = 200, 64
    l = np.round(rng.normal(size=(T, E)) * 4).astype(np.float32) / 4
    for score in ("sigmoid", "softmax"):
        bias = (0.3 - ref.route_scores(l[0].astype(np.float64), score)).astype(np.float32)
        l[1::2] = l[0]
        l[1::2, 7] += 1e-6 * np.arange(100, dtype=np.float32)
        for groups, top, gt in ((1, 1, 1), (8, 4, 2), (8, 4, 1)):
            check(l, 8, score=score, bias=bias, groups=groups, top_groups=top, group_top=gt)


def test_nan_is_out_of_service_and_flagged():
    l = draw(40, 16, 8)
    l[5, 2] = np.nan
    l[6] = np.nan
    ws, o = check(l, 4, score="sigmoid", groups=4, top_groups=2)
    assert (o["topk_idx"][6] == -1).all() and 2 not in o["topk_idx"][5]
    status, flags = tde.moe_status(ws)
    assert flags == tde.DEVERR["NAN_LOGIT"]


def test_another_stream_and_a_graph():
    l = draw(300, 64, 9)
    o = ref.route(l, 6, score="sigmoid", groups=8, top_groups=3, group_top=2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        cfg, router, lg, ws, r = call(l, 6, score="sigmoid", groups=8, top_groups=3, group_top=2,
                                      stream=s)
    s.synchronize()
    assert np.array_equal(np_i(r["topk_idx"]), o["topk_idx"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tde.moe_route_groups(cfg, router, lg, *[r[n] for n in KEYS], ws)
    l2 = draw(300, 64, 10)
    lg.copy_(dev(l2))
    g.replay()
    torch.cuda.synchronize()
    o = ref.route(l2, 6, score="sigmoid", groups=8, top_groups=3, group_top=2)
    for n in KEYS:
        if n != "topk_w":
            assert np.array_equal(np_i(r[n]).reshape(-1), o[n].reshape(-1)), n


# ------------------------------------------------------------------ gradient
def grad(cfg, router, lg, idx, dw, ws):
    out = torch.full_like(lg, 9.0)
    tde.moe_route_groups_bwd(cfg, router, lg, idx, dw, out, ws)
    return out


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (33, 256, 8), (100, 60, 6), (257, 128, 1), (5, 7, 7)])
def test_gradient(score, renorm, T, E, k):
    l = draw(T, E, T + E, 2.0)
    cfg, router, lg, ws, r = call(l, k, score=score, renorm=renorm, scale=2.5)
    dw = np.random.default_rng(1).normal(size=(T, k)).astype(np.float32)
    got = np_i(grad(cfg, router, lg, r["topk_idx"], dev(dw), ws)).astype(np.float64)
    o = ref.route_grad(l, np_i(r["topk_idx"]), dw, score=score, renorm=renorm, scale=2.5)
    tol = weight_tol(l) * 2.5 * np.abs(dw).max(1, keepdims=True)
    assert (np.abs(got - o) <= tol).all()
    if k == 1 and renorm:
        assert (got == 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(score, renorm):
    """Central differences of sum(w dw) in 64 bits, with the choice held fixed."""
    T, E, k = 6, 12, 3
    l = draw(T, E, 4)
    cfg, router, lg, ws, r = call(l, k, score=score, renorm=renorm, scale=1.5)
    dw = np.random.default_rng(2).normal(size=(T, k)).astype(np.float32)
    got = np_i(grad(cfg, router, lg, r["topk_idx"], dev(dw), ws)).astype(np.float64)
    idx = np_i(r["topk_idx"])

    def value(x, t):
        s = ref.route_scores(x, score)
        return float(ref.route_weights(x, idx[t], s, score, renorm, 1.5) @ dw[t])

    h = 1e-5
    for t in range(T):
        for e in range(E):
            x = l[t].astype(np.float64)
            up, dn = x.copy(), x.copy()
            up[e] += h
            dn[e] -= h
            # differences: h^2 / 6 of a third derivative (below 10 here) and rounding / h
            assert abs((value(up, t) - value(dn, t)) / (2 * h) - got[t, e]) <= 1e-8 + 2.0 ** -19 * 4


def test_gradient_with_masks_and_bad_indices():
    l = draw(40, 24, 6)
    l[3] = -np.inf
    l[4, 2:] = -np.inf
    l[5, ::2] = -np.inf
    l[6, 0] = 40.0          # one score carries almost all the weight
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            cfg, router, lg, ws, r = call(l, 4, score=score, renorm=renorm)
            dw = np.random.default_rng(3).normal(size=(40, 4)).astype(np.float32)
            got = np_i(grad(cfg, router, lg, r["topk_idx"], dev(dw), ws)).astype(np.float64)
            with np.errstate(invalid="ignore"):
                o = ref.route_grad(l, np_i(r["topk_idx"]), dw, score=score, renorm=renorm)
            ok = np.arange(40) != 3
            assert (got[3] == 0).all() and np.isfinite(got).all()
            assert (np.abs(got - o)[ok] <= weight_tol(l) * np.abs(dw).max()).all()
            assert tde.moe_status(ws)[1] == 0
            idx = r["topk_idx"].clone()
            idx[7, 1] = 24
            idx[8, 0] = -2
            bad = np_i(grad(cfg, router, lg, idx, dev(dw), ws))
            assert np.isfinite(bad).all()
            assert tde.moe_status(ws)[1] == tde.DEVERR["BAD_INDEX"]


def test_combine_backward_gives_the_weights_gradient():
    """dyp and dw of moe_combine_bwd_dw: dyp as moe_combine_bwd writes it, dw within the rounding
    of d fp32 products summed pairwise in a warp."""
    T, d, E, k = 50, 192, 8, 3
    rng = np.random.default_rng(1)
    l = draw(T, E, 2)
    cfg = tde.make_config(T, d, E, k, 64, capacity=14)
    ws = torch.empty(tde.moe_workspace_size(cfg)[0], dtype=torch.uint8, device="cuda")
    tde.moe_ws_init(ws)
    _, _, lg, _, r = call(l, k, capacity=14)
    dy = dev(rng.normal(size=(T, d)).astype(np.float32)).bfloat16()
    yp = dev(rng.normal(size=(T * k, d)).astype(np.float32)).bfloat16()
    dyp, dyp2 = torch.zeros_like(yp), torch.zeros_like(yp)
    dw, dl = torch.full((T, k), 9.0, device="cuda"), torch.empty_like(lg)
    tde.moe_combine_bwd_dw(cfg, dy, yp, r["topk_w"], r["dest_row"], dyp, dw, ws)
    tde.moe_combine_bwd(cfg, dy, yp, lg, r["topk_idx"], r["topk_w"], r["dest_row"], dyp2, dl, ws)
    assert torch.equal(dyp, dyp2)
    p = np_i(r["dest_row"])
    f = lambda t: t.float().cpu().numpy().astype(np.float64)  # noqa: E731
    o = np.where(p >= 0, np.einsum("td,tkd->tk", f(dy), f(yp)[p]), 0.0)
    assert (p < 0).any()
    mag = np.einsum("td,tkd->tk", np.abs(f(dy)), np.abs(f(yp)[p]))
    assert (np.abs(np_i(dw) - o) <= 32 * 2.0 ** -24 * mag).all() and (np_i(dw)[p < 0] == 0).all()
