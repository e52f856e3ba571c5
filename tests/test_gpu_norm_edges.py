"""The norms and their gradient on rows that hold NaN, infinities or one value throughout, and in
place, at widths of whole vectors, of single elements and past what stays in registers.

A row is compared with the 64-bit definition of that row: where the definition has no number there
must be none, and the other rows must not notice.  Bounds: test_gpu_norm.py's.
"""

import numpy as np
import pytest
import torch

import rows_ref as ref
import token_dispatch_expert_gb300 as tde
from rows_ref import DT, Guarded, U, f32, f64
from test_gpu_norm import E18, check_stats, check_y, rows_of, run_bwd

pytestmark = pytest.mark.gpu
WIDTHS = [1, 64, 129, 300, 513, 1413, 4096, 4097, 12001, 17000, 17001]


def special(C, x):
    """Rows 0, 6 and 7 are ordinary; 1 zeros, 2 and 3 constant, then a NaN and infinities."""
    v = np.random.default_rng(C).normal(size=(10, C))
    v[1], v[2], v[3] = 0.0, 3.0, 0.1
    v[4, C // 2], v[5, C - 1], v[8, 0] = np.nan, np.inf, -np.inf
    v[9, C - 1], v[9, 0] = np.inf, -np.inf
    return ref.typed(v, x)


def quiet(f, *a):
    with np.errstate(all="ignore"):
        return f(*a)


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("x", ["bf16", "fp32"])
def test_special_rows(C, kind, x):
    v = special(C, x)
    X, Y = Guarded(10, C, DT[x]), Guarded(10, C, torch.float32)
    X.put(v)
    g = ref.typed(1 + 0.3 * np.random.default_rng(2).normal(size=C), "fp32")
    gd = torch.from_numpy(g.astype(np.float32)).cuda()
    c, s = ref.checkpoint(10, C, "int8")
    codes = ref.codes_of(c, "int8")
    mean, rstd = torch.empty(10, device="cuda"), torch.empty(10, device="cuda")
    tde.moe_norm(X.t, Y.t, gd, mean=mean if kind == "layer" else None, rstd=rstd, codes=codes, scales=s.t,
                 kind=kind)
    want = quiet(ref.norm, v, g, 0.0, kind, 1e-5)
    got = f64(Y.t)
    assert (np.isnan(got) == np.isnan(want)).all()
    fine = [0, 1, 2, 3, 6, 7]
    check_y("y", got[fine], v[fine], g, 0.0, kind, 1e-5, "fp32")
    check_stats(mean[fine] if kind == "layer" else None, rstd[fine], v[fine], kind, 1e-5)
    Y.check_guards("y")
    # blocks of the checkpoint that hold a NaN or an infinity are NaN, the others theirs
    back = torch.empty((10, C), device="cuda")
    tde.moe_ckpt_load(codes, s.t, back, ws=ref.new_ws())
    nan = np.zeros((10, -(-C // 128)), bool)
    for r, col in np.argwhere(~np.isfinite(v)):
        nan[r, col // 128] = True
    nan = np.repeat(nan, 128, 1)[:, :C]
    assert (np.isnan(f64(back)) == nan).all()
    q, sc = ref.quantise(np.where(nan, 0, v), "int8")
    ref.same("restored", f64(back)[~nan], ref.restore(q, sc)[~nan])


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("fmt", ["", "int8", "e4m3"])
def test_gradient_of_special_rows(C, kind, fmt):
    """The rows' statistics are the definition's, so that NaN and infinities come through them too."""
    rng = np.random.default_rng(C)
    v = special(C, "fp32")
    m, r = (f32(a) for a in quiet(ref.stats, v, kind, 1e-5))
    if fmt:
        finite = np.where(np.isfinite(v), v, 0.0)
        X, scales, _ = ref.device_checkpoint(finite, fmt)
        for row, col in np.argwhere(~np.isfinite(v)):     # as they are kept: the block's scale is no number
            scales[row, col // 128] = float("nan")
            X.view(torch.int8)[row, col // 128 * 128:(col // 128 + 1) * 128] = 0
        v = ref.unrounded(X, scales, C)
    else:
        G = Guarded(10, C, torch.float32)
        X, scales = G.put(v), None
    dy = ref.typed(rng.normal(size=(10, C)), "bf16")
    dy[6, C // 3] = np.nan                       # ... and one in what comes from behind
    DY, DX = Guarded(10, C, torch.bfloat16), Guarded(10, C, torch.float32)
    DY.put(dy)
    ws = ref.new_ws(tde.moe_norm_ws_size(10, C))
    dg, db = torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
    put = lambda a: torch.from_numpy(a.astype(np.float32)).cuda()  # noqa: E731
    tde.moe_norm_bwd(DY.t, X, put(m) if kind == "layer" else None, put(r), DX.t, dg, db, scales=scales, kind=kind,
                     ws=ws)
    dx, dgamma, dbeta = quiet(ref.norm_bwd, dy, v, m, r, 1.0, 0.0, kind)
    got = f64(DX.t)
    assert (np.isnan(got) == np.isnan(dx)).all()
    assert (np.isnan(f64(dg)) == np.isnan(dgamma)).all() and (np.isnan(f64(db)) == np.isnan(dbeta)).all()
    ok = [0, 1, 2, 3, 7]
    xh = np.abs(v[ok] - m[ok, None]) * r[ok, None]
    G_ = np.abs(dy[ok])
    mean = lambda a: a.mean(1, keepdims=True)  # noqa: E731
    ref.check("dx", got[ok], dx[ok], E18 * r[ok, None] * (G_ + mean(G_) + xh * mean(G_ * xh)) + U * np.abs(dx[ok]) + 1e-38)
    DX.check_guards("dx")
    assert tde.moe_status(ws) == (0, 0)


def test_row_without_spread_and_eps():
    """All zeros and eps = 0: 0 / 0."""
    for C in (64, 1413, 17001):
        for kind in ("layer", "rms"):
            x = torch.zeros((3, C), device="cuda")
            x[1].normal_()
            y = torch.empty_like(x)
            tde.moe_norm(x, y, eps=0.0, kind=kind)
            assert torch.isnan(y[0]).all() and torch.isnan(y[2]).all()
            check_y("y", y[1:2], f64(x[1:2]), 1.0, 0.0, kind, 0.0, "fp32")


@pytest.mark.parametrize("C", [64, 513, 1413, 4096, 4097, 12001, 17000, 17001])
@pytest.mark.parametrize("x,pad", [("bf16", 0), ("bf16", 3), ("fp32", 0), ("fp32", 3), ("fp32", 4)])
def test_in_place(C, x, pad):
    """total over x and y over the residual, and the other way round; rows may be strided."""
    rng = np.random.default_rng(C)
    R = 9
    a, b = rows_of(rng, R, C, x), rows_of(rng, R, C, x)
    v = ref.typed(f32(a + b), x)
    for other in (False, True):
        X, S = Guarded(R, C, DT[x], C + pad, pad), Guarded(R, C, DT[x], C + pad, pad)
        X.put(a)
        S.put(b)
        total, y = (S, X) if other else (X, S)
        mean, rstd = torch.empty(R, device="cuda"), torch.empty(R, device="cuda")
        tde.moe_norm(X.t, y.t, residual=S.t, total=total.t, mean=mean, rstd=rstd)
        ref.same("total", total.t, v)
        check_y("y", y.t, v, 1.0, 0.0, "layer", 1e-5, x)
        check_stats(mean, rstd, v, "layer", 1e-5)
        X.check_guards("x")
        S.check_guards("residual")
    X = Guarded(R, C, DT[x], C + pad, pad)       # y over x alone
    X.put(v)
    tde.moe_norm(X.t, X.t)
    check_y("y", X.t, v, 1.0, 0.0, "layer", 1e-5, x)
    X.check_guards("x")


@pytest.mark.parametrize("C", [64, 513, 1413, 4096, 4097, 12001, 17000, 17001])
@pytest.mark.parametrize("x,pad", [("bf16", 0), ("bf16", 3), ("fp32", 0), ("fp32", 3), ("fp32", 4)])
def test_gradient_in_place(C, x, pad):
    """dx over add and dx over dy give the bits of a call with buffers of its own."""
    rng = np.random.default_rng(C)
    R = 9
    v, dy, ad = (rows_of(rng, R, C, x) for _ in range(3))
    m, r = ref.stats(v, "layer", 1e-5)
    md, rd = (torch.from_numpy(a.astype(np.float32)).cuda() for a in (m, r))
    ws = ref.new_ws(tde.moe_norm_ws_size(R, C))

    def buf(a):
        G = Guarded(R, C, DT[x], C + pad, pad)
        G.put(a)
        return G
    V, out = buf(v), []
    for into in ("new", "add", "dy"):
        DY, A = buf(dy), buf(ad)
        DX = {"new": buf(0 * v), "add": A, "dy": DY}[into]
        dg, db = torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
        tde.moe_norm_bwd(DY.t, V.t, md, rd, DX.t, dg, db, add=A.t, ws=ws)
        out.append((DX.t.clone(), dg, db))
        DX.check_guards("dx")
    for o in out[1:]:
        assert all(torch.equal(s, t) for s, t in zip(out[0], o))
    want, _, _ = ref.norm_bwd(dy, v, f64(md), f64(rd), 1.0, ad, "layer")
    xh = np.abs(v - m[:, None]) * r[:, None]
    mean = lambda a: np.abs(a).mean(1, keepdims=True)  # noqa: E731
    ref.check("dx", out[0][0], want, E18 * r[:, None] * (np.abs(dy) + mean(dy) + xh * mean(dy * xh)) +
              2 * U * np.abs(ad) + 1.01 * ref.HALF[x] * np.abs(want) + 1e-38)
    assert tde.moe_status(ws) == (0, 0)


@pytest.mark.parametrize("C,R", [(3, 20001), (77, 20001), (1413, 5001), (4099, 2003)])
@pytest.mark.parametrize("first", [1, 5])
def test_gradient_of_dense_rows_off_16_bytes(C, R, first):
    """The first and last rows' ends are cut off a piece of 16 bytes and written by plain stores; the
    rows that take their places later come whole."""
    run_bwd(np.random.default_rng(C), R, C, "layer", "bf16", "bf16", "fp32", True, "", first=first, offset=1.0)
