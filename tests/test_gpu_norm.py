"""moe_norm, moe_norm_bwd and moe_ckpt_norm against 64-bit numpy.

Bounds.  A sum over a row is a chain of at most 8 elements, 4 chunks (16 in the wide form), 5
shuffles and 16 warps, 45 additions, so it is off by at most 45 U times the sum of magnitudes (U =
2^-24); the mean's error is mended by the mean of the differences, whose own is 45 U of their
magnitudes' mean, at most the standard deviation.  So (v - m) rstd is off by 45 U, plus as much times
|xhat| through rstd (half of the squares' 45 U, and rsqrtf's 2 ulp), and one rounding for each
operation: with xhat = (v - m) rstd,
    y:   2^-18 (|gamma| (|xhat| + 1) + |beta|) + half a step of y's type
    dx:  the two means are off by 50 U of the means of magnitudes: 2^-18 rstd (|G| + mean |G| +
         |xhat| mean |G xhat|), an operation's rounding for add, and half a step
    dgamma, dbeta: rows / 152 rows one after another (fewer CTAs than SMs only for fewer rows), 4
         warps, 38 parts and 16 sums: U (rows / 152 + 80) times the sum of magnitudes, and half a step
2^-18 = 64 U.
"""

import numpy as np
import pytest
import torch

import rows_ref as ref
import token_dispatch_expert_gb300 as tde
from rows_ref import DT, Guarded, U, f32, f64

pytestmark = pytest.mark.gpu
E18 = 2.0 ** -18


def rows_of(rng, R, C, name, offset=0.0):
    """Rows of different scales, as numbers of the type."""
    v = rng.normal(size=(R, C)) * np.exp(rng.uniform(-1, 2, (R, 1))) + offset
    return ref.typed(v, name)


def params(rng, C, name, layer=True):
    g, b = 1 + 0.3 * rng.normal(size=C), 0.2 * rng.normal(size=C)
    g, b = ref.typed(g, name), ref.typed(b, name)
    to = lambda v: torch.from_numpy(v.astype(np.float32)).to(DT[name]).cuda()  # noqa: E731
    return g, b, to(g), to(b)


def check_y(name, got, v, gamma, beta, kind, eps, yt):
    m, r = ref.stats(v, kind, eps)
    want = ref.norm(v, gamma, beta, kind, eps)
    xh = np.abs(v - m[:, None]) * r[:, None]
    ref.check(name, got, want, E18 * (np.abs(gamma) * (xh + 1) + np.abs(beta)) +
              ref.HALF[yt] * np.abs(want) * 1.01 + 1e-38)


def check_stats(mean, rstd, v, kind, eps):
    m, r = ref.stats(v, kind, eps)
    if mean is not None:
        ref.check("mean", mean, m, U * np.abs(m) + E18 * v.std(1) + 1e-38)
    ref.check("rstd", rstd, r, E18 * r)


WIDTHS = [1, 2, 7, 64, 100, 127, 128, 129, 256, 257, 512, 513, 1000, 1024, 1413, 2056, 4096, 7168,
          9001, 11999, 13579, 16002, 16384, 16392, 20010, 33001]


def run_norm(rng, R, C, kind, x, y, p, add, fmt, eps=1e-5, offset=0.0, first=0, pad=0):
    v = rows_of(rng, R, C, x, offset)
    X = Guarded(R, C, DT[x], C + pad, first)
    X.put(v)
    res = Res = T = None
    if add:
        res = rows_of(rng, R, C, x)
        Res = Guarded(R, C, DT[x], C + 2 * pad, first)
        Res.put(res)
        T = Guarded(R, C, DT[x], C + pad, first)
        v = ref.typed(f32(v + res), x)
    g, b, gd, bd = params(rng, C, p)
    Y = Guarded(R, C, DT[y], C + pad, first)
    S = [Guarded(1, R, torch.float32) for _ in range(2)]
    mean, rstd = S[0].t[0], S[1].t[0]
    c = s = None
    if fmt:
        c, s = ref.checkpoint(R, C, fmt)
    tde.moe_norm(X.t, Y.t, gd, bd, residual=Res and Res.t, total=T and T.t,
                 mean=mean if kind == "layer" else None, rstd=rstd,
                 codes=ref.codes_of(c, fmt) if c else None, scales=s.t if s else None, eps=eps,
                 kind=kind)
    check_y("y", Y.t, v, g, b, kind, eps, y)
    check_stats(mean if kind == "layer" else None, rstd, v, kind, eps)
    if add:
        ref.same("total", T.t, v)
        T.check_guards("total")
    if fmt:
        q, sc = ref.quantise(v, fmt)
        ref.same("codes", ref.code_values(c, fmt), q)
        ref.same("scales", s.t, sc)
        c.check_guards("codes")
        s.check_guards("scales")
    Y.check_guards("y")
    for g_ in S:
        g_.check_guards("statistics", None if kind == "layer" or g_ is S[1] else 0)


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("kind,x,y,p,add,fmt", [
    ("layer", "bf16", "bf16", "fp32", True, "int8"), ("layer", "fp32", "bf16", "bf16", False, "e4m3"),
    ("rms", "fp32", "fp32", "fp32", True, "int8"), ("rms", "bf16", "fp32", "bf16", False, "")])
def test_norm(C, kind, x, y, p, add, fmt):
    run_norm(np.random.default_rng(C), 5 if C > 4096 else 37, C, kind, x, y, p, add, fmt)


@pytest.mark.parametrize("C,first,pad", [(64, 1, 1), (512, 2, 6), (1024, 8, 8), (1000, 4, 4),
                                         (4096, 1, 3), (7168, 2, 2), (16640, 3, 5), (300, 8, 12)])
@pytest.mark.parametrize("x", ["bf16", "fp32"])
def test_norm_of_strided_rows(C, first, pad, x):
    run_norm(np.random.default_rng(C), 9, C, "layer", x, "bf16", "fp32", True, "int8", first=first,
             pad=pad)


@pytest.mark.parametrize("R", [1, 2, 3, 4, 5, 700, 3001])
@pytest.mark.parametrize("C", [96, 640, 1413])
def test_norm_of_few_and_many_rows(R, C):
    run_norm(np.random.default_rng(R), R, C, "layer", "bf16", "bf16", "bf16", True, "e4m3")


@pytest.mark.parametrize("C", [100, 2048, 4097, 20000])
def test_norm_far_from_zero(C):
    """A mean of a thousand standard deviations, in fp32: the differences from the mean are exact to
    U of the mean's magnitude, which 64-bit differences of the same numbers see in full."""
    rng = np.random.default_rng(C)
    v = f32(1000 + rng.normal(size=(6, C)))
    X, Y = Guarded(6, C, torch.float32), Guarded(6, C, torch.float32)
    X.put(v)
    mean, rstd = torch.empty(6, device="cuda"), torch.empty(6, device="cuda")
    tde.moe_norm(X.t, Y.t, mean=mean, rstd=rstd)
    check_stats(mean, rstd, v, "layer", 1e-5)
    m, r = ref.stats(v, "layer", 1e-5)
    # v - mean0 is exact (both lie within a factor of two), so xhat's bound stands as it is
    want = ref.norm(v, 1.0, 0.0, "layer", 1e-5)
    ref.check("y", Y.t, want, E18 * (np.abs(want) + 1))


@pytest.mark.parametrize("C", [192, 4096, 17000])
def test_norm_special_rows(C):
    """Constant rows, zeros, NaN and infinities: each row for itself."""
    x = np.random.default_rng(1).normal(size=(8, C))
    x = ref.typed(x, "bf16")
    x[1], x[2] = 0.0, 3.0
    x[3, 5], x[4, C - 1], x[5, 0] = np.nan, np.inf, -np.inf
    xd = torch.from_numpy(x.astype(np.float32)).cuda().bfloat16()
    y, (c, s) = torch.empty_like(xd), ref.checkpoint(8, C, "int8")
    codes = ref.codes_of(c, "int8")
    tde.moe_norm(xd, y, codes=codes, scales=s.t)
    got = f64(y)
    assert np.isnan(got[3:6]).all()
    assert (got[1:3] == 0).all()
    fine = [0, 6, 7]
    check_y("y", got[fine], x[fine], 1.0, 0.0, "layer", 1e-5, "bf16")
    back = torch.empty_like(xd)
    tde.moe_ckpt_load(codes, s.t, back, ws=ref.new_ws())
    b = f64(back)
    # the blocks that hold them restore as NaN, the others as they would without
    for r, col in ((3, 5), (4, C - 1), (5, 0)):
        lo = col // 128 * 128
        assert np.isnan(b[r, lo:lo + 128]).all()
        assert not np.isnan(np.delete(b[r], np.s_[lo:lo + 128])).any()
    assert (ref.code_values(c, "int8")[3, :128] == 0).all()


def test_norm_in_place():
    rng = np.random.default_rng(3)
    for C in (500, 4096, 20000):
        x, r = rows_of(rng, 7, C, "bf16"), rows_of(rng, 7, C, "bf16")
        v = ref.typed(f32(x + r), "bf16")
        xd, rd = (torch.from_numpy(a.astype(np.float32)).cuda().bfloat16() for a in (x, r))
        tde.moe_norm(xd, rd, residual=rd, total=xd)      # total over x, y over the residual
        ref.same("total", xd, v)
        check_y("y", rd, v, 1.0, 0.0, "layer", 1e-5, "bf16")


def test_empty_norm():
    for T in (torch.bfloat16, torch.float32):
        x = torch.empty((0, 64), dtype=T, device="cuda")
        tde.moe_norm(x, torch.empty_like(x))
        g = [torch.full((64,), 7.0, device="cuda") for _ in range(2)]
        none = torch.empty(0, device="cuda")
        tde.moe_norm_bwd(x, x, none, none, torch.empty_like(x), *g, ws=ref.new_ws())
        assert not g[0].any() and not g[1].any()


# --------------------------------------------------------------------------- the gradient
def run_bwd(rng, R, C, kind, x, y, p, add, fmt, gt="fp32", first=0, pad=0, offset=0.0):
    v = rows_of(rng, R, C, x, offset)
    eps = 1e-5
    m, r = (f32(a) for a in ref.stats(v, kind, eps))
    if fmt:
        X, scales, _ = ref.device_checkpoint(v, fmt)
        v = ref.unrounded(X, scales, C)      # code * scale - mean is rounded once
    else:
        G = Guarded(R, C, DT[x], C + pad, first)
        X, scales = G.put(v), None
    dy = rows_of(rng, R, C, y)
    DY = Guarded(R, C, DT[y], C + pad, first)
    DY.put(dy)
    ad, A = 0.0, None
    if add:
        ad = rows_of(rng, R, C, x)
        A = Guarded(R, C, DT[x], C + 2 * pad, first)
        A.put(ad)
    g, _, gd, _ = params(rng, C, p)
    DX = Guarded(R, C, DT[x], C + pad, first)
    D = [Guarded(1, C, DT[gt]) for _ in range(2)]
    md, rd = (torch.from_numpy(a.astype(np.float32)).cuda() for a in (m, r))
    ws = ref.new_ws(tde.moe_norm_ws_size(R, C))
    args = dict(gamma=gd, scales=scales, add=A and A.t, kind=kind, ws=ws)
    tde.moe_norm_bwd(DY.t, X, md if kind == "layer" else None, rd, DX.t, D[0].t[0], D[1].t[0], **args)
    dx, dg, db = ref.norm_bwd(dy, v, m, r, g, ad, kind)
    xh = (v - m[:, None]) * r[:, None]
    G_ = dy * g
    mean = lambda a: np.abs(a).mean(1, keepdims=True)  # noqa: E731
    ref.check("dx", DX.t, dx, E18 * r[:, None] * (np.abs(G_) + mean(G_) + np.abs(xh) * mean(G_ * xh)) +
              2 * U * np.abs(ad) + 1.01 * ref.HALF[x] * np.abs(dx) + 1e-38)
    chain = U * (R / 152 + 80)
    ref.check("dgamma", D[0].t[0], dg, chain * np.abs(dy * xh).sum(0) + 1.01 * ref.HALF[gt] * np.abs(dg))
    ref.check("dbeta", D[1].t[0], db, chain * np.abs(dy).sum(0) + 1.01 * ref.HALF[gt] * np.abs(db))
    for n, o in (("dx", DX), ("dgamma", D[0]), ("dbeta", D[1])):
        o.check_guards(n)
    # the same bits again, also with one of the sums alone
    first = [t.clone() for t in (DX.t, D[0].t, D[1].t)]
    tde.moe_norm_bwd(DY.t, X, md if kind == "layer" else None, rd, DX.t, D[0].t[0], None, **args)
    tde.moe_norm_bwd(DY.t, X, md if kind == "layer" else None, rd, DX.t, None, D[1].t[0], **args)
    assert all(torch.equal(a, b) for a, b in zip(first, (DX.t, D[0].t, D[1].t)))
    tde.moe_norm_bwd(DY.t, X, md if kind == "layer" else None, rd, DX.t, **args)
    assert torch.equal(first[0], DX.t)
    assert tde.moe_status(ws) == (0, 0)


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("kind,x,y,p,add,fmt,gt", [
    ("layer", "bf16", "bf16", "fp32", True, "", "fp32"), ("layer", "fp32", "bf16", "bf16", False, "int8", "bf16"),
    ("rms", "fp32", "fp32", "fp32", True, "e4m3", "fp32"), ("rms", "bf16", "fp32", "bf16", True, "", "fp32"),
    ("layer", "bf16", "bf16", "bf16", False, "e4m3", "fp32")])
def test_norm_bwd(C, kind, x, y, p, add, fmt, gt):
    run_bwd(np.random.default_rng(C), 5 if C > 4096 else 37, C, kind, x, y, p, add, fmt, gt)


@pytest.mark.parametrize("C,first,pad", [(64, 1, 1), (512, 2, 6), (1024, 8, 8), (1000, 4, 4),
                                         (4096, 1, 3), (7168, 2, 2), (16640, 3, 5), (300, 8, 12)])
@pytest.mark.parametrize("x,fmt", [("bf16", ""), ("fp32", ""), ("bf16", "int8")])
def test_norm_bwd_of_strided_rows(C, first, pad, x, fmt):
    run_bwd(np.random.default_rng(C), 9, C, "layer", x, "bf16", "fp32", True, fmt, first=first, pad=pad)


@pytest.mark.parametrize("R", [1, 2, 3, 5, 607, 608, 609, 1300, 5001])
@pytest.mark.parametrize("C", [72, 640, 1413, 2048])
def test_norm_bwd_of_few_and_many_rows(R, C):
    """Around the number of CTAs, and past it."""
    run_bwd(np.random.default_rng(R), R, C, "layer", "bf16", "bf16", "fp32", True, "", offset=2.0)


def test_norm_bwd_in_place():
    rng = np.random.default_rng(5)
    for C in (500, 4096, 20000):
        v, dy, ad = (rows_of(rng, 6, C, "bf16") for _ in range(3))
        to = lambda a: torch.from_numpy(a.astype(np.float32)).cuda().bfloat16()  # noqa: E731
        m, r = ref.stats(v, "layer", 1e-5)
        md, rd = (torch.from_numpy(a.astype(np.float32)).cuda() for a in (m, r))
        ws = ref.new_ws(tde.moe_norm_ws_size(6, C))
        want = torch.empty_like(to(v))
        tde.moe_norm_bwd(to(dy), to(v), md, rd, want, add=to(ad), ws=ws)
        over_add, over_dy = to(ad), to(dy)
        tde.moe_norm_bwd(to(dy), to(v), md, rd, over_add, add=over_add, ws=ws)
        tde.moe_norm_bwd(over_dy, to(v), md, rd, over_dy, add=to(ad), ws=ws)
        assert torch.equal(want, over_add) and torch.equal(want, over_dy)


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_gradient_against_differences(kind):
    """Central differences of the 64-bit definition, step h: off by h^2 / 6 times a third derivative
    of order one and 2^-52 / h, about 1e-8 for h = 1e-5 on these numbers; the kernel's fp32 result
    by E18 of the terms."""
    rng = np.random.default_rng(11)
    R, C, h = 3, 70, 1e-5
    x, g, b, dy = (f32(rng.normal(size=s)) for s in ((R, C), C, C, (R, C)))
    loss = lambda x_, g_, b_: (ref.norm(x_, g_, b_, kind, 1e-5) * dy).sum()  # noqa: E731
    to = lambda a: torch.from_numpy(a.astype(np.float32)).cuda()  # noqa: E731
    y, dx = to(x), to(x)
    mean, rstd = (torch.empty(R, device="cuda") for _ in range(2))
    tde.moe_norm(to(x), y, to(g), to(b), mean=mean if kind == "layer" else None, rstd=rstd, kind=kind)
    dg, db = to(g), to(b)
    tde.moe_norm_bwd(to(dy), to(x), mean if kind == "layer" else None, rstd, dx, dg, db, gamma=to(g),
                     kind=kind, ws=ref.new_ws(tde.moe_norm_ws_size(R, C)))

    def slope(a, i, at):
        args = [x, g, b]
        out = []
        for sign in (1, -1):
            moved = a.copy()
            moved[i] += sign * h
            args[at] = moved
            out.append(loss(*args))
        return (out[0] - out[1]) / (2 * h)

    tol = E18 * 40 + 1e-6
    for at, (a, got) in enumerate(((x, dx), (g, dg), (b, db))):
        want = np.zeros(a.shape)
        for i in np.ndindex(a.shape):
            want[i] = slope(a, i, at)
        ref.check(("dx", "dgamma", "dbeta")[at], got, want, tol)


# --------------------------------------------------------------------------- from the checkpoint
@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("kind,fmt,y,p", [("layer", "int8", "bf16", "fp32"), ("rms", "e4m3", "fp32", "bf16")])
def test_ckpt_norm(C, kind, fmt, y, p):
    rng = np.random.default_rng(C)
    R = 5 if C > 4096 else 37
    v = rows_of(rng, R, C, "bf16", 0.5)
    m, r = (f32(a) for a in ref.stats(v, kind, 1e-5))
    codes, scales, _ = ref.device_checkpoint(v, fmt)
    v = ref.unrounded(codes, scales, C)      # code * scale - mean is rounded once
    g, b, gd, bd = params(rng, C, p)
    Y = Guarded(R, C, DT[y], C + 8, 8)
    md, rd = (torch.from_numpy(a.astype(np.float32)).cuda() for a in (m, r))
    tde.moe_ckpt_norm(codes, scales, md if kind == "layer" else None, rd, Y.t, gd, bd, kind=kind)
    xh = (v - m[:, None]) * r[:, None]
    want = xh * g + b
    # one rounding for each of four operations
    ref.check("y", Y.t, want, 4 * U * (np.abs(xh * g) + np.abs(b)) + 1.01 * ref.HALF[y] * np.abs(want) + 1e-38)
    Y.check_guards("y")


# --------------------------------------------------------------------------- streams, graphs, sizes
def test_norm_on_another_stream_and_in_graphs():
    """Two captured graphs that share one workspace, replayed in turn with other inputs, and calls
    on a stream of their own give what eager calls give."""
    rng = np.random.default_rng(9)
    R, C = 300, 1536
    mk = lambda: torch.from_numpy(rows_of(rng, R, C, "bf16").astype(np.float32)).cuda().bfloat16()  # noqa: E731
    gamma = torch.rand(C, device="cuda") + 0.5
    ws = ref.new_ws(tde.moe_norm_ws_size(R, C))

    def buffers():
        n = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
        return dict(x=mk(), dy=mk(), y=n(R, C, dt=torch.bfloat16), mean=n(R), rstd=n(R),
                    dx=n(R, C, dt=torch.bfloat16), dg=n(C), db=n(C),
                    codes=n(R, C, dt=torch.int8), scales=n(R, C // 128))

    def step(b):
        tde.moe_norm(b["x"], b["y"], gamma, mean=b["mean"], rstd=b["rstd"], codes=b["codes"],
                     scales=b["scales"])
        tde.moe_norm_bwd(b["dy"], b["codes"], b["mean"], b["rstd"], b["dx"], b["dg"], b["db"],
                         gamma=gamma, scales=b["scales"], ws=ws)

    sets = [buffers(), buffers()]
    for b in sets:
        step(b)
    torch.cuda.synchronize()
    graphs = []
    for b in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(b)
        graphs.append(g)
    for _ in range(2):
        for b in sets:
            b["x"].copy_(mk())
            b["dy"].copy_(mk())
        for g in graphs + graphs:
            g.replay()
        got = [{k: v.clone() for k, v in b.items()} for b in sets]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        for b in sets:
            for k in ("y", "dx", "dg", "db", "codes"):
                b[k].zero_()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for b in sets:
                step(b)
        torch.cuda.current_stream().wait_stream(side)
        for b, o in zip(sets, got):
            assert all(torch.equal(b[k], o[k]) for k in b)
            check_y("y", o["y"], f64(o["x"]), f64(gamma), 0.0, "layer", 1e-5, "bf16")


def test_norm_past_2_31_elements():
    """Rows whose offsets pass 31 bits: the last rows are right."""
    R, C = 66000, 32896
    x = torch.empty((R, C), dtype=torch.bfloat16, device="cuda").normal_()
    y = torch.empty_like(x)
    mean, rstd = torch.empty(R, device="cuda"), torch.empty(R, device="cuda")
    tde.moe_norm(x, y, mean=mean, rstd=rstd)
    for r in (0, R // 2, R - 1):
        check_y("y", y[r:r + 1], f64(x[r:r + 1]), 1.0, 0.0, "layer", 1e-5, "bf16")
    n = 3
    at = R - n
    dx = torch.empty_like(y)
    tde.moe_norm_bwd(y, x, mean, rstd, dx, ws=ref.new_ws())
    v, dy = f64(x[at:]), f64(y[at:])
    m, r = f64(mean[at:]), f64(rstd[at:])
    want, _, _ = ref.norm_bwd(dy, v, m, r, 1.0, 0.0, "layer")
    # here G = dy is xhat itself: the terms cancel to eps' share, so the bound is the terms'
    xh = np.abs(v - m[:, None]) * r[:, None]
    tol = E18 * r[:, None] * (np.abs(dy) + 1 + xh * 1.1) + ref.HALF["bf16"] * np.abs(want)
    ref.check("dx", dx[at:], want, tol)
