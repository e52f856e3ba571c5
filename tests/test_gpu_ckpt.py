"""The 8-bit checkpoints and what is computed from them, against 64-bit numpy.

Codes, scales, restored rows and dyp are single roundings of the definition: compared bit by bit.
SwiGLU values: sigma's error (rows_ref.sigmoid_error) and half a bf16 step; in da it enters through
s, through a s (1 - s) and, in 1 - s, absolutely: (1 + 2 |a|) times.  CUDA's fast division gives 0
for a divisor above 2^126, so that a sigma below 2^-126 is lost: LOST = 2^-126 times what multiplies
it.  dw: a chain of 8 products, a
row's 256-column steps and 5 shuffles.
"""

import numpy as np
import pytest
import torch

import rows_ref as ref
import token_dispatch_expert_gb300 as tde
from rows_ref import DT, Guarded, U, f32, f64

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
LOST = 2.0 ** -126
WIDTHS = [1, 2, 6, 16, 100, 127, 128, 130, 256, 264, 384, 1001, 1536, 2050, 2816, 7168]


def values(rng, R, C, name):
    v = rng.normal(size=(R, C)) * np.exp(rng.uniform(-3, 3, (R, 1)))
    v[:, rng.integers(0, C)] *= 20
    return ref.typed(v, name)


def offsets(n, G=3):
    return torch.tensor([0] * G + [n], dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("x,fmt,first,pad", [("bf16", "int8", 0, 0), ("fp32", "e4m3", 0, 0),
                                             ("fp32", "int8", 1, 3), ("bf16", "e4m3", 2, 2)])
def test_save_and_load(C, x, fmt, first, pad):
    rng = np.random.default_rng(C)
    R, live = 41, 33
    v = values(rng, R, C, x)
    v[7] = 0.0
    v[8, :] = 2.0 ** -120 if x == "bf16" else 1e-40     # under the floor of the largest magnitude
    v[9, 0] = 3.0e38
    v = ref.typed(v, x)
    X = Guarded(R, C, DT[x], C + pad, first)
    X.put(v)
    c, s = ref.checkpoint(R, C, fmt)
    ws = ref.new_ws()
    tde.moe_ckpt_save(X.t, ref.codes_of(c, fmt), s.t, offsets=offsets(live), ws=ws)
    q, sc = ref.quantise(v[:live], fmt)
    ref.same("codes", ref.code_values(c, fmt)[:live], q)
    ref.same("scales", s.t[:live], sc)
    c.check_guards("codes", live)
    s.check_guards("scales", live)
    B = Guarded(R, C, DT[x], C + pad, first)
    tde.moe_ckpt_load(ref.codes_of(c, fmt), s.t, B.t, offsets=offsets(live), ws=ws)
    want = ref.restore(q, sc)
    ref.same("rows", B.t[:live], ref.typed(want, x))
    B.check_guards("rows", live)
    if fmt == "int8":    # a value is off by at most half a scale, and the roundings on the way
        off = np.abs(want - v[:live])
        assert (off <= np.repeat(sc, 128, 1)[:, :C] * (0.5 + 200 * U)).all()
    assert tde.moe_status(ws) == (0, 0)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_ties_and_neighbours(fmt):
    """Products that lie on and next to the middle of two codes."""
    v = np.zeros((64, 128))
    rng = np.random.default_rng(0)
    v[:, 0] = 127.0 if fmt == "int8" else 448.0      # factor 1: codes are the rounded values
    v[:, 1:] = np.round(rng.uniform(-120, 120, (64, 127))) + 0.5
    v[1:, 1:] *= 1 + rng.integers(-3, 4, (63, 127)) * 2.0 ** -20
    v[32:] *= rng.uniform(0.1, 9, (32, 1))
    v = f32(v)
    X = Guarded(64, 128, torch.float32)
    X.put(v)
    c, s = ref.checkpoint(64, 128, fmt)
    tde.moe_ckpt_save(X.t, ref.codes_of(c, fmt), s.t, ws=ref.new_ws())
    q, sc = ref.quantise(v, fmt)
    ref.same("codes", ref.code_values(c, fmt), q)
    ref.same("scales", s.t, sc)


def test_e4m3_checkpoint_is_the_quantisers():
    x = torch.randn((300, 1544), device="cuda").bfloat16()
    new = lambda: (torch.zeros((300, 1552), dtype=torch.float8_e4m3fn, device="cuda"),  # noqa: E731
                   torch.zeros((300, 13), device="cuda"))
    a, b = new(), new()
    ws = ref.new_ws()
    tde.moe_fp8_quantize(x, *a, ws=ws)
    tde.moe_ckpt_save(x, *b, ws=ws)
    assert torch.equal(a[0].view(torch.int8), b[0].view(torch.int8)) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("n,flag,rows", [(-1, 8, 0), (21, 8, 20), (20, 0, 20), (0, 0, 0)])
def test_live_rows(n, flag, rows):
    """A count outside the rows is held to them and flagged; nothing behind it is written."""
    x = torch.randn((20, 256), device="cuda").bfloat16()
    ws = ref.new_ws()
    c, s = ref.checkpoint(20, 256, "int8")
    codes = ref.codes_of(c, "int8")
    o = [Guarded(20, w, BF) for w in (256, 256, 128, 256, 128)]
    full = torch.zeros((20, 256), dtype=torch.int8, device="cuda"), torch.ones((20, 2), device="cuda")
    for call in (lambda: tde.moe_ckpt_save(x, codes, s.t, offsets=offsets(n), ws=ws),
                 lambda: tde.moe_ckpt_load(*full, o[0].t, offsets=offsets(n), ws=ws),
                 lambda: tde.moe_ckpt_swiglu(*full, o[1].t, o[2].t, offsets=offsets(n), ws=ws),
                 lambda: tde.moe_ckpt_swiglu_bwd(x[:, :128].contiguous(), *full, o[3].t, o[4].t,
                                                 offsets=offsets(n), ws=ws)):
        call()
        assert tde.moe_status(ws)[1] == flag
    for g in [c, s] + o:
        g.check_guards("output", rows)


@pytest.mark.parametrize("f", [1, 2, 5, 32, 100, 127, 128, 192, 257, 704, 768, 1409, 2052, 4096])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_swiglu(f, fmt):
    rng = np.random.default_rng(f)
    R, live = 19, 17
    ab = values(rng, R, 2 * f, "bf16")
    ab[3, :f] = ref.typed(np.linspace(-150, 150, f), "bf16")
    codes, scales, v = ref.device_checkpoint(ab, fmt)
    a, b = v[:live, :f], v[:live, f:]
    AB, H = Guarded(R, 2 * f, BF), Guarded(R, f, BF)
    ws = ref.new_ws()
    tde.moe_ckpt_swiglu(codes, scales, AB.t, H.t, offsets=offsets(live), ws=ws)
    ref.same("ab", AB.t[:live], ref.typed(v[:live], "bf16"))
    h = ref.swiglu(a, b)
    htol = np.abs(h) * (1.01 * ref.HALF["bf16"] + ref.sigmoid_error(a)) + LOST * (1 + np.abs(a * b))
    ref.check("h", H.t[:live], h, htol)
    AB.check_guards("ab", live)
    H.check_guards("h", live)
    # each alone
    one, two = torch.zeros_like(AB.t), torch.zeros_like(H.t)
    tde.moe_ckpt_swiglu(codes, scales, one, offsets=offsets(live), ws=ws)
    tde.moe_ckpt_swiglu(codes, scales, None, two, offsets=offsets(live), ws=ws)
    assert torch.equal(one[:live], AB.t[:live]) and torch.equal(two[:live], H.t[:live])
    # the gradient
    dh = values(rng, R, f, "bf16")
    D, H2 = Guarded(R, 2 * f, BF), Guarded(R, f, BF)
    dhd = torch.from_numpy(dh.astype(np.float32)).cuda().bfloat16()
    tde.moe_ckpt_swiglu_bwd(dhd, codes, scales, D.t, H2.t, offsets=offsets(live), ws=ws)
    dh = dh[:live]
    da, db = ref.swiglu_bwd(dh, a, b)
    s = ref.sigmoid(a)
    half = 1.01 * ref.HALF["bf16"]
    ref.check("da", D.t[:live, :f], da, half * np.abs(da) + LOST * (1 + np.abs(dh * b) * (1 + np.abs(a))) +
              np.abs(dh * b) * s * (1 + 2 * np.abs(a)) * ref.sigmoid_error(a))
    ref.check("db", D.t[:live, f:], db, np.abs(db) * (half + ref.sigmoid_error(a)) + LOST * (1 + np.abs(dh * a)))
    ref.check("h", H2.t[:live], h, htol)
    D.check_guards("dab", live)
    H2.check_guards("h", live)
    again = torch.zeros_like(D.t)
    tde.moe_ckpt_swiglu_bwd(dhd, codes, scales, again, offsets=offsets(live), ws=ws)
    assert torch.equal(again[:live], D.t[:live])
    assert tde.moe_status(ws) == (0, 0)


def test_swiglu_gradient_against_differences():
    """Central differences of silu(a) b in 64 bits at the restored values (off by about 1e-9)."""
    rng = np.random.default_rng(2)
    R, f, h = 16, 64, 1e-5
    codes, scales, v = ref.device_checkpoint(ref.typed(rng.normal(size=(R, 2 * f)) * 2, "bf16"), "int8")
    dh = ref.typed(rng.normal(size=(R, f)), "bf16")
    D = torch.empty((R, 2 * f), dtype=BF, device="cuda")
    tde.moe_ckpt_swiglu_bwd(torch.from_numpy(dh.astype(np.float32)).cuda().bfloat16(), codes, scales, D,
                            ws=ref.new_ws())
    a, b = v[:, :f], v[:, f:]
    da = dh * (ref.swiglu(a + h, b) - ref.swiglu(a - h, b)) / (2 * h)
    db = dh * (ref.swiglu(a, b + h) - ref.swiglu(a, b - h)) / (2 * h)
    for n, got, want in (("da", D[:, :f], da), ("db", D[:, f:], db)):
        ref.check(n, got, want, 1.01 * ref.HALF["bf16"] * np.abs(want) + 1e-4)


def test_nonfinite_values_stay_in_their_block():
    v = np.ones((6, 512))
    v[1, 3], v[2, 130], v[3, 300] = np.nan, np.inf, -np.inf
    for fmt in ("int8", "e4m3"):
        X = Guarded(6, 512, torch.float32)
        X.put(v)
        c, s = ref.checkpoint(6, 512, fmt)
        ws = ref.new_ws()
        codes = ref.codes_of(c, fmt)
        tde.moe_ckpt_save(X.t, codes, s.t, ws=ws)
        back = torch.empty((6, 512), device="cuda")
        tde.moe_ckpt_load(codes, s.t, back, ws=ws)
        h = torch.empty((6, 256), dtype=BF, device="cuda")
        tde.moe_ckpt_swiglu(codes, s.t, None, h, ws=ws)
        bad = np.zeros((6, 4), bool)
        bad[1, 0] = bad[2, 1] = bad[3, 2] = True
        nan = np.repeat(bad, 128, 1)
        assert (np.isnan(f64(back)) == nan).all()
        assert (np.isnan(f64(h)) == (nan[:, :256] | nan[:, 256:])).all()
        assert np.allclose(f64(back)[~nan], 1, rtol=2 * U, atol=0)


def dispatch(rng, T, k, dropped):
    """Rows of the slots: a random permutation with holes; dropped slots -1."""
    d = rng.permutation(T * k).reshape(T, k)
    return np.where(rng.random((T, k)) < dropped, -1, d).astype(np.int32)


@pytest.mark.parametrize("T,k,d,dropped", [(1, 1, 64, 0.0), (1, 8, 7168, 0.0), (13, 2, 128, 0.3),
                                           (50, 3, 320, 0.1), (70, 4, 1024, 0.0), (33, 5, 2048, 0.2),
                                           (40, 6, 192, 0.0), (300, 7, 512, 0.1), (20, 8, 4096, 1.0),
                                           (2000, 2, 256, 0.05)])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_combine_bwd(T, k, d, dropped, fmt):
    rng = np.random.default_rng(T * k)
    cfg = tde.make_config(T, d, 16, k, 64)
    codes, scales, yp = ref.device_checkpoint(values(rng, T * k, d, "bf16"), fmt)
    # as the definition has it: code times scale, not yet rounded to 32 bits
    q = f64(codes)[:, :d]
    yp = q * np.repeat(f64(scales), 128, 1)[:, :d]
    dest = dispatch(rng, T, k, dropped)
    dy = values(rng, T, d, "bf16")
    w = f32(rng.random((T, k)))
    P, W = Guarded(T * k, d, BF), Guarded(T, k, torch.float32)
    ws = ref.new_ws()
    dev = lambda a: torch.from_numpy(np.asarray(a, np.float32)).cuda()  # noqa: E731
    tde.moe_ckpt_combine_bwd(cfg, dev(dy).bfloat16(), codes, scales, dev(w),
                             torch.from_numpy(dest).cuda(), P.t, W.t, ws)
    got, keep = f64(P.t), np.ones(T * k, bool)
    pattern = f64(torch.full((2,), ref.PATTERN, dtype=torch.uint8).view(BF))[0]
    for t in range(T):
        for j in range(k):
            p = dest[t, j]
            if p < 0:
                assert float(W.t[t, j]) == 0
                continue
            keep[p] = False
            ref.same("dyp", got[p], ref.typed(f32(w[t, j] * dy[t]), "bf16"))
            tol = U * (16 + d / 256 + 6) * np.abs(dy[t] * yp[p]).sum()
            ref.check("dw", f64(W.t)[t, j:j + 1], np.array([dy[t] @ yp[p]]), tol)
    assert (got[keep] == pattern).all()          # rows that no slot names are left as they were
    P.check_guards("dyp")
    W.check_guards("dw")
    assert tde.moe_status(ws) == (0, 0)


def test_combine_bwd_flags_bad_rows():
    T, k, d = 4, 2, 128
    cfg = tde.make_config(T, d, 8, k, 64)
    codes, scales, _ = ref.device_checkpoint(np.ones((8, d)), "int8")
    dest = torch.tensor([[0, 1], [2, 8], [-2, 3], [4, 5]], dtype=torch.int32, device="cuda")
    P, W = Guarded(8, d, BF), torch.full((T, k), 9.0, device="cuda")
    ws = ref.new_ws()
    tde.moe_ckpt_combine_bwd(cfg, torch.ones((T, d), dtype=BF, device="cuda"), codes, scales,
                             torch.ones((T, k), device="cuda"), dest, P.t, W, ws)
    assert tde.moe_status(ws)[1] == tde.DEVERR["BAD_INDEX"]
    assert f64(W)[1, 1] == 0 and f64(W)[2, 0] == 0
    P.check_guards("dyp", 6)


def test_past_2_31_elements():
    """Codes, rows and both halves of [a | b] whose offsets pass 31 bits."""
    R, C = 66000, 33024
    x = torch.empty((R, C), dtype=BF, device="cuda").normal_()
    codes = torch.empty((R, C), dtype=torch.int8, device="cuda")
    scales = torch.empty((R, C // 128), device="cuda")
    ws = ref.new_ws()
    tde.moe_ckpt_save(x, codes, scales, ws=ws)
    at = [0, 65000, R - 1]
    q, s = ref.quantise(f64(x[at]), "int8")
    ref.same("codes", codes[at], q)
    ref.same("scales", scales[at], s)
    v = ref.restore(q, s)
    tde.moe_ckpt_load(codes, scales, x, ws=ws)
    ref.same("rows", x[at], ref.typed(v, "bf16"))
    h = torch.empty((R, C // 2), dtype=BF, device="cuda")
    tde.moe_ckpt_swiglu(codes, scales, x, h, ws=ws)
    a, b = v[:, :C // 2], v[:, C // 2:]
    want = ref.swiglu(a, b)
    ref.check("h", h[at], want, np.abs(want) * (1.01 * ref.HALF["bf16"] + ref.sigmoid_error(a)) + 1e-38)
    tde.moe_ckpt_swiglu_bwd(h, codes, scales, x, ws=ws)
    dh = f64(h[at])
    db = ref.swiglu_bwd(dh, a, b)[1]
    ref.check("db", x[at][:, C // 2:], db,
              np.abs(db) * (1.01 * ref.HALF["bf16"] + ref.sigmoid_error(a)) + 1e-38)


def test_checkpoints_in_graphs_and_on_another_stream():
    R, f = 700, 320
    x = torch.empty((R, 2 * f), dtype=BF, device="cuda")
    dh = torch.randn((R, f), device="cuda").bfloat16()
    ws = ref.new_ws()
    off = offsets(650)
    new = lambda: dict(codes=torch.zeros((R, 2 * f), dtype=torch.int8, device="cuda"),  # noqa: E731
                       scales=torch.zeros((R, 5), device="cuda"), x=torch.zeros_like(x),
                       ab=torch.zeros_like(x), h=torch.zeros_like(dh), dab=torch.zeros_like(x))

    def step(o):
        tde.moe_ckpt_save(x, o["codes"], o["scales"], offsets=off, ws=ws)
        c = o["codes"], o["scales"]
        tde.moe_ckpt_load(*c, o["x"], offsets=off, ws=ws)
        tde.moe_ckpt_swiglu(*c, o["ab"], o["h"], offsets=off, ws=ws)
        tde.moe_ckpt_swiglu_bwd(dh, *c, o["dab"], offsets=off, ws=ws)

    o = new()
    g = torch.cuda.CUDAGraph()
    x.normal_()
    step(o)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step(o)
    x.normal_()
    g.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    e = new()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(e)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(o[k], e[k]) for k in o)
    assert torch.equal(o["x"], o["ab"])
