"""8-bit operands with a scale per block of 128, against the plain 64-bit references.

Codes and scales are compared exactly: their definition spells out every rounding.  Products:
with S = sum |A| |B| over the contraction (values, scales applied), the tensor core's fp32 sum of
128 products is off by at most 2^-23 of the sum of magnitudes for each of its additions
(truncation allowed for), the scale's product, its multiplication and the sum over K/128 blocks
by 2^-24 each, so |error| <= (2 * 128 + K / 128 + 3) 2^-24 S, plus half a step of the output
type (bf16 2^-8, fp32 2^-24, relative).  With random signs the actual errors are far smaller;
the typical one is bounded too: rel-L2 <= 2e-6 for fp32 outputs (a random walk of 128 + K / 128
roundings of 2^-24 is below 16 * 6e-8 = 1e-6) and 2^-8 / sqrt(3) + 1e-6 for bf16, over outputs
of at least 1000 elements (a few may all lie next to a rounding border).
"""

import numpy as np
import pytest
import torch

import block_ref as ref
import token_dispatch_expert_gb300 as tde
from gpu_util import dev

pytestmark = pytest.mark.gpu
E4 = torch.float8_e4m3fn


def up(n, m):
    return -(-n // m) * m


def ws_new():
    ws = torch.empty(tde.FP8_WS_BYTES, dtype=torch.uint8, device="cuda")
    tde.moe_ws_init(ws)
    return ws


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def codes_new(shape):
    return torch.full(shape, 0x7f, dtype=torch.uint8, device="cuda").view(E4)   # NaN


def normal(shape, seed, scale=1.0):
    x = np.random.default_rng(seed).normal(size=shape).astype(np.float32) * scale
    return dev(x).bfloat16()


def offsets_of(lengths):
    return [0] + [int(v) for v in np.cumsum(lengths)]


def odev(off):
    return torch.tensor(off, dtype=torch.int32, device="cuda")


def same(got, want, name):
    assert np.array_equal(np.isnan(got), np.isnan(want)), name
    assert np.array_equal(np.nan_to_num(got), np.nan_to_num(want)), name


def check_rows(codes, scales, x, pow2, n=None):
    n = x.shape[0] if n is None else n
    q, s = ref.quantise_rows(x[:n], pow2)
    same(f64(codes[:n, :x.shape[1]]), q, "codes")
    same(f64(scales[:n]), s, "scales")


def check_tokens(codes_t, scales_t, x, off, pow2):
    q, s = ref.quantise_tokens(x, off, pow2)
    same(f64(codes_t[:, :q.shape[1]]), q, "codes_t")
    same(f64(scales_t[:s.shape[0]]), s, "scales_t")


LENGTHS = [[1], [128], [0, 1, 0], [127, 129, 5, 0, 200], [300, 0, 0, 77], [0, 0]]


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("C", [1, 8, 100, 128, 129, 136, 1000, 1024, 1032])
@pytest.mark.parametrize("lengths", LENGTHS)
def test_quantise_rows_and_tokens(lengths, C, pow2):
    off = offsets_of(lengths)
    R, G = off[-1], len(lengths)
    x = normal((max(R, 1), C), R + C)[:R]
    if R > 3 and C > 3:
        x[1] = 0.0
        x[2, :3] = 448.0
        x[:, 2] = 0.0
    ws = ws_new()
    B = tde.moe_fp8_token_blocks(R, G)
    ld = up(C, 16)
    both = [codes_new((R, ld)), torch.empty((R, -(-C // 128)), device="cuda"),
            codes_new((C, 128 * B)), torch.empty((B, C), device="cuda")]
    one = [codes_new((R, ld)), torch.empty_like(both[1]), codes_new((C, 128 * B)),
           torch.empty_like(both[3])]
    o = odev(off)
    tde.moe_fp8_quantize(x, *both, offsets=o, pow2=pow2, ws=ws)
    tde.moe_fp8_quantize(x, one[0], one[1], offsets=o, pow2=pow2, ws=ws)
    tde.moe_fp8_quantize(x, codes_t=one[2], scales_t=one[3], offsets=o, pow2=pow2, ws=ws)
    xv = f64(x)
    for c in (both, one):
        check_rows(c[0], c[1], xv, pow2)
        check_tokens(c[2], c[3], xv, off, pow2)
    assert tde.moe_status(ws)[1] == 0


def test_quantise_without_offsets_strided_and_off_alignment():
    base = normal((70, 400), 3)
    for x in (base[:, :256], base[:, 1:258], base[3:, 8:8 + 130], base[::2, :64], base[:1, 5:6]):
        R, C = x.shape
        ws = ws_new()
        B = tde.moe_fp8_token_blocks(R, 1)
        c = [codes_new((R, up(C, 16) + 16)), torch.empty((R, -(-C // 128)), device="cuda"),
             codes_new((C, 128 * B)), torch.empty((B, C), device="cuda")]
        tde.moe_fp8_quantize(x, *c, ws=ws)
        check_rows(c[0], c[1], f64(x), False)
        check_tokens(c[2], c[3], f64(x), [0, R], False)


def test_quantise_gather_and_bad_indices():
    T, C = 40, 264
    x = normal((T, C), 4)
    src = np.random.default_rng(0).integers(0, T, 150).astype(np.int32)
    off = offsets_of([90, 0, 60])
    ws = ws_new()
    B = tde.moe_fp8_token_blocks(160, 3)
    idx = np.full(160, -1, np.int32)     # ten rows past the segments, as routing leaves them
    idx[:150] = src
    c = [codes_new((160, 272)), torch.empty((160, 3), device="cuda"), codes_new((C, 128 * B)),
         torch.empty((B, C), device="cuda")]
    for parts in (slice(0, 4), slice(0, 2)):
        got = c[parts] + [None] * (4 - len(c[parts]))
        tde.moe_fp8_quantize(x, *got, offsets=odev(off), src_tok=dev(idx), ws=ws)
        check_rows(c[0], c[1], f64(x)[src], False, 150)
    check_tokens(c[2], c[3], f64(x)[src], off, False)
    assert tde.moe_status(ws)[1] == 0
    for bad in (T, -1, 2 ** 30):
        j = idx.copy()
        j[77] = bad
        for got in (c, c[:2] + [None, None]):
            tde.moe_fp8_quantize(x, *got, offsets=odev(off), src_tok=dev(j), ws=ws)
            assert tde.moe_status(ws)[1] == tde.DEVERR["BAD_INDEX"]


def test_bad_offsets_are_flagged():
    x, ws = normal((20, 128), 1), ws_new()
    B = tde.moe_fp8_token_blocks(20, 2)
    c = [codes_new((20, 128)), torch.empty((20, 1), device="cuda"), codes_new((128, 128 * B)),
         torch.empty((B, 128), device="cuda")]
    out = torch.zeros((20, 128), device="cuda")
    dw = torch.zeros((2, 128, 128), device="cuda")
    w = (codes_new((2, 128, 128)), torch.ones((2, 1, 1), device="cuda"))
    for off in ([0, 21, 20], [0, 5, 40], [0, -1, 20], [1, 5, 20]):
        o = odev(off)
        calls = [lambda: tde.moe_fp8_quantize(x, *c, offsets=o, ws=ws),
                 lambda: tde.moe_fp8_gemm(c[0], c[1], *w, out, 128, offsets=o, ws=ws),
                 lambda: tde.moe_fp8_wgrad(c[2], c[3], c[2], c[3], dw, offsets=o, rows=20, ws=ws)]
        for call in calls:
            call()
            assert tde.moe_status(ws)[1] == tde.DEVERR["BAD_OFFSETS"], off


@pytest.mark.parametrize("pow2", [False, True])
def test_extremes(pow2):
    """Zeros, subnormals, the largest numbers, infinities and NaN, in a block of their own."""
    x = np.random.default_rng(5).normal(size=(8, 640)).astype(np.float32)
    big = float(torch.finfo(torch.bfloat16).max)
    x[0, :128] = 0
    x[1, :128] = 1e-39
    x[2, :128] = np.linspace(-1, 1, 128) * big
    x[3, 5] = np.inf
    x[4, 6] = -np.inf
    x[5, 7] = np.nan
    x[6, :128] *= 1e-30
    x[7, :4] = [np.nan, np.inf, -np.inf, big]
    xb = dev(x).bfloat16()
    ws = ws_new()
    B = tde.moe_fp8_token_blocks(8, 1)
    c = [codes_new((8, 640)), torch.empty((8, 5), device="cuda"), codes_new((640, 128 * B)),
         torch.empty((B, 640), device="cuda")]
    tde.moe_fp8_quantize(xb, *c, pow2=pow2, ws=ws)
    v = f64(xb)
    with np.errstate(all="ignore"):
        q, s = ref.quantise_rows(v, pow2)
    same(f64(c[0]), q, "codes")
    same(f64(c[1]), s, "scales")
    # an infinity: the others are 0, itself NaN; a NaN: all NaN
    assert np.isnan(f64(c[0])[3, 5]) and (f64(c[0])[3, :5] == 0).all()
    assert np.isnan(f64(c[0])[5, :128]).all() and np.isfinite(f64(c[0])[5, 128:]).all()


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("G,N,K", [(1, 1, 1), (2, 128, 256), (3, 130, 100), (1, 257, 136),
                                   (2, 16, 1000), (1, 300, 17)])
def test_quantise_weights(G, N, K, pow2):
    w = normal((G, N, K), N + K, 0.02)
    c = [codes_new((G, N, up(K, 16))), torch.empty((G, -(-N // 128), -(-K // 128)), device="cuda"),
         codes_new((G, K, up(N, 16))), torch.empty((G, -(-K // 128), -(-N // 128)), device="cuda")]
    tde.moe_fp8_quantize_weights(w, *c, pow2=pow2)
    for g in range(G):
        q, s = ref.quantise_weights(f64(w[g]), pow2)
        same(f64(c[0][g, :, :K]), q, "codes")
        same(f64(c[1][g]), s, "scales")
        same(f64(c[2][g, :, :N]), q.T, "codes_t")
        same(f64(c[3][g]), s.T, "scales_t")
    d = codes_new((G, N, up(K, 16)))
    tde.moe_fp8_quantize_weights(w, d, torch.empty_like(c[1]), pow2=pow2)
    same(f64(d[..., :K]), f64(c[0][..., :K]), "without the transpose")


# ------------------------------------------------------------------ SwiGLU
def act_inputs(R, f, seed):
    rng = np.random.default_rng(seed)
    ab = rng.normal(size=(R, 2 * f)).astype(np.float32) * 2
    if R > 4 and f > 8:
        ab[0, :f] = 0
        ab[1, f:] = 0
        ab[2, :6] = [-100, -88, -60, 60, 100, 3e38]
        ab[3, :8] = [-1.28125, -1.2734375, -1e-30, 1e-38, -0.0, 1e30, -80, -81]
    dh = rng.normal(size=(R, f)).astype(np.float32)
    return dev(ab).bfloat16(), dev(dh).bfloat16()


@pytest.mark.parametrize("f", [1, 8, 64, 100, 128, 257, 768, 1032])
@pytest.mark.parametrize("lengths", [[1], [130, 0, 63], [0, 257]])
def test_swiglu_and_its_backward(lengths, f):
    off = offsets_of(lengths)
    R, G = off[-1], len(lengths)
    B = tde.moe_fp8_token_blocks(R, G)
    ab, dh = act_inputs(R, f, R + f)
    ws, o = ws_new(), odev(off)

    def out(w):
        return [codes_new((R, up(w, 16))), torch.empty((R, -(-w // 128)), device="cuda"),
                codes_new((w, 128 * B)), torch.empty((B, w), device="cuda")]

    with np.errstate(all="ignore"):
        h, d = ref.swiglu(f64(ab)), ref.swiglu_bwd(f64(dh), f64(ab))
    for pow2 in (False, True):
        c, n = out(f), out(f)
        tde.moe_fp8_swiglu(ab, *c, offsets=o, pow2=pow2, ws=ws)
        tde.moe_fp8_swiglu(ab, n[0], n[1], offsets=o, pow2=pow2, ws=ws)
        for got in (c, n):
            check_rows(got[0], got[1], h, pow2)
        check_tokens(c[2], c[3], h, off, pow2)
        g, m = out(2 * f), out(f)
        tde.moe_fp8_swiglu_bwd(dh, ab, *g, m[2], m[3], offsets=o, pow2=pow2, ws=ws)
        check_rows(g[0], g[1], d, pow2)
        check_tokens(g[2], g[3], d, off, pow2)
        check_tokens(m[2], m[3], h, off, pow2)
        g = out(2 * f)
        tde.moe_fp8_swiglu_bwd(dh, ab, g[0], g[1], offsets=o, pow2=pow2, ws=ws)
        check_rows(g[0], g[1], d, pow2)
    assert tde.moe_status(ws)[1] == 0


def test_swiglu_rounds_once_over_every_gate():
    """Every finite bf16 gate below 60 in magnitude, against up values of 8 significant bits:
    the stored h is the exact value rounded once (seen through pow2 codes of a block of one)."""
    bits = np.arange(65536, dtype=np.uint32) << 16
    a = bits.view(np.float32)
    a = a[np.isfinite(a) & (np.abs(a) < 60)]
    rng = np.random.default_rng(1)
    b = (1 + rng.integers(0, 128, a.size) / 128).astype(np.float32)
    n = a.size // 256 * 256
    ab = np.concatenate([a[:n].reshape(-1, 256), b[:n].reshape(-1, 256)], 1)
    abd, ws = dev(ab).bfloat16(), ws_new()
    dh = dev(rng.normal(size=(n // 256, 256)).astype(np.float32)).bfloat16()
    h, d = ref.swiglu(f64(abd)), ref.swiglu_bwd(f64(dh), f64(abd))
    R = n // 256
    c = [codes_new((R, 256)), torch.empty((R, 2), device="cuda")]
    tde.moe_fp8_swiglu(abd, *c, ws=ws)
    check_rows(*c, h, False)
    g = [codes_new((R, 512)), torch.empty((R, 4), device="cuda")]
    tde.moe_fp8_swiglu_bwd(dh, abd, *g, ws=ws)
    check_rows(*g, d, False)


# ------------------------------------------------------------------ products
def operand(shape, seed, blocks):
    """Codes as the quantisers leave them, and scales of any fp32 value."""
    rng = np.random.default_rng(seed)
    v = ref.e4m3(rng.normal(size=shape) * 120)
    s = np.exp(rng.normal(size=blocks)).astype(np.float32) / 100
    return v, s


def to_codes(v, ld):
    t = codes_new(v.shape[:-1] + (ld,))     # NaN past the row's end: never read
    t.view(torch.uint8)[..., :v.shape[-1]] = dev(v.astype(np.float32)).to(E4).view(torch.uint8)
    return t


def check_product(got, o, mag, blocks, fp32, name):
    eps = 2.0 ** -24 if fp32 else 2.0 ** -8
    err = np.abs(got - o)
    # half a step of the output on the largest value the sum may have, and one more step of
    # fp32 subnormals
    bound = (256 + blocks + 3) * 2.0 ** -24 * mag
    assert np.isfinite(got).all(), name
    assert (err <= bound + eps * (np.abs(o) + bound) + 1e-37).all(), (name, err.max())
    n = np.linalg.norm(o)
    if n and o.size >= 1000:
        rel = np.linalg.norm(err) / n
        assert rel <= (2e-6 if fp32 else 2.0 ** -8 / 3 ** 0.5 + 1e-6), (name, rel)


PRODUCTS = [  # segment lengths, N, K
    ([1], 1, 1), ([1], 128, 128), ([5], 256, 384), ([128], 256, 256), ([129], 300, 200),
    ([0, 3, 0, 130, 257], 520, 640), ([1, 1, 0, 1], 1000, 1000), ([64] * 5, 96, 1536),
    ([400, 1, 299], 257, 129), ([0, 0], 64, 64), ([7, 9, 0, 40, 2, 33, 1, 16], 768, 2048),
    ([17], 2048, 7168), ([260, 140], 128, 4096)]


# few rows: segments of several 16-row tiles, blocks shared by 2, 4 and 8 CTAs (in two rounds,
# too), more tiles than SMs
FEW = [
    ([1], 128, 1024), ([16], 130, 2048), ([3], 1000, 4100), ([0, 2, 0, 5, 0, 0], 384, 7168),
    ([40] + [0] * 7, 257, 1024), ([16, 1, 17, 0], 520, 2048), ([64], 250, 1024), ([33], 77, 7000),
    ([150, 0, 3, 0, 1], 130, 1030), ([200] + [0] * 30 + [1], 128, 1152), ([1] * 40, 1000, 300),
    ([30, 40, 0, 26], 4096, 520), ([2] * 256, 64, 130),
    ([13], 200, 12400), ([29, 1, 1, 1], 2294, 3100)]


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("lengths,N,K", PRODUCTS + FEW)
def test_product(lengths, N, K, fp32):
    off = offsets_of(lengths)
    R, G = off[-1], len(lengths)
    KB, NB = -(-K // 128), -(-N // 128)
    av, sa = operand((R, K), 1, (R, KB))
    bv, sb = operand((G, N, K), 2, (G, NB, KB))
    a, b = to_codes(av, up(K, 16)), to_codes(bv, up(K, 16) + 16)
    out = torch.full((R + 1, N), float("nan"), dtype=torch.float32 if fp32 else torch.bfloat16,
                     device="cuda")
    ws = ws_new()
    tde.moe_fp8_gemm(a, dev(sa), b, dev(sb), out[:R], K, offsets=odev(off), ws=ws)
    assert tde.moe_status(ws)[1] == 0
    A = av * ref.spread(sa.astype(np.float64), K, 1)
    o, mag = np.zeros((R, N)), np.zeros((R, N))
    for g in range(G):
        at = slice(off[g], off[g + 1])
        B = bv[g] * ref.spread(ref.spread(sb[g].astype(np.float64), N, 0), K, 1)
        o[at], mag[at] = A[at] @ B.T, np.abs(A[at]) @ np.abs(B.T)
    check_product(f64(out[:R]), o, mag, KB, fp32, "out")
    assert torch.isnan(out[R]).all()


def test_product_dense_strided_and_part_of_the_rows():
    """No offsets; an output inside a wider one, off 16 bytes; rows past the segments kept."""
    R, N, K = 150, 130, 256
    av, sa = operand((R, K), 3, (R, 2))
    bv, sb = operand((1, N, K), 4, (1, 2, 2))
    a, b, ws = to_codes(av, K), to_codes(bv, K), ws_new()
    A = av * ref.spread(sa.astype(np.float64), K, 1)
    B = bv[0] * ref.spread(ref.spread(sb[0].astype(np.float64), N, 0), K, 1)
    for col in (0, 1, 7):
        for dt in (torch.bfloat16, torch.float32):
            wide = torch.zeros((R, N + 9), dtype=dt, device="cuda")
            tde.moe_fp8_gemm(a, dev(sa), b, dev(sb), wide[:, col:col + N], K, ws=ws)
            check_product(f64(wide[:, col:col + N]), A @ B.T, np.abs(A) @ np.abs(B.T), 2,
                          dt == torch.float32, "strided")
            assert (wide[:, :col] == 0).all() and (wide[:, col + N:] == 0).all()
    out = torch.full((R, N), 5.0, device="cuda")
    tde.moe_fp8_gemm(a, dev(sa), b, dev(sb), out, K, offsets=odev([0, 77]), ws=ws)
    assert (out[77:] == 5).all()
    check_product(f64(out[:77]), (A @ B.T)[:77], (np.abs(A) @ np.abs(B.T))[:77], 2, True, "part")


@pytest.mark.parametrize("R,K", [(9, 4096), (50, 1024), (11, 12800)])
def test_few_rows_strided_bad_and_repeated(R, K):
    """An output inside a wider one; a row of NaN codes in the middle of a tile; the same bits from
    every call and from a captured one."""
    N, KB = 130, K // 128
    av, sa = operand((R, K), 7, (R, KB))
    bv, sb = operand((1, N, K), 8, (1, 2, KB))
    a, b, ws = to_codes(av, K), to_codes(bv, K), ws_new()
    a.view(torch.uint8)[4] = 0x7f
    A = av * ref.spread(sa.astype(np.float64), K, 1)
    B = bv[0] * ref.spread(ref.spread(sb[0].astype(np.float64), N, 0), K, 1)
    rows = [r for r in range(R) if r != 4]
    for dt in (torch.bfloat16, torch.float32):
        wide = torch.zeros((R, N + 9), dtype=dt, device="cuda")
        args = (a, dev(sa), b, dev(sb), wide[:, 3:3 + N], K)
        tde.moe_fp8_gemm(*args, ws=ws)
        first = wide.clone()
        assert torch.isnan(wide[4, 3:3 + N]).all()
        assert (wide[:, :3] == 0).all() and (wide[:, 3 + N:] == 0).all()
        check_product(f64(wide[:, 3:3 + N])[rows], (A @ B.T)[rows],
                      (np.abs(A) @ np.abs(B.T))[rows], KB, dt == torch.float32, "few")
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            tde.moe_fp8_gemm(*args, ws=ws)
        for _ in range(3):
            wide.zero_()
            graph.replay()
            assert same_bits(wide, first)
    assert tde.moe_status(ws)[1] == 0


def same_bits(x, y):
    return bool((x.view(torch.uint8) == y.view(torch.uint8)).all())


def test_product_keeps_a_bad_row_to_itself():
    """A NaN or an infinite scale in one row of A, or one row of B, reaches that row or column of
    the output alone; a segment's neighbours stay clean."""
    R, N, K = 200, 300, 384
    av, sa = operand((R, K), 5, (R, 3))
    bv, sb = operand((2, N, K), 6, (2, 3, 3))
    ws, off = ws_new(), odev([0, 100, 200])
    clean = torch.empty((R, N), device="cuda")
    tde.moe_fp8_gemm(to_codes(av, K), dev(sa), to_codes(bv, K), dev(sb), clean, K, offsets=off,
                     ws=ws)
    a, b = to_codes(av, K), to_codes(bv, K)
    a.view(torch.uint8)[99, 200] = 0x7f
    b.view(torch.uint8)[0, 17, 3] = 0x7f
    sa2 = sa.copy()
    sa2[150, 1] = np.inf
    out = torch.empty((R, N), device="cuda")
    tde.moe_fp8_gemm(a, dev(sa2), b, dev(sb), out, K, offsets=off, ws=ws)
    bad = torch.zeros((R, N), dtype=torch.bool, device="cuda")
    bad[99] = True
    bad[150] = True
    bad[:100, 17] = True
    assert torch.equal(out[~bad], clean[~bad])
    assert not torch.isfinite(out[99]).any() and not torch.isfinite(out[:100, 17]).any()
    assert not torch.isfinite(out[150]).any()


WGRADS = [([1], 1, 1), ([128], 128, 256), ([130, 0, 5], 136, 300), ([0, 0, 0], 64, 64),
          ([700], 256, 512), ([1, 0, 129, 300, 64], 1000, 129), ([40] * 8, 257, 768)]


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("lengths,M,N", WGRADS)
def test_weight_gradient(lengths, M, N, fp32):
    off = offsets_of(lengths)
    R, G = off[-1], len(lengths)
    x, y = normal((max(R, 1), M), 7)[:R], normal((max(R, 1), N), 8)[:R]
    ws, o = ws_new(), odev(off)
    B = tde.moe_fp8_token_blocks(R, G)
    ops = []
    for t, C in ((x, M), (y, N)):
        c = [codes_new((C, 128 * B)), torch.empty((B, C), device="cuda")]
        tde.moe_fp8_quantize(t, codes_t=c[0], scales_t=c[1], offsets=o, ws=ws)
        ops += c
    dw = torch.full((G, M, N), float("nan"), dtype=torch.float32 if fp32 else torch.bfloat16,
                    device="cuda")
    tde.moe_fp8_wgrad(*ops, dw, offsets=o, rows=R, ws=ws)
    assert tde.moe_status(ws)[1] == 0
    qa, sa = ref.quantise_tokens(f64(x), off)
    qb, sb = ref.quantise_tokens(f64(y), off)
    A, Bv = qa * np.repeat(sa, 128, 0).T, qb * np.repeat(sb, 128, 0).T
    first = 0
    for g, n in enumerate(lengths):
        nb = -(-n // 128)
        at = slice(first * 128, (first + nb) * 128)
        first += nb
        check_product(f64(dw[g]), A[:, at] @ Bv[:, at].T, np.abs(A[:, at]) @ np.abs(Bv[:, at]).T,
                      nb, fp32, g)


def test_repeatable_and_captured():
    """The same bits on every call, from a graph and on another stream."""
    R, N, K, G = 500, 768, 512, 6
    off = odev(offsets_of([100, 0, 250, 3, 47, 100]))
    x, w = normal((R, K), 1), normal((G, N, K), 2, 0.05)
    ws = ws_new()
    B = tde.moe_fp8_token_blocks(R, G)
    wq = [codes_new((G, N, K)), torch.empty((G, 6, 4), device="cuda")]
    tde.moe_fp8_quantize_weights(w, *wq)

    def step(stream=None):
        q = [codes_new((R, K)), torch.empty((R, 4), device="cuda"), codes_new((K, 128 * B)),
             torch.empty((B, K), device="cuda")]
        y = torch.zeros((R, N), dtype=torch.bfloat16, device="cuda")
        dw = torch.zeros((G, K, K), device="cuda")
        tde.moe_fp8_quantize(x, *q, offsets=off, ws=ws, stream=stream)
        tde.moe_fp8_gemm(q[0], q[1], *wq, y, K, offsets=off, ws=ws, stream=stream)
        tde.moe_fp8_wgrad(q[2], q[3], q[2], q[3], dw, offsets=off, rows=R, ws=ws, stream=stream)
        return y, dw

    first = step()
    for a, b in zip(first, step()):
        assert torch.equal(a, b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = step(s)
    s.synchronize()
    for a, b in zip(first, other):
        assert torch.equal(a, b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = step()
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(first, cap):
        assert torch.equal(a, b)


def test_swiglu_backward_against_differences():
    """[da | db] against central differences of silu(a) b in 64 bits: half a step of bf16 and of
    E4M3 (2^-8 and 2^-4, relative; below its normal numbers 2^-10 of the scale); the differences
    are off by h^2 / 6 of a third derivative (below 2)."""
    R, f, h = 40, 96, 1e-4
    ab, dh = normal((R, 2 * f), 31), normal((R, f), 32)
    c, ws = [codes_new((R, 2 * f)), torch.empty((R, 2), device="cuda")], ws_new()
    tde.moe_fp8_swiglu_bwd(dh, ab, *c, ws=ws)
    a, b, d = f64(ab)[:, :f], f64(ab)[:, f:], f64(dh)

    def fn(a, b):
        return a / (1 + np.exp(-a)) * b
    want = np.hstack([d * (fn(a + h, b) - fn(a - h, b)),
                      d * (fn(a, b + h) - fn(a, b - h))]) / (2 * h)
    s = ref.spread(f64(c[1]), 2 * f, 1)
    slack = np.hstack([np.abs(d * b), np.abs(d)]) * (h * h / 3) + 1e-11
    bound = (np.abs(want) + slack) * (2.0 ** -4 * (1 + 2.0 ** -8) + 2.0 ** -8 + 2.0 ** -20)
    assert (np.abs(f64(c[0]) * s - want) <= bound + slack + s * 2.0 ** -10).all()


def test_rows_past_32_bits():
    """More than 2^31 elements: rows, columns along the tokens, an output's strided rows."""
    R, C = 300_001, 7168
    ws, B = ws_new(), tde.moe_fp8_token_blocks(R, 1)
    x = torch.randn((R, C), device="cuda", dtype=torch.bfloat16)
    c = [codes_new((R, C)), torch.empty((R, 56), device="cuda"), codes_new((C, 128 * B)),
         torch.empty((B, C), device="cuda")]
    tde.moe_fp8_quantize(x, *c, ws=ws)
    at = slice(R - 130, R)
    check_rows(c[0][at], c[1][at], f64(x[at]), False)
    rows = [codes_new((R, C)), torch.empty((R, 56), device="cuda")]
    tde.moe_fp8_quantize(x, *rows, ws=ws)
    assert torch.equal(rows[0].view(torch.uint8)[at], c[0].view(torch.uint8)[at])
    assert torch.equal(rows[1], c[1])
    check_tokens(c[2][C - 3:], c[3][:, C - 3:], f64(x[:, C - 3:]), [0, R], False)
    del x, c, rows
    M, N, K, ld = 300, 130, 256, 1 << 23
    av, sa = operand((M, K), 41, (M, 2))
    bv, sb = operand((1, N, K), 42, (1, 2, 2))
    out = torch.zeros((M, ld), device="cuda", dtype=torch.bfloat16)
    for lo, n in ((0, M), (M - 9, 9)):
        part = out[lo:, ld - N:]
        part.zero_()
        tde.moe_fp8_gemm(to_codes(av[lo:], K), dev(sa[lo:]), to_codes(bv, K), dev(sb), part, K,
                         ws=ws)
        A = av[lo:] * ref.spread(sa[lo:].astype(np.float64), K, 1)
        Bv = bv[0] * ref.spread(ref.spread(sb[0].astype(np.float64), N, 0), K, 1)
        check_product(f64(part), A @ Bv.T, np.abs(A) @ np.abs(Bv.T), 2, False, n)
    assert tde.moe_status(ws)[1] == 0
    del out, part
    torch.cuda.empty_cache()


def test_weights_past_32_bits():
    """More than 2^31 elements of weights and of their gradients: the last expert's."""
    G, N, K = 160, 2048, 7168
    ws = ws_new()
    w = torch.zeros((G, N, K), device="cuda", dtype=torch.bfloat16)
    w[-1] = normal((N, K), 51, 0.05)
    q = [codes_new((G, N, K)), torch.empty((G, 16, 56), device="cuda"), codes_new((G, K, N)),
         torch.empty((G, 56, 16), device="cuda")]
    tde.moe_fp8_quantize_weights(w, *q)
    codes, scales = ref.quantise_weights(f64(w[-1]))
    same(f64(q[0][-1]), codes, "codes")
    same(f64(q[2][-1]), codes.T, "codes_t")
    same(f64(q[1][-1]), scales, "scales")
    del w
    Bv = codes[:64] * ref.spread(ref.spread(scales, N, 0), K, 1)[:64]
    for R in (3, 1400):
        av, sa = operand((R, K), R, (R, 56))
        out = torch.empty((R, N), device="cuda", dtype=torch.bfloat16)
        tde.moe_fp8_gemm(to_codes(av, K), dev(sa), *q[:2], out, K, offsets=odev([0] * G + [R]),
                         ws=ws)
        A = av * ref.spread(sa.astype(np.float64), K, 1)
        check_product(f64(out[:, :64]), A @ Bv.T, np.abs(A) @ np.abs(Bv.T), 56, False, R)
    del q
    R, off = 200, odev([0] * G + [200])
    x, y = normal((R, N), 52), normal((R, K), 53)
    B = tde.moe_fp8_token_blocks(R, G)
    ops = []
    for t, C in ((x, N), (y, K)):
        c = [codes_new((C, 128 * B)), torch.empty((B, C), device="cuda")]
        tde.moe_fp8_quantize(t, codes_t=c[0], scales_t=c[1], offsets=off, ws=ws)
        ops += c
    dw = torch.full((G, N, K), float("nan"), device="cuda", dtype=torch.bfloat16)
    tde.moe_fp8_wgrad(*ops, dw, offsets=off, rows=R, ws=ws)
    assert (dw[G - 2] == 0).all() and (dw[0] == 0).all()
    qa, sa = ref.quantise_tokens(f64(x)[:, -40:], [0, R])
    qb, sb = ref.quantise_tokens(f64(y), [0, R])
    A, Bv = qa * np.repeat(sa, 128, 0).T, qb * np.repeat(sb, 128, 0).T
    check_product(f64(dw[-1, -40:]), A @ Bv.T, np.abs(A) @ np.abs(Bv).T, 2, False, "dw")
    assert tde.moe_status(ws)[1] == 0
    del dw
    torch.cuda.empty_cache()
