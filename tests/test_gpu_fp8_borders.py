"""Every output of the 8-bit operators as a view inside a larger buffer of a known pattern: the live
part is exactly what the 64-bit references give, and not a byte outside it changes -- in front of the
view, behind it, in the rows past the segments' end and in the token blocks past the last segment's.
(Bytes between a row's last code and its distance may become zero, as include/moe.h says.)

Codes and scales are compared exactly, products within the bound of tests/test_gpu_fp8.py.
"""

import numpy as np
import pytest
import torch

import block_ref as ref
import token_dispatch_expert_gb300 as tde
from gpu_util import dev
from test_gpu_fp8 import (act_inputs, check_product, f64, normal, odev, offsets_of, operand, same,
                          to_codes, up, ws_new)

pytestmark = pytest.mark.gpu
E4 = torch.float8_e4m3fn
PATTERN = 0xa5
MARGIN = 4096   # bytes before and behind: more than a stray block's scales or codes lie away


class Guarded:
    """A tensor inside a buffer of PATTERN bytes."""

    def __init__(self, shape, dtype):
        n = int(np.prod(shape)) * dtype.itemsize
        self.buf = torch.full((MARGIN + n + MARGIN,), PATTERN, dtype=torch.uint8, device="cuda")
        self.t = self.buf[MARGIN:MARGIN + n].view(dtype).view(shape)

    def bytes(self):
        """The view's bytes, [rows][bytes of a row]; what lies around it is checked here."""
        b = self.buf.cpu().numpy()
        assert (b[:MARGIN] == PATTERN).all(), "written in front of the output"
        assert (b[-MARGIN:] == PATTERN).all(), "written behind the output"
        rows = self.t.shape[0]
        return b[MARGIN:-MARGIN].reshape(rows, -1) if rows else np.zeros((0, 0), np.uint8)


def untouched(b, name):
    assert (b == PATTERN).all(), f"{name}: written past the live part"


class Outputs:
    """Both orientations of `cols` columns of `rows` rows, and their check."""

    def __init__(self, rows, G, cols, along_rows, along_tokens):
        self.cols, self.kb, B = cols, -(-cols // 128), tde.moe_fp8_token_blocks(rows, G)
        f32 = torch.float32
        self.row = self.tok = None
        if along_rows:
            self.row = Guarded((rows, up(cols, 16)), E4), Guarded((rows, self.kb), f32)
        if along_tokens:
            self.tok = Guarded((cols, 128 * B), E4), Guarded((B, cols), f32)

    def args(self):
        return [x.t if x else None for p in (self.row, self.tok) for x in (p or (None, None))]

    def check(self, v, off, pow2, name):
        live = off[-1]
        if self.row:
            codes, scales = self.row
            q, s = ref.quantise_rows(v[:live], pow2)
            same(f64(codes.t[:live, :self.cols]), q, name + " codes")
            same(f64(scales.t[:live]), s, name + " scales")
            b = codes.bytes()
            untouched(b[live:], name + " codes")
            pad = b[:live, self.cols:]
            assert ((pad == PATTERN) | (pad == 0)).all(), name + " padding"
            untouched(scales.bytes()[live:], name + " scales")
        if self.tok:
            codes, scales = self.tok
            q, s = ref.quantise_tokens(v, off, pow2)
            nb = s.shape[0]
            same(f64(codes.t[:, :128 * nb]), q[:, :128 * nb], name + " codes_t")
            same(f64(scales.t[:nb]), s, name + " scales_t")
            untouched(codes.bytes()[:, 128 * nb:], name + " codes_t")
            untouched(scales.bytes()[nb:], name + " scales_t")


FORMS = [(True, False), (False, True), (True, True)]
LIVE = [0, 1, 2, 3, 4, 5, 6, 7, 21, 42, 51, 93]   # every remainder by 4, several chunks a warp


@pytest.mark.parametrize("dead", [0, 3])
@pytest.mark.parametrize("f", [8, 16, 24, 32, 64, 72, 80, 128, 264, 640, 768, 1024, 1408, 1536, 2048])
def test_swiglu_rows(f, dead):
    ws = ws_new()
    for live in LIVE:
        rows = live + dead
        if rows == 0:
            continue
        ab, _ = act_inputs(rows, f, rows + f)
        off = offsets_of([live])
        with np.errstate(all="ignore"):
            h = ref.swiglu(f64(ab))
        for offsets in [odev(off)] + ([None] if dead == 0 else []):
            o = Outputs(rows, 1, f, True, False)
            tde.moe_fp8_swiglu(ab, *o.args(), offsets=offsets, ws=ws)
            o.check(h, off, False, f"{live} of {rows} x {f}")
    assert tde.moe_status(ws)[1] == 0


@pytest.mark.parametrize("f", [776, 896, 1000, 1016, 2040])
def test_swiglu_rows_of_four_chunks(f):
    """Widths whose chunks of 256 columns come in fours, the last of them short."""
    test_swiglu_rows(f, 3)


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("lengths,dead", [([1], 0), ([2], 2), ([7, 0, 128], 5), ([129, 3, 0, 61], 1),
                                          ([0, 0], 3)])
@pytest.mark.parametrize("f", [1, 8, 64, 72, 80, 100, 128, 129, 640, 1408])
def test_quantisers(f, lengths, dead, pow2):
    off, G = offsets_of(lengths), len(lengths)
    rows = off[-1] + dead
    ab, dh = act_inputs(rows, f, rows + f)
    x, ws, o = normal((rows, f), f), ws_new(), odev(off)
    with np.errstate(all="ignore"):
        h, d = ref.swiglu(f64(ab)), ref.swiglu_bwd(f64(dh), f64(ab))
    for form in FORMS:
        r = Outputs(rows, G, f, *form)
        tde.moe_fp8_quantize(x, *r.args(), offsets=o, pow2=pow2, ws=ws)
        r.check(f64(x), off, pow2, "rows")
        s = Outputs(rows, G, f, *form)
        tde.moe_fp8_swiglu(ab, *s.args(), offsets=o, pow2=pow2, ws=ws)
        s.check(h, off, pow2, "SwiGLU")
        if not form[0]:
            continue
        for with_h in (False, True):
            if with_h and not form[1]:
                continue
            b = Outputs(rows, G, 2 * f, *form)
            hh = Outputs(rows, G, f, False, True) if with_h else None
            tde.moe_fp8_swiglu_bwd(dh, ab, *b.args(), *(hh.args()[2:] if with_h else ()), offsets=o,
                                   pow2=pow2, ws=ws)
            b.check(d, off, pow2, "SwiGLU backward")
            if with_h:
                hh.check(h, off, pow2, "h")
    assert tde.moe_status(ws)[1] == 0


@pytest.mark.parametrize("form", FORMS)
def test_gathered_rows(form):
    """Source rows in any order, -1 past the segments."""
    T, C, off = 40, 264, offsets_of([90, 0, 61])
    x, ws = normal((T, C), 4), ws_new()
    src = np.random.default_rng(0).integers(0, T, 160).astype(np.int32)
    src[151:] = -1
    r = Outputs(160, 3, C, *form)
    tde.moe_fp8_quantize(x, *r.args(), offsets=odev(off), src_tok=dev(src), ws=ws)
    r.check(f64(x)[src], off, False, "gathered")
    assert tde.moe_status(ws)[1] == 0


@pytest.mark.parametrize("C", [264, 262, 263, 8])
def test_a_bad_source_row_is_skipped_along_the_row_and_read_as_row_0_along_the_tokens(C):
    """The same codes and scales from each form, whichever outputs are asked for together."""
    T, n, bad = 40, 151, [0, 31, 32, 77, 90, 150]
    off = offsets_of([90, 0, 61])
    x, ws = normal((T, C), 4), ws_new()
    src = np.random.default_rng(0).integers(1, T, n).astype(np.int32)
    src[bad] = [T, -1, 2 ** 30, -2 ** 31, T, -5]
    good = np.setdiff1d(np.arange(n), bad)
    v = f64(x)[np.where((src < 0) | (src >= T), 0, src)]
    for form in FORMS:
        r = Outputs(n, 3, C, *form)
        tde.moe_fp8_quantize(x, *r.args(), offsets=odev(off), src_tok=dev(src), ws=ws)
        assert tde.moe_status(ws)[1] == tde.DEVERR["BAD_INDEX"]
        if r.row:
            q, s = ref.quantise_rows(v)
            same(f64(r.row[0].t[good, :C]), q[good], "codes")
            same(f64(r.row[1].t[good]), s[good], "scales")
            untouched(r.row[0].bytes()[bad], "codes of a bad row")
            untouched(r.row[1].bytes()[bad], "scales of a bad row")
        if r.tok:
            r.row = None
            r.check(v, off, False, "tokens")


@pytest.mark.parametrize("G,N,K", [(1, 1, 1), (2, 130, 100), (3, 17, 257), (1, 300, 128)])
def test_weights(G, N, K):
    w = normal((G, N, K), N + K, 0.02)
    f32, nb, kb = torch.float32, -(-N // 128), -(-K // 128)
    c = [Guarded((G, N, up(K, 16)), E4), Guarded((G, nb, kb), f32), Guarded((G, K, up(N, 16)), E4),
         Guarded((G, kb, nb), f32)]
    for n in (4, 2):
        tde.moe_fp8_quantize_weights(w, *[x.t for x in c[:n]])
        for g in range(G):
            q, s = ref.quantise_weights(f64(w[g]))
            same(f64(c[0].t[g, :, :K]), q, "codes")
            same(f64(c[1].t[g]), s, "scales")
            same(f64(c[2].t[g, :, :N]), q.T, "codes_t")
            same(f64(c[3].t[g]), s.T, "scales_t")
        for x in c:
            x.bytes()


def product_inside(lengths, dead, N, K, fp32, ld, col=0):
    off, G = offsets_of(lengths), len(lengths)
    live, rows = off[-1], off[-1] + dead
    KB, NB, dt = -(-K // 128), -(-N // 128), torch.float32 if fp32 else torch.bfloat16
    av, sa = operand((rows, K), 1, (rows, KB))
    bv, sb = operand((G, N, K), 2, (G, NB, KB))
    ws = ws_new()
    a, b = to_codes(av, up(K, 16)), to_codes(bv, up(K, 16))
    A = av * ref.spread(sa.astype(np.float64), K, 1)
    out = Guarded((rows, ld), dt)
    tde.moe_fp8_gemm(a, dev(sa), b, dev(sb), out.t[:, col:col + N], K, offsets=odev(off), ws=ws)
    got = f64(out.t[:live, col:col + N])
    for g in range(G):
        r = slice(off[g], off[g + 1])
        B = bv[g] * ref.spread(ref.spread(sb[g].astype(np.float64), N, 0), K, 1)
        check_product(got[r], A[r] @ B.T, np.abs(A[r]) @ np.abs(B).T, KB, fp32, f"ld {ld}")
    raw = out.bytes()
    untouched(raw[live:], "out")
    untouched(raw[:, :col * dt.itemsize], "out")
    untouched(raw[:, (col + N) * dt.itemsize:], "out")
    assert tde.moe_status(ws)[1] == 0


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("lengths,dead,N,K", [
    ([3], 2, 130, 200), ([5, 0, 9], 1, 64, 300), ([70, 0, 131], 6, 257, 136),   # few rows; tiles
    ([1600], 40, 264, 128)])                                                    # pairs
def test_product(lengths, dead, N, K, fp32):
    for ld in (N, N + 1):
        product_inside(lengths, dead, N, K, fp32, ld)


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("N", [1, 63, 65, 130, 250, 257, 321])
@pytest.mark.parametrize("lengths", [[70, 0, 131], [1600], [9]])
def test_product_inside_rows_on_16_bytes(lengths, N, fp32):
    """Columns off 16 bytes of an output whose rows lie on them: the next columns stay as they are."""
    for ld, col in ((up(N, 8), 0), (up(N, 8) + 24, 8)):
        product_inside(lengths, 3, N, 200, fp32, ld, col)


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("M,N", [(1, 1), (100, 130), (129, 257), (300, 64)])
def test_weight_gradient(M, N, fp32):
    lengths, rows = [70, 0, 131], 210
    off, G = offsets_of(lengths), 3
    B = tde.moe_fp8_token_blocks(rows, G)
    x, y, ws = normal((rows, M), 1), normal((rows, N), 2), ws_new()
    q = []
    for v in (x, y):
        o = Outputs(rows, G, v.shape[1], False, True)
        tde.moe_fp8_quantize(v, *o.args(), offsets=odev(off), ws=ws)
        q += o.args()[2:]
    dw = Guarded((G, M, N), torch.float32 if fp32 else torch.bfloat16)
    tde.moe_fp8_wgrad(*q, dw.t, offsets=odev(off), rows=rows, ws=ws)
    xs = []
    for v in (x, y):
        c, s = ref.quantise_tokens(f64(v), off, False)
        xs.append(c * np.repeat(s.T, 128, axis=1))
    first = 0
    for g in range(G):
        nb = -(-lengths[g] // 128)
        a, b = (v[:, 128 * first:128 * (first + nb)] for v in xs)
        check_product(f64(dw.t)[g], a @ b.T, np.abs(a) @ np.abs(b).T, nb, fp32, f"segment {g}")
        first += nb
    dw.bytes()
    assert tde.moe_status(ws)[1] == 0
