"""Plain 64-bit references of the normalisation and the 8-bit checkpoints, written from their
definitions (include/moe.h); buffers with guards around them; bounds on rounding errors.

A value rounded to bf16 is off by at most 2^-8 of itself (half a step), one in fp32 by 2^-24.
"""

import numpy as np
import torch

import block_ref

BLOCK = 128
U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "fp32": U}
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
PATTERN = 0xa5
MARGIN = 4096


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def f32(a):
    return np.asarray(a, np.float64).astype(np.float32).astype(np.float64)


def typed(a, name):
    """The numbers of a type nearest to a (a's numbers are of 32 bits)."""
    return torch.from_numpy(np.asarray(a, np.float32)).to(DT[name]).double().numpy()


def quantise(x, fmt):
    """Codes (as numbers) and scales of rows x: a loop over the blocks."""
    if fmt == "e4m3":
        return block_ref.quantise_rows(x)
    R, C = x.shape
    q = np.zeros((R, C))
    s = np.zeros((R, -(-C // BLOCK)))
    for b in range(s.shape[1]):
        v = x[:, b * BLOCK:(b + 1) * BLOCK]
        amax = np.maximum(np.abs(v).max(1), 2.0 ** -110)
        s[:, b] = f32(amax / 127)
        q[:, b * BLOCK:(b + 1) * BLOCK] = np.rint(v * f32(127 / amax)[:, None])   # exact products
    return q, s


def restore(q, s):
    """code * scale, rounded to 32 bits."""
    return f32(q * np.repeat(s, BLOCK, 1)[:, :q.shape[1]])


def stats(v, kind, eps):
    m = v.mean(1) if kind == "layer" else np.zeros(len(v))
    return m, 1 / np.sqrt(((v - m[:, None]) ** 2).mean(1) + eps)


def norm(v, gamma, beta, kind, eps):
    m, r = stats(v, kind, eps)
    return (v - m[:, None]) * r[:, None] * gamma + beta


def norm_bwd(dy, v, m, r, gamma, add, kind):
    xh = (v - m[:, None]) * r[:, None]
    g = dy * gamma
    c1 = g.mean(1, keepdims=True) if kind == "layer" else 0.0
    c2 = (g * xh).mean(1, keepdims=True)
    dx = r[:, None] * (g - c1 - xh * c2) + add
    return dx, (dy * xh).sum(0), dy.sum(0)


def sigmoid(a):
    e = np.exp(-np.abs(a))
    return np.where(a >= 0, 1 / (1 + e), e / (1 + e))


def swiglu(a, b):
    return a * sigmoid(a) * b


def swiglu_bwd(dh, a, b):
    s = sigmoid(a)
    return dh * b * s * (1 + a * sigmoid(-a)), dh * a * s


def sigmoid_error(a):
    """The relative error of sigma through CUDA's fast exponential (2 + |1.173 a| units in the last
    place of 2^-23) and division (2), the addition and what multiplies it."""
    return (8 + 1.2 * np.abs(a)) * 2.0 ** -23


def check(name, got, want, tol):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    off = np.abs(got - want)
    bad = ~(off <= tol)
    assert not bad.any(), (f"{name}: {bad.sum()} of {bad.size} off, worst {np.nanmax(off):.3e}, first at "
                           f"{np.argwhere(bad)[0]}: {got[tuple(np.argwhere(bad)[0])]} for "
                           f"{want[tuple(np.argwhere(bad)[0])]}")


def same(name, got, want):
    check(name, got, want, 0.0)


class Guarded:
    """A tensor [rows, cols] inside a buffer of PATTERN bytes, `ld` elements between its rows and
    its first element `first` elements after a 256-byte border."""

    def __init__(self, rows, cols, dtype, ld=None, first=0):
        size = dtype.itemsize
        self.rows, self.cols, self.size = rows, cols, size
        self.ld = cols if ld is None else ld
        self.front = MARGIN + first * size
        n = self.front + max(rows, 1) * self.ld * size
        self.buf = torch.full((n + MARGIN,), PATTERN, dtype=torch.uint8, device="cuda")
        room = self.buf[self.front:n].view(dtype)
        self.t = room.as_strided((rows, cols), (self.ld, 1))

    def put(self, values):
        self.t.copy_(torch.as_tensor(np.asarray(values, np.float32)))
        return self.t

    def check_guards(self, name, live=None):
        """Nothing changed outside the live rows' columns."""
        b = self.buf.cpu().numpy()
        keep = np.ones(b.size, bool)
        for r in range(self.rows if live is None else live):
            at = self.front + r * self.ld * self.size
            keep[at:at + self.cols * self.size] = False
        assert (b[keep] == PATTERN).all(), f"{name}: written outside its rows"


def checkpoint(rows, C, fmt):
    """Guarded codes and scales."""
    c = Guarded(rows, C, torch.int8, ld=-(-C // 16) * 16)
    s = Guarded(rows, -(-C // BLOCK), torch.float32)
    return c, s


def codes_of(c, fmt):
    """The tensor that a call takes: [rows, ld]."""
    return c.buf[c.front:c.front + c.rows * c.ld].view(CODES[fmt]).view(c.rows, c.ld)


def code_values(c, fmt):
    """The codes as numbers, [rows, C]."""
    return f64(codes_of(c, fmt))[:, :c.cols]


def device_checkpoint(x, fmt):
    """codes, scales (tensors) and the restored values of rows x, made by the reference."""
    q, s = quantise(x, fmt)
    R, C = x.shape
    c, g = checkpoint(R, C, fmt)
    codes = codes_of(c, fmt)
    codes.view(torch.int8)[:, :C] = (torch.from_numpy(q.astype(np.int8)) if fmt == "int8" else
                                     torch.from_numpy(q.astype(np.float32)).to(CODES[fmt])
                                     .view(torch.int8)).cuda()
    g.put(s)
    return codes, g.t, restore(q, s)


def unrounded(codes, scales, C):
    """code * scale of a checkpoint, the products not yet rounded to 32 bits."""
    return f64(codes)[:, :C] * np.repeat(f64(scales), BLOCK, 1)[:, :C]


def new_ws(n=256):
    import token_dispatch_expert_gb300 as tde
    ws = torch.full((n,), PATTERN, dtype=torch.uint8, device="cuda")
    tde.moe_ws_init(ws)
    return ws
