"""The cases that the normalisation and the 8-bit checkpoints are measured on, with their plain forms.

What a block that trains a mixture of experts does around its products, as a program calls it:

  norm          y = xhat * gamma + beta of each row, xhat = (v - mean) * rstd, v = x or the sum of
                the residual stream and a branch, which is written too; layer norm, or the root mean
                square alone; v also as an 8-bit checkpoint for the backward pass
  norm_bwd      its gradient: dv (plus the stream's own gradient), dgamma and dbeta, from v or from
                v's checkpoint
  save          rows -> 8-bit codes with one fp32 scale for each block of 128 along the row
  restore       back from the checkpoint: the rows themselves; the pre-activation [a | b] with
                h = silu(a) * b; or the normalised rows
  swiglu_bwd    the SwiGLU's gradient [da | db], and h, from dh and the checkpoint of [a | b]
  combine_bwd   the gradient of the experts' weighted sum, from dy and the checkpoint of the
                experts' outputs: the rows' gradients and the weights'

`own` selects between the plain forms below and the framework's operators.
"""

import math
import random

import numpy as np
import torch

own = False

BLOCK = 128
TOP = {"e4m3": 448.0, "int8": 127.0}     # the largest code of each format
AMAX_FLOOR = 2.0 ** -110                 # a block's largest magnitude is held above this
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------ the cases
def listed():
    return [
        # one token on its way through a served model: pure latency
        dict(name="norm_one_token", kind="norm", T=1, C=7168, norm="layer", x="bf16", y="bf16",
             p="bf16", add=False, ckpt="", offset=0.5),
        # a training batch: the branch is added to the stream, the sum normalised for the experts
        # and kept in 8 bits
        dict(name="norm_add_batch", kind="norm", T=16384, C=4096, norm="layer", x="bf16", y="bf16",
             p="fp32", add=True, ckpt="int8", offset=0.5),
        # the gradient of the same, from the stream kept as it is
        dict(name="norm_bwd_batch", kind="norm_bwd", T=16384, C=4096, norm="layer", x="bf16",
             y="bf16", p="fp32", add=True, ckpt="", offset=0.5),
        # a 32-bit stream of odd width and length, kept in 8 bits
        dict(name="norm_bwd_odd", kind="norm_bwd", T=8191, C=1413, norm="layer", x="fp32",
             y="bf16", p="fp32", add=True, ckpt="e4m3", offset=0.0),
        # the first product's output [a | b] of a fine-grained layer, put away after the forward
        dict(name="save_pre_activation", kind="save", R=65536, C=1536, x="bf16", ckpt="int8",
             live=1.0),
        # few rows of odd width, some of the buffer's rows without a token
        dict(name="save_odd", kind="save", R=999, C=1001, x="fp32", ckpt="e4m3", live=0.8),
        # [a | b] and h back for the gradient's products; capacity left some rows empty
        dict(name="restore_swiglu", kind="restore", what="swiglu", R=49152, C=2816, x="bf16",
             y="bf16", p="fp32", ckpt="int8", live=0.9, norm="layer", offset=0.0),
        # the experts' input again, from the stream's checkpoint
        dict(name="restore_norm", kind="restore", what="norm", R=4096, C=7168, x="bf16", y="bf16",
             p="bf16", ckpt="int8", live=1.0, norm="rms", offset=0.0),
        # the SwiGLU's gradient over all rows of a fine-grained layer
        dict(name="swiglu_bwd_fine", kind="swiglu_bwd", R=65536, f=768, ckpt="int8", live=1.0),
        # odd width and length, E4M3 codes, rows behind the last segment
        dict(name="swiglu_bwd_odd", kind="swiglu_bwd", R=16383, f=1409, ckpt="e4m3", live=0.95),
        # the combine's gradient of a wide layer with eight experts to a token
        dict(name="combine_bwd_batch", kind="combine_bwd", T=4096, k=8, E=256, C=7168,
             ckpt="int8", dropped=0.0),
        # a short batch with dropped slots
        dict(name="combine_bwd_short", kind="combine_bwd", T=61, k=6, E=64, C=2048, ckpt="e4m3",
             dropped=0.1),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi, step):
    """Mostly widths of whole vectors, some odd."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.35 else max(step, n // step * step)


def draw(rng):
    kind = rng.choice(["norm", "norm", "norm_bwd", "norm_bwd", "save", "restore", "swiglu_bwd",
                       "combine_bwd"])
    fmt = rng.choice(["int8", "int8", "e4m3"])
    if kind in ("norm", "norm_bwd"):
        x = rng.choice(["bf16", "bf16", "fp32"])
        C = _width(rng, 64, 16384, 64)
        return dict(kind=kind, T=_log(rng, 1, min(32768, int(6e7 / C))), C=C,
                    norm=rng.choice(["layer", "layer", "rms"]), x=x,
                    y=x if rng.random() < 0.5 else "bf16", p=rng.choice(["bf16", "fp32"]),
                    add=rng.random() < 0.5, ckpt=fmt if rng.random() < 0.5 else "",
                    offset=rng.choice([0.0, 0.5, 8.0]))
    live = rng.choice([1.0, 1.0, 0.9, 0.5])
    if kind == "save":
        C = _width(rng, 64, 16384, 16)
        return dict(kind=kind, R=_log(rng, 1, min(65536, int(9e7 / C))), C=C,
                    x=rng.choice(["bf16", "bf16", "fp32"]), ckpt=fmt, live=live)
    if kind == "restore":
        what = rng.choice(["rows", "swiglu", "norm"])
        C = _width(rng, 64, 8192, 16)
        C += what == "swiglu" and C % 2
        return dict(kind=kind, what=what, R=_log(rng, 1, min(65536, int(9e7 / C))), C=C,
                    x=rng.choice(["bf16", "fp32"]) if what == "rows" else "bf16",
                    y=rng.choice(["bf16", "bf16", "fp32"]), p=rng.choice(["bf16", "fp32"]),
                    ckpt=fmt, live=1.0 if what == "norm" else live,
                    norm=rng.choice(["layer", "rms"]), offset=rng.choice([0.0, 0.5]))
    if kind == "swiglu_bwd":
        f = _width(rng, 32, 4096, 16)
        return dict(kind=kind, R=_log(rng, 1, min(65536, int(4e7 / f))), f=f, ckpt=fmt, live=live)
    k = rng.randint(1, 8)
    C = 64 * _log(rng, 1, 112)
    return dict(kind=kind, T=_log(rng, 1, min(8192, int(1.5e8 / (C * k)))), k=k,
                E=rng.choice([8, 16, 64, 256]), C=C, ckpt=fmt,
                dropped=rng.choice([0.0, 0.0, 0.1]))


def _size(name):
    return 4 if name == "fp32" else 2


def _live(c):
    return int(c["R"] * c["live"])


def work(case):
    """Each input read once, each output written once; a multiply-add counts two."""
    c = case
    kind = c["kind"]
    eight = 1.0 + 4.0 / BLOCK                       # a code and its share of a scale
    if kind in ("norm", "norm_bwd"):
        n, x, y, p = c["T"] * c["C"], _size(c["x"]), _size(c["y"]), _size(c["p"])
        stats = (8 if c["norm"] == "layer" else 4) * c["T"]
        vectors = (2 if c["norm"] == "layer" else 1) * c["C"]
        if kind == "norm":
            a = x * (3 if c["add"] else 1) + y + (eight if c["ckpt"] else 0.0)
            return {"bytes": n * a + stats + p * vectors, "flops": (8 + 3 * bool(c["ckpt"])) * n}
        a = y + (eight if c["ckpt"] else x) + x * (2 if c["add"] else 1)
        return {"bytes": n * a + stats + p * c["C"] + 4 * vectors, "flops": 14 * n}
    if kind == "save":
        n = _live(c) * c["C"]
        return {"bytes": n * (_size(c["x"]) + eight), "flops": 3 * n}
    if kind == "restore":
        n = _live(c) * c["C"]
        if c["what"] == "rows":
            return {"bytes": n * (eight + _size(c["x"])), "flops": n}
        if c["what"] == "swiglu":
            return {"bytes": n * (eight + 2 + 1), "flops": 4 * n}
        return {"bytes": n * (eight + _size(c["y"])) + 8 * c["R"] + 2 * _size(c["p"]) * c["C"],
                "flops": 5 * n}
    if kind == "swiglu_bwd":
        n = _live(c) * c["f"]
        return {"bytes": n * (2 + 2 * eight + 4 + 2), "flops": 16 * n}
    n = c["T"] * c["C"]
    return {"bytes": 2 * n + n * c["k"] * (eight + 2) + 12 * c["T"] * c["k"],
            "flops": 4 * n * c["k"]}


# ------------------------------------------------------------------------------ the inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(shape, seed, scale=1.0, offset=0.0, dtype=torch.bfloat16):
    x = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(generator=_gen(seed))
    return (x * scale + offset).to(dtype)


def _stream(R, C, seed, offset, dtype):
    """Rows of a residual stream: unit scale around the offset, a few channels ten times larger."""
    x = torch.empty((R, C), dtype=torch.float32, device="cuda").normal_(generator=_gen(seed))
    wide = torch.rand(C, generator=_gen(seed + 1), device="cuda") < 0.01
    return (x * (1.0 + 9.0 * wide) + offset).to(dtype)


def _up(n, m):
    return -(-n // m) * m


def _codes(R, C, fmt):
    c = torch.zeros((R, _up(C, 16)), dtype=torch.int8, device="cuda")
    return c if fmt == "int8" else c.view(torch.float8_e4m3fn)


def _checkpoint(x, fmt, n=None):
    """x's first n rows in 8 bits; the buffers' other rows stay zero."""
    R, C = x.shape
    codes = _codes(R, C, fmt)
    scales = torch.zeros((R, -(-C // BLOCK)), dtype=torch.float32, device="cuda")
    _plain_save(x, fmt, codes, scales, R if n is None else n)
    return codes, scales


def _offsets(c):
    """The expert segments' offsets; only the last one, the number of live rows, matters here."""
    n = _live(c)
    return torch.tensor([0, n // 3, n // 3, n], dtype=torch.int32, device="cuda")


def _parameters(c, C, seed):
    dt = TYPES[c["p"]]
    gamma = _normal((C,), seed + 20, 0.3, 1.0, dt)
    return gamma, _normal((C,), seed + 21, 0.2, 0.0, dt) if c["norm"] == "layer" else None


def _zeros(shape, dt):
    return torch.zeros(shape, dtype=dt, device="cuda")


def prepare(case, seed):
    c = dict(case)
    s = {"case": c}
    kind = c["kind"]
    f32, bf = torch.float32, torch.bfloat16
    if kind in ("norm", "norm_bwd"):
        T, C, dt = c["T"], c["C"], TYPES[c["x"]]
        s["x"] = _stream(T, C, seed, c["offset"], dt)
        s["gamma"], s["beta"] = _parameters(c, C, seed)
        if kind == "norm":
            s["residual"] = _normal((T, C), seed + 2, 0.5, 0.0, dt) if c["add"] else None
            s["out"] = {"y": _zeros((T, C), TYPES[c["y"]]), "rstd": _zeros((T,), f32)}
            if c["norm"] == "layer":
                s["out"]["mean"] = _zeros((T,), f32)
            if c["add"]:
                s["out"]["total"] = _zeros((T, C), dt)
            if c["ckpt"]:
                s["out"]["codes"] = _codes(T, C, c["ckpt"])
                s["out"]["scales"] = _zeros((T, -(-C // BLOCK)), f32)
            return s
        s["mean"], s["rstd"] = _plain_stats(s["x"].float(), c["norm"])
        if c["ckpt"]:
            s["x"], s["scales"] = _checkpoint(s["x"], c["ckpt"])
        s["dy"] = _normal((T, C), seed + 3, 0.1, 0.0, TYPES[c["y"]])
        s["add"] = _normal((T, C), seed + 4, 0.1, 0.0, dt) if c["add"] else None
        s["out"] = {"dx": _zeros((T, C), dt), "dgamma": _zeros((C,), f32)}
        if c["norm"] == "layer":
            s["out"]["dbeta"] = _zeros((C,), f32)
        return s
    if kind == "save":
        s["x"] = _stream(c["R"], c["C"], seed, 0.0, TYPES[c["x"]])
        s["offsets"] = _offsets(c)
        s["out"] = {"codes": _codes(c["R"], c["C"], c["ckpt"]),
                    "scales": _zeros((c["R"], -(-c["C"] // BLOCK)), f32)}
        return s
    if kind == "restore":
        R, C, what = c["R"], c["C"], c["what"]
        if what == "norm":
            x = _stream(R, C, seed, c["offset"], bf)
            s["mean"], s["rstd"] = _plain_stats(x.float(), c["norm"])
            s["gamma"], s["beta"] = _parameters(c, C, seed)
            s["out"] = {"y": _zeros((R, C), TYPES[c["y"]])}
        else:
            x = _stream(R, C, seed, 0.0, TYPES[c["x"]])
            s["out"] = ({"x": _zeros((R, C), TYPES[c["x"]])} if what == "rows" else
                        {"ab": _zeros((R, C), bf), "h": _zeros((R, C // 2), bf)})
        s["codes"], s["scales"] = _checkpoint(x, c["ckpt"], _live(c))
        s["offsets"] = _offsets(c)
        return s
    if kind == "swiglu_bwd":
        R, f = c["R"], c["f"]
        s["codes"], s["scales"] = _checkpoint(_normal((R, 2 * f), seed, 1.3), c["ckpt"], _live(c))
        s["dh"] = _normal((R, f), seed + 1, 0.1)
        s["offsets"] = _offsets(c)
        s["out"] = {"dab": _zeros((R, 2 * f), bf), "h": _zeros((R, f), bf)}
        return s
    T, k, E, C = c["T"], c["k"], c["E"], c["C"]
    choice = torch.rand((T, E), generator=_gen(seed + 5), device="cuda").topk(k, -1).indices
    drop = torch.rand((T, k), generator=_gen(seed + 6), device="cuda") < c["dropped"]
    by = torch.where(drop, E, choice).reshape(-1)
    order = by.sort(stable=True).indices
    rank = torch.empty_like(order)
    rank[order] = torch.arange(T * k, device="cuda")
    s["dest_row"] = torch.where(drop, -1, rank.view(T, k)).to(torch.int32)
    s["topk_w"] = torch.softmax(_normal((T, k), seed + 7, dtype=f32), -1)
    s["codes"], s["scales"] = _checkpoint(_normal((T * k, C), seed + 8, 0.6), c["ckpt"])
    s["dy"] = _normal((T, C), seed + 9, 0.1)
    s["out"] = {"dyp": _zeros((T * k, C), bf), "dw": _zeros((T, k), f32)}
    return s


# ------------------------------------------------------------------------- the plain forms
EPS = 1e-5


def _plain_save(x, fmt, codes, scales, n):
    """One scale for each 128 elements of a row; the last block of a row may be short."""
    C = x.shape[1]
    v = torch.nn.functional.pad(x[:n].float(), (0, _up(C, BLOCK) - C)).view(n, -1, BLOCK)
    amax = v.abs().amax(-1).clamp(min=AMAX_FLOOR)
    top = torch.full_like(amax, TOP[fmt])
    inv = (top / amax)[..., None]       # (a quotient of two tensors: correctly rounded)
    if fmt == "int8":
        # 64 bits: the product is rounded once, to a whole number
        q = (v.double() * inv.double()).round().to(torch.int8)
    else:
        q = (v * inv).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.int8)
    codes.view(torch.int8)[:n, :C] = q.view(n, -1)[:, :C]
    scales[:n] = amax / top


def _plain_load(codes, scales, n, C):
    """The values that the codes stand for, in 32 bits."""
    return codes[:n, :C].float() * scales[:n].repeat_interleave(BLOCK, -1)[:, :C]


def _plain_stats(v, norm):
    mean = v.mean(-1) if norm == "layer" else None
    d = v if mean is None else v - mean[:, None]
    return mean, torch.rsqrt(d.square().mean(-1) + EPS)


def _plain_xhat(v, mean, rstd):
    return (v if mean is None else v - mean[:, None]) * rstd[:, None]


def _plain_affine(xhat, gamma, beta):
    y = xhat * gamma.float()
    return y if beta is None else y + beta.float()


def _plain_norm(s):
    c, out = s["case"], s["out"]
    v = s["x"]
    if c["add"]:
        v = (v.float() + s["residual"].float()).to(v.dtype)
        out["total"].copy_(v)
    mean, rstd = _plain_stats(v.float(), c["norm"])
    out["rstd"].copy_(rstd)
    if mean is not None:
        out["mean"].copy_(mean)
    out["y"].copy_(_plain_affine(_plain_xhat(v.float(), mean, rstd), s["gamma"], s["beta"]))
    if c["ckpt"]:
        _plain_save(v, c["ckpt"], out["codes"], out["scales"], c["T"])
    return out


def _plain_norm_bwd(s):
    c, out = s["case"], s["out"]
    v = _plain_load(s["x"], s["scales"], c["T"], c["C"]) if c["ckpt"] else s["x"].float()
    xhat = _plain_xhat(v, s["mean"], s["rstd"])
    dy = s["dy"].float()
    g = dy * s["gamma"].float()
    d = g - xhat * (g * xhat).mean(-1, keepdim=True)
    if c["norm"] == "layer":
        d = d - g.mean(-1, keepdim=True)
        out["dbeta"].copy_(dy.sum(0))
    d = d * s["rstd"][:, None]
    if c["add"]:
        d = d + s["add"].float()
    out["dx"].copy_(d)
    out["dgamma"].copy_((dy * xhat).sum(0))
    return out


def _plain(s):
    c, out = s["case"], s["out"]
    kind = c["kind"]
    if kind == "norm":
        return _plain_norm(s)
    if kind == "norm_bwd":
        return _plain_norm_bwd(s)
    if kind == "save":
        _plain_save(s["x"], c["ckpt"], out["codes"], out["scales"], _live(c))
        return out
    if kind == "restore":
        n = _live(c)
        v = _plain_load(s["codes"], s["scales"], n, c["C"])
        if c["what"] == "rows":
            out["x"][:n] = v.to(out["x"].dtype)
        elif c["what"] == "swiglu":
            a, b = v[:, :c["C"] // 2], v[:, c["C"] // 2:]
            out["ab"][:n] = v.to(torch.bfloat16)
            out["h"][:n] = (a * torch.sigmoid(a) * b).to(torch.bfloat16)
        else:
            xhat = _plain_xhat(v, s["mean"], s["rstd"])
            out["y"].copy_(_plain_affine(xhat, s["gamma"], s["beta"]))
        return out
    if kind == "swiglu_bwd":
        n, f = _live(c), c["f"]
        v = _plain_load(s["codes"], s["scales"], n, 2 * f)
        a, b, dh = v[:, :f], v[:, f:], s["dh"][:n].float()
        sg = torch.sigmoid(a)
        out["dab"][:n, :f] = (dh * b * sg * (1.0 + a * torch.sigmoid(-a))).to(torch.bfloat16)
        out["dab"][:n, f:] = (dh * a * sg).to(torch.bfloat16)
        out["h"][:n] = (a * sg * b).to(torch.bfloat16)
        return out
    dy = s["dy"].float()
    p = s["dest_row"].long()
    kept = p >= 0
    yp = _plain_load(s["codes"], s["scales"], c["T"] * c["k"], c["C"])[p.clamp(min=0)]
    out["dw"].copy_(torch.where(kept, (dy[:, None, :] * yp).sum(-1), 0.0))
    out["dyp"][p[kept]] = (s["topk_w"][..., None] * dy[:, None, :]).to(torch.bfloat16)[kept]
    return out


# ------------------------------------------------------------------ the framework's operators
def _handle(s):
    """What a program keeps from call to call: the configuration and the workspace."""
    if "handle" not in s:
        import token_dispatch_expert_gb300 as tde
        c = s["case"]
        h = {"tde": tde}
        size = tde.FP8_WS_BYTES
        if c["kind"] == "norm_bwd":
            size = tde.moe_norm_ws_size(c["T"], c["C"])
        elif c["kind"] == "combine_bwd":
            h["cfg"] = tde.make_config(c["T"], c["C"], c["E"], c["k"], 64)
        h["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        tde.moe_ws_init(h["ws"])
        s["handle"] = h
    return s["handle"]


def _own(s):
    c, out = s["case"], s["out"]
    h = _handle(s)
    tde, ws = h["tde"], h["ws"]
    kind = c["kind"]
    if kind == "norm":
        tde.moe_norm(s["x"], out["y"], s["gamma"], s["beta"], residual=s["residual"],
                     total=out.get("total"), mean=out.get("mean"), rstd=out["rstd"],
                     codes=out.get("codes"), scales=out.get("scales"), eps=EPS, kind=c["norm"])
    elif kind == "norm_bwd":
        tde.moe_norm_bwd(s["dy"], s["x"], s["mean"], s["rstd"], out["dx"], out["dgamma"],
                         out.get("dbeta"), gamma=s["gamma"], scales=s.get("scales"), add=s["add"],
                         kind=c["norm"], ws=ws)
    elif kind == "save":
        tde.moe_ckpt_save(s["x"], out["codes"], out["scales"], offsets=s["offsets"], ws=ws)
    elif kind == "restore" and c["what"] == "rows":
        tde.moe_ckpt_load(s["codes"], s["scales"], out["x"], offsets=s["offsets"], ws=ws)
    elif kind == "restore" and c["what"] == "swiglu":
        tde.moe_ckpt_swiglu(s["codes"], s["scales"], out["ab"], out["h"], offsets=s["offsets"],
                            ws=ws)
    elif kind == "restore":
        tde.moe_ckpt_norm(s["codes"], s["scales"], s["mean"], s["rstd"], out["y"], s["gamma"],
                          s["beta"], kind=c["norm"])
    elif kind == "swiglu_bwd":
        tde.moe_ckpt_swiglu_bwd(s["dh"], s["codes"], s["scales"], out["dab"], out["h"],
                                offsets=s["offsets"], ws=ws)
    else:
        tde.moe_ckpt_combine_bwd(h["cfg"], s["dy"], s["codes"], s["scales"], s["topk_w"],
                                 s["dest_row"], out["dyp"], out["dw"], ws)
    return out


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------- the definitions in 64 bits
def _exact_save(x, fmt, n, like):
    """Codes and scales; a step over the blocks of the row."""
    codes = torch.zeros(like["codes"].shape, dtype=torch.float64, device="cuda")
    scales = torch.zeros(like["scales"].shape, dtype=torch.float64, device="cuda")
    for i, lo in enumerate(range(0, x.shape[1], BLOCK)):
        v = x[:n, lo:lo + BLOCK].double()
        top = v.abs().amax(1).clamp(min=AMAX_FLOOR)
        scales[:n, i] = top / TOP[fmt]
        # the factor is a number of 32 bits
        p = v * (TOP[fmt] / top).float().double()[:, None]
        if fmt == "int8":
            q = torch.floor(p.abs() + 0.5)
            q -= ((q - p.abs() == 0.5) & (q % 2 == 1)).double()     # ties to the even number
            q = torch.copysign(q, p)
        else:
            # three fraction bits down to an exponent of -6, of the product in 32 bits
            p = p.float().double()
            m = p.abs().clamp(max=448.0)
            step = torch.exp2(torch.frexp(m).exponent.double().sub(1).clamp(min=-6) - 3)
            q = torch.copysign(torch.round(m / step) * step, p)
        codes[:n, lo:lo + v.shape[1]] = q
    return codes.to(torch.int8) if fmt == "int8" else codes, scales


def _exact_load(codes, scales, n, C):
    v = codes[:n, :C].float().double()
    for i, lo in enumerate(range(0, C, BLOCK)):
        v[:, lo:lo + BLOCK] *= scales[:n, i, None].double()
    return v


def exact(case, seed):
    s = prepare(case, seed)
    c, out, kind = s["case"], s["out"], s["case"]["kind"]
    r = {}
    if kind == "norm":
        v = s["x"]
        if c["add"]:
            # the stream holds the 32-bit sum, rounded to its type
            v = (v.double() + s["residual"].double()).float().to(v.dtype)
            r["total"] = v.double()
        z = v.double()
        if c["norm"] == "layer":
            r["mean"] = z.sum(1) / c["C"]
            z = z - r["mean"][:, None]
        r["rstd"] = 1.0 / torch.sqrt((z * z).sum(1) / c["C"] + EPS)
        z = z * r["rstd"][:, None] * s["gamma"].double()
        r["y"] = z if s["beta"] is None else z + s["beta"].double()
        if c["ckpt"]:
            r["codes"], r["scales"] = _exact_save(v, c["ckpt"], c["T"], out)
        return {n: r[n] for n in out}
    if kind == "norm_bwd":
        v = (_exact_load(s["x"], s["scales"], c["T"], c["C"]) if c["ckpt"] else s["x"].double())
        # the Jacobian of the row's map at xhat, as a product of its factors
        z = v * s["rstd"].double()[:, None]
        if c["norm"] == "layer":
            z -= (s["mean"].double() * s["rstd"].double())[:, None]
            r["dbeta"] = s["dy"].double().sum(0)
        r["dgamma"] = torch.einsum("tc,tc->c", s["dy"].double(), z)
        g = s["dy"].double() * s["gamma"].double()
        along = torch.einsum("tc,tc->t", g, z) / c["C"]
        if c["norm"] == "layer":
            g = g - (g.sum(1) / c["C"])[:, None]
        dx = (g - along[:, None] * z) * s["rstd"].double()[:, None]
        r["dx"] = dx if s["add"] is None else dx + s["add"].double()
        return {n: r[n] for n in out}
    if kind == "save":
        return dict(zip(("codes", "scales"), _exact_save(s["x"], c["ckpt"], _live(c), out)))
    if kind in ("restore", "swiglu_bwd"):
        n = _live(c)
        w = c["C"] if kind == "restore" else 2 * c["f"]
        r = {m: torch.zeros(t.shape, dtype=torch.float64, device="cuda") for m, t in out.items()}
        v = _exact_load(s["codes"], s["scales"], n, w)
        if kind == "restore" and c["what"] == "rows":
            r["x"][:n] = v
            return r
        if kind == "restore" and c["what"] == "norm":
            if c["norm"] == "layer":
                v -= s["mean"].double()[:, None]
            r["y"][:n] = v * (s["rstd"].double()[:, None] * s["gamma"].double())
            if s["beta"] is not None:
                r["y"] += s["beta"].double()
            return r
        a, b = v[:, :w // 2], v[:, w // 2:]
        e = torch.exp(-a)
        r["h"][:n] = a * b / (1.0 + e)
        if kind == "restore":
            r["ab"][:n] = v
            return r
        dh = s["dh"][:n].double()
        r["dab"][:n, :w // 2] = dh * b * (1.0 + e + a * e) / (1.0 + e) ** 2
        r["dab"][:n, w // 2:] = dh * a / (1.0 + e)
        return r
    r = {m: torch.zeros(t.shape, dtype=torch.float64, device="cuda") for m, t in out.items()}
    token = torch.arange(c["T"], device="cuda").repeat_interleave(c["k"])
    p = s["dest_row"].reshape(-1).long()
    w = s["topk_w"].reshape(-1).double()
    dw = r["dw"].view(-1)
    for lo in range(0, p.numel(), 4096):
        at = torch.arange(lo, min(lo + 4096, p.numel()), device="cuda")
        at = at[p[at] >= 0]
        dy = s["dy"][token[at]].double()
        yp = _exact_load(s["codes"][p[at]], s["scales"][p[at]], at.numel(), c["C"])
        dw[at] = torch.einsum("pc,pc->p", dy, yp)
        r["dyp"][p[at]] = w[at, None] * dy
    return r


if __name__ == "__main__":
    rng = random.Random(0)
    for example in listed() + [draw(rng) for _ in range(12)]:
        print(example, {n: float(np.float32(v)) for n, v in work(example).items()})
