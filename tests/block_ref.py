"""Plain 64-bit references of the routing and 8-bit operators, written from their definitions
(include/moe.h) with loops over tokens and blocks.  They share no code with the kernels."""

import math

import numpy as np

BLOCK = 128


# ------------------------------------------------------------------ routing
def route_scores(l, score):
    if score == "sigmoid":
        e = np.exp(-np.abs(l))
        return np.where(l >= 0, 1 / (1 + e), e / (1 + e))
    m = l.max() if np.isfinite(l.max()) else 0.0
    e = np.exp(l - m)
    return e / e.sum() if e.sum() > 0 else e


def route(logits, k, *, score="softmax", groups=1, top_groups=None, group_top=1, renorm=True,
          bias=None, scale=1.0, capacity=0):
    T, E = logits.shape
    top_groups = groups if top_groups is None else top_groups
    per = E // groups
    idx = np.full((T, k), -1, np.int64)
    w = np.zeros((T, k))
    with np.errstate(over="ignore", invalid="ignore", under="ignore"):
        for t in range(T):
            l = np.where(np.isnan(logits[t]), -np.inf, logits[t].astype(np.float64))
            l = np.minimum(l, float(np.finfo(np.float32).max))
            live = l > -np.inf
            if not live.any():
                continue
            s = route_scores(l, score)
            key = l if bias is None else s + bias.astype(np.float64)
            worth = []
            for g in range(groups):
                mine = [e for e in range(g * per, (g + 1) * per) if live[e]]
                vals = sorted(((s if bias is None and group_top == 2 else key)[e] for e in mine),
                              reverse=True)
                worth.append(sum(vals[:group_top]) if vals else -math.inf)
            stay = sorted(range(groups), key=lambda g: (-worth[g], g))[:top_groups]
            cand = [e for g in stay for e in range(g * per, (g + 1) * per) if live[e]]
            best = sorted(cand, key=lambda e: (-key[e], e))[:k]
            idx[t, :len(best)] = best
            w[t, :len(best)] = route_weights(l, best, s, score, renorm, scale)
    return {"topk_idx": idx, "topk_w": w, **route_order(idx, E, capacity)}


def route_weights(l, best, s, score, renorm, scale):
    z = l[best]
    if not renorm:
        return scale * s[best]
    if score == "sigmoid":   # log sigma
        z = np.minimum(z, 0) - np.log1p(np.exp(-np.abs(z)))
    e = np.exp(z - z.max())
    return scale * e / e.sum()


def route_order(idx, E, capacity):
    T, k = idx.shape
    counts = np.zeros(E, np.int64)
    rank = np.full((T, k), -1, np.int64)
    for t in range(T):
        for j in range(k):
            if idx[t, j] >= 0:
                rank[t, j] = counts[idx[t, j]]
                counts[idx[t, j]] += 1
    kept = np.minimum(counts, capacity) if capacity else counts
    off = np.concatenate([[0], np.cumsum(kept)])
    dest = np.full((T, k), -1, np.int64)
    src = np.full(T * k, -1, np.int64)
    for t in range(T):
        for j in range(k):
            e = idx[t, j]
            if e >= 0 and rank[t, j] < kept[e]:
                dest[t, j] = off[e] + rank[t, j]
                src[dest[t, j]] = t * k + j
    return {"counts": counts, "kept": kept, "offsets": off, "dest_row": dest,
            "src_tok": np.where(src < 0, -1, src // k), "src_slot": src,
            "drop_mask": (dest < 0).astype(np.int64)}


def route_grad(logits, idx, dw, *, score="softmax", renorm=True, scale=1.0):
    """Jacobian form: dl = J^T dw with J the derivative of the weights, one token at a time."""
    T, E = logits.shape
    out = np.zeros((T, E))
    for t in range(T):
        l = logits[t].astype(np.float64)
        sel = [(j, e) for j, e in enumerate(idx[t]) if e >= 0]
        if not sel:
            continue
        js, es = [j for j, _ in sel], [e for _, e in sel]
        s = route_scores(l, score)
        ds = np.diag(s * (1 - s)) if score == "sigmoid" else np.diag(s) - np.outer(s, s)
        J = ds[es]                                    # d score / d logit
        if renorm:
            S = s[es].sum()
            J = J / S - np.outer(s[es], J.sum(0)) / S ** 2
        out[t] = scale * dw[t, js].astype(np.float64) @ J
    return out


# ------------------------------------------------------------------ blocks of 128
def e4m3(v):
    """The value of the E4M3 number nearest to v (ties to even, saturated at 448)."""
    v = np.asarray(v, np.float64)
    a = np.minimum(np.abs(v), 448.0)
    _, e = np.frexp(a)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.where(np.isnan(v), np.nan, np.copysign(np.rint(a / step) * step, v))


def scale_of(amax, pow2):
    """(stored scale, factor) as fp32 numbers held in 64 bits."""
    amax = np.where(amax < 2.0 ** -110, 2.0 ** -110, amax).astype(np.float32)
    with np.errstate(all="ignore"):
        if not pow2:
            return ((amax / np.float32(448)).astype(np.float64),
                    (np.float32(448) / amax).astype(np.float64))
        m, e = np.frexp(amax.astype(np.float64) / 448.0)
        n = np.where(m == 0.5, e - 1, e)
        fine = np.isfinite(amax)   # an infinite or NaN scale has no next power of two
        return (np.where(fine, np.ldexp(1.0, n), amax / 448.0),
                np.where(fine, np.ldexp(1.0, -n), 448.0 / amax.astype(np.float64)))


def quantise_rows(x, pow2=False):
    """x [R, C] -> (values of the codes [R, C], scales [R, ceil(C/128)])."""
    R, C = x.shape
    codes = np.zeros((R, C))
    scales = np.zeros((R, -(-C // BLOCK)))
    for b in range(scales.shape[1]):
        v = x[:, b * BLOCK:(b + 1) * BLOCK].astype(np.float64)
        with np.errstate(all="ignore"):
            scales[:, b], f = scale_of(np.abs(v).max(1), pow2)
            codes[:, b * BLOCK:b * BLOCK + v.shape[1]] = e4m3((v * f[:, None]).astype(np.float32))
    return codes, scales


def quantise_tokens(x, offsets, pow2=False):
    """x [R, C] -> (values [C, 128 B], scales [B, C], B blocks used), from the segments' starts."""
    C = x.shape[1]
    codes, scales = [], []
    for lo, hi in zip(offsets, offsets[1:]):
        for r in range(lo, hi, BLOCK):
            c, s = quantise_rows(x[r:min(r + BLOCK, hi)].T, pow2)
            codes.append(np.pad(c, ((0, 0), (0, BLOCK - c.shape[1]))))
            scales.append(s[:, 0])
    if not codes:
        return np.zeros((C, 0)), np.zeros((0, C))
    return np.concatenate(codes, 1), np.stack(scales)


def quantise_weights(w, pow2=False):
    """w [N, K] -> (values, scales [ceil(N/128), ceil(K/128)])."""
    N, K = w.shape
    codes = np.zeros((N, K))
    scales = np.zeros((-(-N // BLOCK), -(-K // BLOCK)))
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            at = np.s_[i * BLOCK:min((i + 1) * BLOCK, N), j * BLOCK:min((j + 1) * BLOCK, K)]
            v = w[at].astype(np.float64)
            s, f = scale_of(np.abs(v).max()[None], pow2)
            scales[i, j] = s[0]
            codes[at] = e4m3((v * f[0]).astype(np.float32))
    return codes, scales


def spread(scales, n, axis):
    return np.repeat(scales, BLOCK, axis).take(range(n), axis)


def bf16(v):
    """Nearest bf16 number (through fp32, ties to even) of 64-bit values."""
    u = np.ascontiguousarray(np.asarray(v, np.float64).astype(np.float32)).view(np.uint32)
    r = ((u.astype(np.uint64) + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32)
    return np.where(np.isnan(v), np.nan, r.view(np.float32).astype(np.float64))


def swiglu(ab):
    f = ab.shape[1] // 2
    a, b = ab[:, :f].astype(np.float64), ab[:, f:].astype(np.float64)
    return bf16(a / (1 + np.exp(-a)) * b)


def swiglu_bwd(dh, ab):
    f = dh.shape[1]
    a, b, d = ab[:, :f].astype(np.float64), ab[:, f:].astype(np.float64), dh.astype(np.float64)
    s = 1 / (1 + np.exp(-a))
    return bf16(np.concatenate([d * b * s * (1 + a * (1 - s)), d * a * s], 1))
