"""The cases that the routing and 8-bit operators are measured on, with their plain forms.

Six kinds of call, as a program that trains or serves a mixture of experts makes them:

  route         router scores (softmax or sigmoid), a balance bias that only the choice sees,
                group-limited top-k, weights renormalised or not, capacity, and the side arrays
                of the padding-free expert order
  route_grad    the gradient of the weights with respect to the logits
  quantise      bf16 rows -> E4M3 codes with one scale for each block of 128 along the row
                (optionally gathered into expert order), and along the tokens of each expert's
                segment for a weight gradient; weights with one scale for each 128 x 128 block
  swiglu        silu(a) * b quantised for the next product; its backward quantises [da | db]
  product       out[p] = A[p] B[e]^T for the rows p of each expert e, on codes and scales
  weight_grad   dW[e] = A_e^T B_e over each expert's rows, on codes scaled along the tokens

`own` selects between the plain forms below and the framework's operators.
"""

import math
import random

import numpy as np
import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -110      # a block's largest magnitude is held above this
F32_MAX = torch.finfo(torch.float32).max


# ------------------------------------------------------------------------------ the cases
def listed():
    return [
        # one token being decoded by a 256-expert layer with eight groups: pure latency
        dict(name="route_one_token", kind="route", T=1, E=256, k=8, groups=8, top_groups=4,
             group_top=2, score="sigmoid", bias=True, renorm=True, scale=2.5, capacity=0,
             masked=0.0),
        # a training batch of the same layer, some rows of it padding (every expert masked)
        dict(name="route_grouped_batch", kind="route", T=4096, E=256, k=8, groups=8,
             top_groups=4, group_top=2, score="sigmoid", bias=True, renorm=True, scale=2.5,
             capacity=0, masked=0.02),
        # the gradient of softmax weights that are not renormalised: dense over the experts
        dict(name="route_grad_softmax", kind="route_grad", T=8192, E=128, k=8, groups=1,
             top_groups=1, group_top=1, score="softmax", bias=False, renorm=False, scale=1.0,
             capacity=0, masked=0.0),
        # dispatch: the tokens of a batch gathered into expert order and quantised on the way
        dict(name="quantise_dispatch", kind="quantise", what="gather", T=4096, k=8, G=256,
             C=7168, skew=1.2, pow2=False),
        # upstream gradients, both ways of a step: along the row and along the tokens; ragged
        dict(name="quantise_both_ragged", kind="quantise", what="both", T=8191, k=2, G=8,
             C=2056, skew=0.5, pow2=False),
        # the activation between the two products of a fine-grained layer
        dict(name="swiglu_rows", kind="swiglu", back=False, R=65536, G=128, f=768, skew=0.55,
             tokens=False, pow2=False),
        # its backward for a layer of wide experts, with what the weight gradients read
        dict(name="swiglu_back_tokens", kind="swiglu", back=True, R=16383, G=64, f=1408,
             skew=1.5, tokens=True, pow2=False),
        # one token's eight experts: weights stream past a single row each
        dict(name="product_one_token", kind="product", R=8, G=256, N=4096, K=7168, skew=0.0,
             out="bf16"),
        # a batch over 128 fine-grained experts of uneven load, gate and up projections
        dict(name="product_fine_grained", kind="product", R=65536, G=128, N=1536, K=2048,
             skew=0.55, out="bf16"),
        # a batch over eight wide experts: the largest product
        dict(name="product_wide", kind="product", R=8192, G=8, N=28672, K=4096, skew=0.0,
             out="bf16"),
        # weight gradients of the fine-grained layer's down projection
        dict(name="weight_grad_fine_grained", kind="weight_grad", R=65536, G=128, M=2048, N=768,
             skew=0.55, out="bf16"),
        # odd sizes, few experts of uneven and partly empty segments, a 32-bit gradient
        dict(name="weight_grad_odd", kind="weight_grad", R=5001, G=8, M=1000, N=1413, skew=2.0,
             out="fp32"),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    n = max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n - (n == 3072)


def _blocks(rng, most):
    """A multiple of the block, up to `most` blocks."""
    return BLOCK * rng.choice([n for n in range(1, most + 1) if n not in (12, 24)])


def draw(rng):
    kind = rng.choice(["route", "route_grad", "quantise", "swiglu", "product", "weight_grad"])
    if kind in ("route", "route_grad"):
        groups = rng.choice([1, 1, 2, 4, 8, 16])
        per = rng.choice([p for p in (2, 4, 5, 8, 16, 32, 60) if groups * p <= 256])
        top = rng.randint(max(1, -(-2 // per)), groups)
        k = rng.randint(1, min(8, top * per))
        T = _log(rng, 1, 16384)
        return dict(kind=kind, T=T, E=groups * per, k=k, groups=groups, top_groups=top,
                    group_top=rng.choice([1, 2]), score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, renorm=rng.random() < 0.5,
                    scale=rng.choice([1.0, 2.5]),
                    capacity=rng.choice([0, 0, max(1, T * k // (groups * per))]),
                    masked=rng.choice([0.0, 0.0, 0.1]))
    skew = rng.choice([0.0, 0.55, 1.2])
    G = rng.choice([1, 8, 64, 128, 256])
    pow2 = rng.random() < 0.25
    if kind == "quantise":
        what = rng.choice(["rows", "gather", "both", "tokens", "weights"])
        C = _log(rng, 64, 7168) if rng.random() < 0.4 else _blocks(rng, 56)
        if what == "weights":
            return dict(kind=kind, what=what, T=_log(rng, 64, 4096), k=1,
                        G=rng.choice([1, 2, 5, 8]), C=C, skew=0.0, pow2=pow2)
        return dict(kind=kind, what=what, T=_log(rng, 1, 8192), k=rng.choice([1, 2, 4]), G=G,
                    C=C, skew=skew, pow2=pow2)
    if kind == "swiglu":
        f = _log(rng, 32, 2048) if rng.random() < 0.4 else _blocks(rng, 16)
        return dict(kind=kind, back=rng.random() < 0.5, R=_log(rng, 1, 16384), G=G, f=f,
                    skew=skew, tokens=rng.random() < 0.5, pow2=pow2)
    out = rng.choice(["bf16", "bf16", "fp32"])
    odd = rng.random() < 0.4
    size = (lambda lo, hi: _log(rng, lo, hi) if odd
            else min((n for n in range(BLOCK, 8193, BLOCK) if n // BLOCK not in (12, 24)),
                     key=lambda n, v=_log(rng, lo, hi): abs(n - v)))
    if kind == "product":
        R, K = _log(rng, 1, 16384), size(64, 7168)
        N = size(64, min(8192, max(64, int(4e8 / (G * K)))))
        return dict(kind=kind, R=R, G=G, N=N, K=K, skew=skew, out=out)
    M = size(64, 4096)
    N = size(64, min(4096, max(64, int(2e8 / (G * M)))))
    return dict(kind=kind, R=_log(rng, 1, 16384), G=G, M=M, N=N, skew=skew, out=out)


def work(case):
    """Each input read once, each output written once; two operations a multiply-add."""
    c = case
    if c["kind"] == "route":
        slots = c["T"] * c["k"]
        # idx, weight, destination, token, slot (4 bytes each) and the drop mask
        return {"bytes": 4 * c["T"] * c["E"] + 21 * slots + 12 * c["E"], "flops": 8 * c["T"] * c["E"]}
    if c["kind"] == "route_grad":
        read = c["E"] if c["score"] == "softmax" and not c["renorm"] else c["k"]
        return {"bytes": 4 * c["T"] * (read + c["E"]) + 8 * c["T"] * c["k"],
                "flops": 8 * c["T"] * read}
    if c["kind"] == "quantise":
        blocks = -(-c["C"] // BLOCK)
        if c["what"] == "weights":
            n = c["G"] * c["T"] * c["C"]
            return {"bytes": 4 * n + 8 * c["G"] * blocks * -(-c["T"] // BLOCK), "flops": 3 * n}
        R = c["T"] * c["k"]
        read = 2 * (c["T"] if c["what"] == "gather" else R) * c["C"]
        wrote = 0
        if c["what"] != "tokens":
            wrote += R * c["C"] + 4 * R * blocks
        if c["what"] in ("both", "tokens"):
            wrote += R * c["C"] + 4 * -(-R // BLOCK) * c["C"]
        return {"bytes": read + wrote, "flops": 3 * R * c["C"]}
    if c["kind"] == "swiglu":
        n = c["R"] * c["f"]
        read, wrote = (6 * n, 2 * n) if c["back"] else (4 * n, n)
        if c["tokens"]:
            wrote += 3 * n if c["back"] else n
        return {"bytes": read + wrote * (1 + 4.0 / BLOCK), "flops": (20 if c["back"] else 8) * n}
    size = 4 if c["out"] == "fp32" else 2
    if c["kind"] == "product":
        used = min(c["G"], c["R"])
        return {"bytes": c["R"] * c["K"] + used * c["N"] * c["K"] + size * c["R"] * c["N"],
                "flops": 2 * c["R"] * c["N"] * c["K"]}
    return {"bytes": c["R"] * (c["M"] + c["N"]) + size * c["G"] * c["M"] * c["N"],
            "flops": 2 * c["R"] * c["M"] * c["N"]}


# ------------------------------------------------------------------------------ the inputs
def _gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed))
    return g


def _segments(case, R, seed):
    """Lengths of the experts' segments: R rows spread by a Zipf law of the given strength."""
    G = case["G"]
    r = np.random.default_rng([int(seed), 7])
    p = r.permutation(np.arange(1, G + 1)).astype(np.float64) ** -case["skew"]
    if R <= G and case["skew"] == 0.0:      # a token's experts: one row each
        rows = np.zeros(G, np.int64)
        rows[np.sort(r.permutation(G)[:R])] = 1
    else:
        rows = r.multinomial(R, p / p.sum())
    return [int(v) for v in np.concatenate([[0], np.cumsum(rows)])]


def _normal(shape, seed, scale=1.0, dtype=torch.bfloat16):
    x = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(generator=_gen(seed))
    return (x * scale).to(dtype)


def _activations(R, C, seed):
    """Rows as a trained network has them: unit scale, a few channels twenty times larger."""
    x = torch.empty((R, C), dtype=torch.float32, device="cuda").normal_(generator=_gen(seed))
    wide = torch.rand(C, generator=_gen(seed + 1), device="cuda") < 0.01
    return (x * (1.0 + 19.0 * wide)).to(torch.bfloat16)


def _up(n, m):
    return -(-n // m) * m


def _token_blocks(offsets):
    """First 128-row block of each segment, in the order that the segments' blocks follow."""
    first = [0]
    for a, b in zip(offsets, offsets[1:]):
        first.append(first[-1] + -(-(b - a) // BLOCK))
    return first


def _block_cap(R, G):
    return -(-R // BLOCK) + G


def _codes(shape):
    return torch.zeros(shape, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)


def prepare(case, seed):
    c = dict(case)
    s = {"case": c}
    kind = c["kind"]
    if kind in ("route", "route_grad"):
        T, E, k = c["T"], c["E"], c["k"]
        lg = torch.empty((T, E), dtype=torch.float32, device="cuda").normal_(generator=_gen(seed))
        rank = torch.randperm(E, generator=_gen(seed + 1), device="cuda") + 1
        lg -= 0.6 * torch.log(rank.float())           # uneven popularity
        if c["masked"]:
            # experts out of service for a token, and padding tokens with none in service
            lg[torch.rand((T, E), generator=_gen(seed + 2), device="cuda") < c["masked"]] = -math.inf
            lg[torch.rand(T, generator=_gen(seed + 3), device="cuda") < c["masked"]] = -math.inf
        s["logits"] = lg
        s["bias"] = None
        if c["bias"]:
            s["bias"] = 0.05 * torch.log(rank.float()) + 0.01 * torch.empty(
                E, device="cuda").normal_(generator=_gen(seed + 4))
        if kind == "route_grad":
            s["idx"] = _plain_route(s)["topk_idx"]
            s["dw"] = _normal((T, k), seed + 5, dtype=torch.float32)
            s["out"] = {"dlogits": torch.empty_like(lg)}
        else:
            i32 = dict(dtype=torch.int32, device="cuda")
            s["out"] = {"topk_idx": torch.empty((T, k), **i32),
                        "topk_w": torch.empty((T, k), dtype=torch.float32, device="cuda"),
                        "counts": torch.empty(E, **i32), "kept": torch.empty(E, **i32),
                        "offsets": torch.empty(E + 1, **i32),
                        "dest_row": torch.empty((T, k), **i32),
                        "src_tok": torch.empty(T * k, **i32),
                        "src_slot": torch.empty(T * k, **i32),
                        "drop_mask": torch.empty((T, k), dtype=torch.uint8, device="cuda")}
        return s
    if kind == "quantise" and c["what"] == "weights":
        G, N, K = c["G"], c["T"], c["C"]
        s["x"] = _normal((G, N, K), seed, 0.02)
        s["out"] = {"codes": _codes((G, N, _up(K, 16))), "codes_t": _codes((G, K, _up(N, 16))),
                    "scales": torch.zeros((G, -(-N // BLOCK), -(-K // BLOCK)), device="cuda"),
                    "scales_t": torch.zeros((G, -(-K // BLOCK), -(-N // BLOCK)), device="cuda")}
        return s
    R = c["R"] if "R" in c else c["T"] * c["k"]
    G = c["G"]
    s["offsets_host"] = _segments(c, R, seed)
    s["blocks_host"] = _token_blocks(s["offsets_host"])
    s["offsets"] = torch.tensor(s["offsets_host"], dtype=torch.int32, device="cuda")
    cap = _block_cap(R, G)
    if kind == "quantise":
        C, what = c["C"], c["what"]
        if what == "gather":
            # every token appears k times among the rows, in ascending order in a segment
            perm = torch.randperm(R, generator=_gen(seed + 9), device="cuda") // c["k"]
            group = torch.bucketize(torch.arange(R, device="cuda"), s["offsets"][1:-1].contiguous(),
                                    right=True)
            order = torch.argsort(group * c["T"] + perm)
            s["src_tok"] = perm[order].to(torch.int32)
            s["x"] = _activations(c["T"], C, seed)
        else:
            s["x"] = _activations(R, C, seed)
        s["out"] = {}
        if what != "tokens":
            s["out"] |= {"codes": _codes((R, _up(C, 16))),
                         "scales": torch.zeros((R, -(-C // BLOCK)), device="cuda")}
        if what in ("both", "tokens"):
            s["out"] |= {"codes_t": _codes((C, BLOCK * cap)),
                         "scales_t": torch.zeros((cap, C), device="cuda")}
        return s
    if kind == "swiglu":
        f = c["f"]
        s["ab"] = _normal((R, 2 * f), seed, 1.3)
        w = 2 * f if c["back"] else f
        if c["back"]:
            s["dh"] = _normal((R, f), seed + 1, 0.1)
        s["out"] = {"codes": _codes((R, _up(w, 16))),
                    "scales": torch.zeros((R, -(-w // BLOCK)), device="cuda")}
        if c["tokens"]:
            s["out"] |= {"codes_t": _codes((w, BLOCK * cap)),
                         "scales_t": torch.zeros((cap, w), device="cuda")}
            if c["back"]:
                s["out"] |= {"h_codes_t": _codes((f, BLOCK * cap)),
                             "h_scales_t": torch.zeros((cap, f), device="cuda")}
        return s
    dt = torch.float32 if c["out"] == "fp32" else torch.bfloat16
    if kind == "product":
        N, K = c["N"], c["K"]
        s["a"], s["a_scales"] = _codes((R, _up(K, 16))), torch.zeros((R, -(-K // BLOCK)), device="cuda")
        _plain_rows(_activations(R, K, seed), False, s["a"], s["a_scales"])
        s["b"] = _codes((G, N, _up(K, 16)))
        s["b_scales"] = torch.zeros((G, -(-N // BLOCK), -(-K // BLOCK)), device="cuda")
        for g in range(G):
            _plain_weights(_normal((1, N, K), seed + 100 + g, 0.02), False, s["b"][g:g + 1],
                           s["b_scales"][g:g + 1])
        s["out"] = {"out": torch.zeros((R, N), dtype=dt, device="cuda")}
        return s
    M, N = c["M"], c["N"]
    for name, C, at in (("a", M, seed), ("b", N, seed + 50)):
        s[name], s[name + "_scales"] = _codes((C, BLOCK * cap)), torch.zeros((cap, C), device="cuda")
        _plain_tokens(_activations(R, C, at), False, s["offsets"], s["blocks_host"], s[name],
                      s[name + "_scales"])
    s["out"] = {"dw": torch.empty((G, M, N), dtype=dt, device="cuda")}
    return s


# ------------------------------------------------------------------------- the plain forms
def _scale_and_inverse(amax, pow2):
    """A block's scale and the factor its values are multiplied by, in 32 bits."""
    amax = torch.where(amax.isnan(), amax, amax.clamp(min=AMAX_FLOOR))
    if not pow2:
        # quotients of two tensors: each correctly rounded (a quotient with a Python number may
        # be a product with its rounded reciprocal)
        top = torch.full_like(amax, E4M3_MAX)
        return amax / top, top / amax
    # the next power of two at or above amax / 448
    m, e = torch.frexp(amax.double() / E4M3_MAX)
    e = torch.where(m == 0.5, e - 1, e)
    return torch.exp2(e.double()).float(), torch.exp2(-e.double()).float()


def _e4m3(v):
    return v.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _u8(t):
    return t.view(torch.uint8)


def _plain_rows(x, pow2, codes, scales):
    """One scale for each 128 elements of a row; the last block of a row may be short."""
    R, C = x.shape
    v = torch.nn.functional.pad(x.float(), (0, _up(C, BLOCK) - C)).view(R, -1, BLOCK)
    sc, inv = _scale_and_inverse(v.abs().amax(-1), pow2)
    _u8(codes)[:, :C] = _u8(_e4m3(v * inv[..., None])).view(R, -1)[:, :C]
    scales.copy_(sc)


def _plain_tokens(x, pow2, offsets, blocks, codes_t, scales_t):
    """One scale for each column and each 128 rows of a segment, counted from its first row;
    codes transposed, a segment's last block filled up with zeros."""
    R, C = x.shape
    row = torch.arange(R, device=x.device)
    seg = torch.bucketize(row, offsets[1:-1].contiguous(), right=True)
    first = torch.tensor(blocks, device=x.device)
    at = first[seg] * BLOCK + row - offsets.long()[seg]
    padded = torch.zeros((blocks[-1] * BLOCK, C), dtype=torch.float32, device=x.device)
    padded[at] = x.float()
    v = padded.view(-1, BLOCK, C)
    sc, inv = _scale_and_inverse(v.abs().amax(1), pow2)
    q = _u8(_e4m3(v * inv[:, None, :])).view(-1, C)
    _u8(codes_t)[:, : q.shape[0]] = q.t()
    scales_t[: sc.shape[0]] = sc


def _plain_weights(w, pow2, codes, scales, codes_t=None, scales_t=None):
    G, N, K = w.shape
    v = torch.nn.functional.pad(w.float(), (0, _up(K, BLOCK) - K, 0, _up(N, BLOCK) - N))
    v = v.view(G, v.shape[1] // BLOCK, BLOCK, -1, BLOCK)
    sc, inv = _scale_and_inverse(v.abs().amax(4).amax(2), pow2)
    q = _u8(_e4m3(v * inv[:, :, None, :, None]))
    q = q.reshape(G, v.shape[1] * BLOCK, -1)[:, :N, :K]
    _u8(codes)[:, :, :K] = q
    scales.copy_(sc)
    if codes_t is not None:
        _u8(codes_t)[:, :, :N] = q.transpose(1, 2)
        scales_t.copy_(sc.transpose(1, 2))


def _plain_route(s):
    c, bias = s["case"], s["bias"]
    T, E, k, groups = c["T"], c["E"], c["k"], c["groups"]
    # the choice is made in 64 bits: two experts' scores may lie next to each other
    l = s["logits"].double()
    l = torch.where(l.isnan(), -math.inf, l).clamp(max=F32_MAX)
    dead = l == -math.inf
    if c["score"] == "sigmoid":
        p = torch.sigmoid(l)
    else:
        m = l.amax(-1, keepdim=True).clamp(min=-F32_MAX)
        e = torch.exp(l - m)
        p = e / e.sum(-1, keepdim=True).clamp(min=1e-300)
    key = l if bias is None else p + bias.double()
    key = torch.where(dead, -math.inf, key)
    if groups > 1:
        if c["group_top"] == 1:
            worth = key.view(T, groups, -1).amax(-1)
        else:
            two = torch.where(dead, -math.inf, p if bias is None else key).view(T, groups, -1)
            two = two.topk(2, dim=-1).values
            worth = two[..., 0] + torch.where(two[..., 1] == -math.inf, 0.0, two[..., 1])
        order = worth.sort(dim=-1, descending=True, stable=True).indices
        allowed = torch.zeros((T, groups), dtype=torch.bool, device=l.device)
        allowed.scatter_(1, order[:, : c["top_groups"]], True)
        key = torch.where(allowed.repeat_interleave(E // groups, 1), key, -math.inf)
    best = key.sort(dim=-1, descending=True, stable=True)
    idx = best.indices[:, :k]
    taken = best.values[:, :k] > -math.inf
    chosen = l.gather(1, idx)
    if c["renorm"]:
        z = torch.nn.functional.logsigmoid(chosen) if c["score"] == "sigmoid" else chosen
        z = torch.where(taken, z, -math.inf)
        w = torch.exp(z - z.amax(-1, keepdim=True).clamp(min=-F32_MAX))
        w = w / w.sum(-1, keepdim=True).clamp(min=1e-300)
    else:
        w = torch.where(taken, p.gather(1, idx), 0.0)
    idx = torch.where(taken, idx, -1)
    # expert order: a stable sort of the slots by expert, unfilled slots last
    slot = idx.reshape(-1)
    by = torch.where(slot < 0, E, slot)
    counts = torch.bincount(by, minlength=E + 1)[:E]
    kept = counts.clamp(max=c["capacity"]) if c["capacity"] else counts
    zero = counts.new_zeros(1)
    offsets = torch.cat([zero, kept.cumsum(0)])
    start = torch.cat([zero, counts.cumsum(0)])
    order = by.sort(stable=True).indices
    rank = torch.empty_like(order)
    rank[order] = torch.arange(T * k, device=l.device)
    rank = rank - start[by]
    stays = (slot >= 0) & (rank < torch.cat([kept, zero])[by])
    dest = torch.where(stays, offsets[by] + rank, -1)
    src = torch.full((T * k + 1,), -1, dtype=torch.int64, device=l.device)
    src[torch.where(stays, dest, T * k)] = torch.arange(T * k, device=l.device)
    src = src[: T * k]
    i32 = torch.int32
    return {"topk_idx": idx.to(i32), "topk_w": (c["scale"] * w).float(), "counts": counts.to(i32),
            "kept": kept.to(i32), "offsets": offsets.to(i32), "dest_row": dest.view(T, k).to(i32),
            "src_tok": torch.where(src < 0, -1, src // k).to(i32), "src_slot": src.to(i32),
            "drop_mask": (~stays).view(T, k).to(torch.uint8)}


def _plain_route_grad(s):
    c, l, idx, dw = s["case"], s["logits"], s["idx"].long(), s["dw"]
    live = idx >= 0
    at = idx.clamp(min=0)
    dw = torch.where(live, dw, 0.0)
    z = l.gather(1, at)
    if c["renorm"]:
        u = torch.where(live, torch.nn.functional.logsigmoid(z) if c["score"] == "sigmoid" else z,
                        -math.inf)
        u = torch.exp(u - u.amax(-1, keepdim=True).clamp(min=-F32_MAX))
        u = u / u.sum(-1, keepdim=True).clamp(min=1e-37)
        d = c["scale"] * u * (u[:, None, :] * (dw[:, :, None] - dw[:, None, :])).sum(-1)
        if c["score"] == "sigmoid":
            d = d * torch.sigmoid(-z)
    elif c["score"] == "sigmoid":
        d = c["scale"] * dw * torch.sigmoid(z) * torch.sigmoid(-z)
    else:
        e = torch.exp(l - l.amax(-1, keepdim=True).clamp(min=-F32_MAX))
        p = e / e.sum(-1, keepdim=True).clamp(min=1e-37)
        g = torch.zeros_like(l).scatter_add_(1, at, torch.where(live, c["scale"] * dw, 0.0))
        return {"dlogits": p * (g - (p * g).sum(-1, keepdim=True))}
    d = torch.where(live, d, 0.0)
    return {"dlogits": torch.zeros_like(l).scatter_add_(1, at, d)}


def _plain_swiglu(s):
    """h, or [da | db] and h, each value rounded once to bf16 as the layer's path holds it."""
    f = s["case"]["f"]
    # 64 bits: a value next to the border of two bf16 numbers decides a code of the block
    a, b = s["ab"][:, :f].double(), s["ab"][:, f:].double()
    sg = torch.sigmoid(a)
    h = (a * sg * b).to(torch.float32).to(torch.bfloat16)
    if not s["case"]["back"]:
        return h, h
    dh = s["dh"].double()
    da = dh * b * sg * (1.0 + a * torch.sigmoid(-a))
    return torch.cat([da, dh * a * sg], 1).to(torch.float32).to(torch.bfloat16), h


def _dequant(codes, scales, n):
    return codes[..., :n].float() * scales.repeat_interleave(BLOCK, -1)[..., :n]


def _plain(s):
    c, out = s["case"], s["out"]
    kind = c["kind"]
    if kind == "route":
        return _plain_route(s)
    if kind == "route_grad":
        return _plain_route_grad(s)
    if kind == "quantise":
        if c["what"] == "weights":
            _plain_weights(s["x"], c["pow2"], out["codes"], out["scales"], out["codes_t"],
                           out["scales_t"])
            return out
        x = s["x"][s["src_tok"].long()] if c["what"] == "gather" else s["x"]
        if "codes" in out:
            _plain_rows(x, c["pow2"], out["codes"], out["scales"])
        if "codes_t" in out:
            _plain_tokens(x, c["pow2"], s["offsets"], s["blocks_host"], out["codes_t"],
                          out["scales_t"])
        return out
    if kind == "swiglu":
        y, h = _plain_swiglu(s)
        _plain_rows(y, c["pow2"], out["codes"], out["scales"])
        if c["tokens"]:
            _plain_tokens(y, c["pow2"], s["offsets"], s["blocks_host"], out["codes_t"],
                          out["scales_t"])
            if c["back"]:
                _plain_tokens(h, c["pow2"], s["offsets"], s["blocks_host"], out["h_codes_t"],
                              out["h_scales_t"])
        return out
    off, blk = s["offsets_host"], s["blocks_host"]
    if kind == "product":
        N, K = c["N"], c["K"]
        for g in range(c["G"]):
            lo, hi = off[g], off[g + 1]
            if hi > lo:
                a = _dequant(s["a"][lo:hi], s["a_scales"][lo:hi], K)
                b = _dequant(s["b"][g], s["b_scales"][g].repeat_interleave(BLOCK, 0)[:N], K)
                out["out"][lo:hi] = (a @ b.t()).to(out["out"].dtype)
        return out
    for g in range(c["G"]):
        lo, hi = blk[g], blk[g + 1]
        if hi > lo:
            a = _dequant(s["a"][:, lo * BLOCK:hi * BLOCK], s["a_scales"][lo:hi].t(), (hi - lo) * BLOCK)
            b = _dequant(s["b"][:, lo * BLOCK:hi * BLOCK], s["b_scales"][lo:hi].t(), (hi - lo) * BLOCK)
            out["dw"][g] = (a @ b.t()).to(out["dw"].dtype)
        else:
            out["dw"][g] = 0
    return out


# ------------------------------------------------------------------ the framework's operators
def _handle(s):
    """What a program keeps from call to call: the configuration and the workspace."""
    if "handle" not in s:
        import token_dispatch_expert_gb300 as tde
        c = s["case"]
        h = {"tde": tde}
        if c["kind"] in ("route", "route_grad"):
            h["cfg"] = tde.make_config(c["T"], 64, c["E"], c["k"], 64, route_scale=c["scale"],
                                       capacity=c["capacity"])
            h["router"] = tde.make_router(c["score"], groups=c["groups"],
                                          top_groups=c["top_groups"], group_top=c["group_top"],
                                          renorm=c["renorm"], bias=s["bias"])
            size = tde.moe_workspace_size(h["cfg"])[0]
        else:
            size = tde.FP8_WS_BYTES
        h["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        tde.moe_ws_init(h["ws"])
        s["handle"] = h
    return s["handle"]


def _own(s):
    c, out = s["case"], s["out"]
    h = _handle(s)
    tde, ws = h["tde"], h["ws"]
    kind = c["kind"]
    if kind == "route":
        tde.moe_route_groups(h["cfg"], h["router"], s["logits"], out["topk_idx"], out["topk_w"],
                             out["counts"], out["kept"], out["offsets"], out["dest_row"],
                             out["src_tok"], out["src_slot"], out["drop_mask"], ws)
    elif kind == "route_grad":
        tde.moe_route_groups_bwd(h["cfg"], h["router"], s["logits"], s["idx"], s["dw"],
                                 out["dlogits"], ws)
    elif kind == "quantise" and c["what"] == "weights":
        tde.moe_fp8_quantize_weights(s["x"], out["codes"], out["scales"], out["codes_t"],
                                     out["scales_t"], pow2=c["pow2"])
    elif kind == "quantise":
        tde.moe_fp8_quantize(s["x"], out.get("codes"), out.get("scales"), out.get("codes_t"),
                             out.get("scales_t"), offsets=s["offsets"], src_tok=s.get("src_tok"),
                             pow2=c["pow2"], ws=ws)
    elif kind == "swiglu" and not c["back"]:
        tde.moe_fp8_swiglu(s["ab"], out["codes"], out["scales"], out.get("codes_t"),
                           out.get("scales_t"), offsets=s["offsets"], pow2=c["pow2"], ws=ws)
    elif kind == "swiglu":
        tde.moe_fp8_swiglu_bwd(s["dh"], s["ab"], out["codes"], out["scales"], out.get("codes_t"),
                               out.get("scales_t"), out.get("h_codes_t"), out.get("h_scales_t"),
                               offsets=s["offsets"], pow2=c["pow2"], ws=ws)
    elif kind == "product":
        tde.moe_fp8_gemm(s["a"], s["a_scales"], s["b"], s["b_scales"], out["out"], c["K"],
                         offsets=s["offsets"], ws=ws)
    else:
        tde.moe_fp8_wgrad(s["a"], s["a_scales"], s["b"], s["b_scales"], out["dw"],
                          offsets=s["offsets"], ws=ws)
    return out


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------- the definitions in 64 bits
def _grid(v):
    """The E4M3 number nearest to v (ties to the even one): three fraction bits down to an
    exponent of -6, at most 448."""
    m, e = torch.frexp(v.abs().clamp(max=E4M3_MAX))
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3.0)
    return torch.copysign(torch.round(v.abs().clamp(max=E4M3_MAX) / step) * step, v)


def _exact_scale(top, pow2):
    """The stored scale and the 32-bit factor that the definition multiplies by."""
    top = torch.maximum(top, torch.full_like(top, AMAX_FLOOR))
    if pow2:
        e = torch.ceil(torch.log2(top / E4M3_MAX))
        e = torch.where(torch.exp2(e - 1) >= top / E4M3_MAX, e - 1, e)
        return torch.exp2(e), torch.exp2(-e)
    return top / E4M3_MAX, (E4M3_MAX / top).float().double()


def _exact_rows(x, pow2, wide):
    """Codes and scales along the rows of x; a step over the blocks of the row."""
    R, C = x.shape
    codes = torch.zeros((R, wide), dtype=torch.float64, device=x.device)
    scales = torch.zeros((R, -(-C // BLOCK)), dtype=torch.float64, device=x.device)
    for i, lo in enumerate(range(0, C, BLOCK)):
        v = x[:, lo:lo + BLOCK].double()
        scales[:, i], inv = _exact_scale(v.abs().amax(1), pow2)
        codes[:, lo:lo + v.shape[1]] = _grid((v * inv[:, None]).float().double())
    return codes, scales


def _exact_tokens(x, pow2, off, cap):
    R, C = x.shape
    codes = torch.zeros((C, BLOCK * cap), dtype=torch.float64, device=x.device)
    scales = torch.zeros((cap, C), dtype=torch.float64, device=x.device)
    b = 0
    for lo, hi in zip(off, off[1:]):
        for r in range(lo, hi, BLOCK):
            v = x[r:min(r + BLOCK, hi)].double()
            scales[b], inv = _exact_scale(v.abs().amax(0), pow2)
            codes[:, b * BLOCK:b * BLOCK + v.shape[0]] = _grid((v * inv).float().double()).t()
            b += 1
    return codes, scales


def _exact_weights_of_route(c, logits, bias, idx):
    l = torch.where(logits.isnan(), -math.inf, logits.double()).clamp(max=F32_MAX)
    live = idx >= 0
    z = l.gather(1, idx.long().clamp(min=0))
    if c["renorm"]:
        # weight_j = 1 / sum_i score_i / score_j, the quotients of the scores in log space
        v = z - torch.log1p(torch.exp(-z.abs())) - z.clamp(min=0) if c["score"] == "sigmoid" else z
        q = torch.where(live[:, None, :], torch.exp(v[:, None, :] - v[:, :, None]), 0.0).sum(-1)
        w = 1.0 / q
    elif c["score"] == "sigmoid":
        w = 1.0 / (1.0 + torch.exp(-z))
    else:
        w = torch.exp(z - torch.logsumexp(l, -1, keepdim=True))
    return torch.where(live, c["scale"] * w, 0.0)


def exact(case, seed):
    s = prepare(case, seed)
    c, out, kind = s["case"], s["out"], s["case"]["kind"]
    if kind == "route":
        w = _exact_weights_of_route(c, s["logits"], s["bias"], _plain_route(s)["topk_idx"])
        return {**dict.fromkeys(out), "topk_w": w}
    if kind == "route_grad":
        # the derivative of the weights' definition, by reverse differentiation in 64 bits
        l = s["logits"].double().requires_grad_()
        live = s["idx"] >= 0
        z = l.gather(1, s["idx"].long().clamp(min=0))
        p = torch.sigmoid(z) if c["score"] == "sigmoid" else torch.exp(
            z - l.detach().amax(-1, keepdim=True).clamp(min=-F32_MAX))
        if c["renorm"]:
            w = torch.where(live, p, 0.0)
            w = w / w.sum(-1, keepdim=True).clamp(min=1e-300)
        elif c["score"] == "softmax":
            w = p / torch.exp(l - l.detach().amax(-1, keepdim=True).clamp(min=-F32_MAX)).sum(
                -1, keepdim=True).clamp(min=1e-300)
        else:
            w = p
        (torch.where(live, w, 0.0) * (c["scale"] * s["dw"].double())).sum().backward()
        return {"dlogits": l.grad}
    if kind == "quantise":
        if c["what"] == "weights":
            q = torch.zeros(out["codes"].shape, dtype=torch.float64, device="cuda")
            sc = torch.zeros(out["scales"].shape, dtype=torch.float64, device="cuda")
            qt = torch.zeros(out["codes_t"].shape, dtype=torch.float64, device="cuda")
            for i in range(sc.shape[1]):
                for j in range(sc.shape[2]):
                    at = slice(i * BLOCK, (i + 1) * BLOCK), slice(j * BLOCK, min((j + 1) * BLOCK, c["C"]))
                    v = s["x"][:, at[0], at[1]].double()
                    sc[:, i, j], inv = _exact_scale(v.abs().amax((1, 2)), c["pow2"])
                    q[:, at[0], at[1]] = _grid((v * inv[:, None, None]).float().double())
            qt[:, :, :c["T"]] = q[:, :, :c["C"]].transpose(1, 2)
            return {"codes": q, "scales": sc, "codes_t": qt, "scales_t": sc.transpose(1, 2)}
        x = s["x"][s["src_tok"].long()] if c["what"] == "gather" else s["x"]
        r = {}
        if "codes" in out:
            r["codes"], r["scales"] = _exact_rows(x, c["pow2"], out["codes"].shape[1])
        if "codes_t" in out:
            r["codes_t"], r["scales_t"] = _exact_tokens(x, c["pow2"], s["offsets_host"],
                                                        out["scales_t"].shape[0])
        return r
    if kind == "swiglu":
        f = c["f"]
        a, b = s["ab"][:, :f].double(), s["ab"][:, f:].double()
        e = torch.exp(-a)
        h = (a * b / (1.0 + e)).to(torch.bfloat16)
        y = h
        if c["back"]:
            dh = s["dh"].double()
            da = dh * b * (1.0 + e + a * e) / (1.0 + e) ** 2
            y = torch.cat([da, dh * a / (1.0 + e)], 1).to(torch.bfloat16)
        r = dict(zip(("codes", "scales"), _exact_rows(y, c["pow2"], out["codes"].shape[1])))
        if c["tokens"]:
            cap = out["scales_t"].shape[0]
            r["codes_t"], r["scales_t"] = _exact_tokens(y, c["pow2"], s["offsets_host"], cap)
            if c["back"]:
                r["h_codes_t"], r["h_scales_t"] = _exact_tokens(h, c["pow2"], s["offsets_host"], cap)
        return r
    off, blk = s["offsets_host"], s["blocks_host"]
    if kind == "product":
        y = torch.zeros(out["out"].shape, dtype=torch.float64, device="cuda")
        for g in range(c["G"]):
            lo, hi = off[g], off[g + 1]
            for k, at in enumerate(range(0, c["K"] if hi > lo else 0, BLOCK)):
                to = min(at + BLOCK, c["K"])
                rows = s["b_scales"][g, :, k].double().repeat_interleave(BLOCK)[:c["N"]]
                d = s["a"][lo:hi, at:to].double() @ s["b"][g, :, at:to].double().t()
                y[lo:hi] += d * s["a_scales"][lo:hi, k].double()[:, None] * rows
        return {"out": y}
    y = torch.zeros(out["dw"].shape, dtype=torch.float64, device="cuda")
    for g in range(c["G"]):
        for k in range(blk[g], blk[g + 1]):
            at = slice(k * BLOCK, (k + 1) * BLOCK)
            d = s["a"][:, at].double() @ s["b"][:, at].double().t()
            y[g] += d * s["a_scales"][k].double()[:, None] * s["b_scales"][k].double()
    return {"dw": y}


if __name__ == "__main__":
    r = random.Random(0)
    for example in listed() + [draw(r) for _ in range(6)]:
        print(example, work(example))
