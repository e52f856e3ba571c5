/*
 * moe.h -- C ABI of the single-GPU Mixture-of-Experts layer for GB300 (sm_103a).
 *
 * The layer: top-k router gating, padding-free token dispatch (per-expert histogram,
 * exclusive scan, permute-gather into one contiguous expert-ordered buffer with no
 * per-expert padding, optional capacity dropping), a grouped SwiGLU expert FFN over
 * the ragged expert segments, and a weighted un-permute/combine, with the matching
 * backward.
 *
 * Where each operation is defined (page title, then section / figure / field):
 *   - "MoE Training Optimization with Primus" (AMD blog), Figure 7 dataflow: router
 *     top-k per token; a permutation into expert order; the grouped gate/up projection
 *     (FC1), SwiGLU and the grouped down projection (FC2); a last step that un-permutes
 *     the rows, scales them by the gate weights and sums each token's k of them.
 *     MegaMoE section: the backward mirrors dispatch and combine, and adds the two
 *     weight-gradient GEMMs whose K is each expert's row count.  JAX section: a single
 *     grouped-GEMM launch covers all expert groups, each of its own length; the token
 *     counts never leave the GPU (no host synchronisation).
 *   - X-MoE verdict page (pith.science, arXiv 2508.13337), "key machinery": the
 *     padding-free token buffer -- only the routed tokens, stored contiguously per
 *     expert, plus side arrays giving each row's source token, its expert, the rows per
 *     expert and the combine weight; referee minor comment on section 4.1.1 Listing 1:
 *     max_token_count and c = 1.25; major comment on section 5.6: an assignment is
 *     dropped only when its expert is over capacity.
 *
 * Conventions shared by every call
 *   - Every pointer argument is a DEVICE pointer owned by the caller, except the
 *     moe_config_t pointer and the size_t/int32_t out-parameters of the host-only
 *     helpers, which are host pointers.  The library never allocates or frees
 *     device memory.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Calls only
 *     enqueue work and never synchronise with the host (the token counts stay on
 *     the device), except moe_status(), which synchronises `stream`.
 *   - Arguments are validated on the host before anything is enqueued; an invalid
 *     call returns MOE_ERR_INVALID_ARG or MOE_ERR_UNSUPPORTED with nothing enqueued.
 *   - Anomalies seen on the device (a NaN logit, an out-of-range index in an input
 *     index array, inconsistent segment offsets, a pipeline wait that gave up) set
 *     bits in an error word at the start of `ws`; kernels never trap.  Read and
 *     clear it with moe_status().
 *   - Dtypes: logits fp32; activations, weights and their gradients bf16 (raw 16-bit
 *     patterns, `void*` here); gate weights and dlogits fp32; indices int32.
 *     Matrix products accumulate in fp32.
 *   - Layouts are row-major.  W1 is [E, 2f, d] (rows 0..f-1 gate, f..2f-1 up, i.e.
 *     nn.Linear (out, in)), W2 is [E, d, f]; the shared expert's W1s [2fs, d] and
 *     W2s [d, fs].  Every buffer indexed by an expert-ordered row ("xp", "ab", ...)
 *     is sized for T*k rows; the live row count is offsets[E] on the device.
 *   - Alignment: every device pointer 16-byte aligned.
 *   - Limits: 1 <= k <= 8, k <= E <= 256, 1 <= T, T*k < 2^31, d and f (and fs if
 *     non-zero) multiples of 64.  Anything else returns MOE_ERR_UNSUPPORTED.
 *   - Thread safety: calls on different streams with disjoint buffers may run
 *     concurrently; the library keeps no mutable state of its own between calls
 *     (the error word lives in the caller's `ws`) -- except the fixed scratch behind
 *     moe_route_noalloc, whose own comment says how it is shared.
 */
#ifndef MOE_GB300_H
#define MOE_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = 1,   /* null pointer, bad shape, k > E, ... (nothing enqueued) */
    MOE_ERR_UNSUPPORTED = 2,   /* valid but outside the limits above (nothing enqueued)  */
    MOE_ERR_CUDA = 3,          /* a CUDA runtime call failed                             */
    MOE_ERR_DEVICE_FLAG = 4,   /* moe_status(): a device-side anomaly was flagged        */
    MOE_ERR_TIMEOUT = 5        /* moe_status(): a device pipeline wait gave up           */
} moe_status_t;

typedef enum {
    MOE_GATE_SOFTMAX_TOPK = 0, /* w_j = exp(l_j) / sum_{i in top-k} exp(l_i)            */
    MOE_GATE_SIGMOID_TOPK = 1  /* w_j = route_scale * sigma(l_j) / sum_{i in top-k} sigma(l_i) */
} moe_gate_t;

/* Device error bits reported by moe_status() through *flags. */
#define MOE_DEVERR_NAN_LOGIT   0x1   /* a router logit was NaN (it ranks below -inf)      */
#define MOE_DEVERR_BAD_INDEX   0x2   /* an index array held an out-of-range entry        */
#define MOE_DEVERR_TIMEOUT     0x4   /* a GEMM pipeline wait exceeded its bound          */
#define MOE_DEVERR_BAD_OFFSETS 0x8   /* segment offsets not monotone or past capacity    */

typedef struct {
    int64_t T;            /* tokens                                                    */
    int32_t d;            /* model width                                               */
    int32_t E;            /* routed experts                                            */
    int32_t k;            /* experts per token                                         */
    int32_t ffn;          /* routed expert SwiGLU width f                              */
    int32_t ffn_shared;   /* shared (always-on) expert width fs; 0 = none              */
    int32_t gate;         /* moe_gate_t                                                */
    float route_scale;    /* 1.0 for softmax; the sigmoid gate's scale (e.g. 2.5)      */
    int32_t capacity;     /* per-expert capacity; 0 = unlimited                        */
    /* Routing variants and memory trade-off (zero-initialise for the plain layer): */
    const float *select_bias; /* [E] device fp32, or NULL: added (fp32) to the logits for the
                                 top-k choice only -- the gate weights use the raw logits
                                 (a DeepSeek-V3-style balancing bias)                     */
    int32_t drop_negative;    /* 1: an assignment whose raw logit is negative is dropped
                                 before the capacity ranking and is not counted (DeepSpeed-
                                 MoE's rule, X-MoE verdict page, major comment on 5.6)    */
    int32_t recompute;        /* 1: selective rematerialisation -- ctx keeps neither ab nor
                                 h (nor ab_s, h_s); moe_layer_bwd recomputes FC1 from the
                                 saved xp (MegaScale-MoE notes: selective activation
                                 rematerialisation).  Results are bit-identical.         */
    int32_t drop_by_score;    /* 1 (with capacity > 0): an expert over capacity keeps the
                                 assignments with the largest raw logit (ties: lower token)
                                 instead of the earliest tokens; kept rows stay in token
                                 order inside its segment.  Needs (E+1 + T*k)*4 more bytes
                                 of ws.                                                   */
    int32_t mxfp8;            /* 1: the routed experts' forward GEMMs run on MXFP8 operands
                                 (moe_layer_fwd_mx), and with moe_layer_bwd_mx the data-
                                 gradient GEMMs of the backward too; needs d and ffn
                                 multiples of 128 and more ws for the quantised
                                 activations.  The weight gradients stay bf16.
                                 2: as 1, and the weight gradients too: their operands
                                 (dyp, h, dab, xp) are quantised along each segment's
                                 tokens, in 32-row blocks from the segment's first row
                                 (the Primus MoE blog, FP8 section: permuted tokens padded
                                 to the quantisation block boundary); needs about
                                 (2d + 3ffn) * (T*k + 128*E) * 33/32 more bytes of ws.
                                 0, 1, 2 only.                                            */
} moe_config_t;

/* Index of each saved tensor inside the forward context `ctx` (see moe_ctx_offsets). */
typedef enum {
    MOE_CTX_TOPK_IDX = 0,  /* int32 [T,k]                                               */
    MOE_CTX_TOPK_W,        /* fp32  [T,k]                                               */
    MOE_CTX_COUNTS,        /* int32 [E]                                                 */
    MOE_CTX_KEPT,          /* int32 [E]                                                 */
    MOE_CTX_OFFSETS,       /* int32 [E+1]                                               */
    MOE_CTX_DEST_ROW,      /* int32 [T,k]  (-1 = dropped)                               */
    MOE_CTX_SRC_TOK,       /* int32 [T*k]                                               */
    MOE_CTX_SRC_SLOT,      /* int32 [T*k]                                               */
    MOE_CTX_DROP_MASK,     /* uint8 [T,k]                                               */
    MOE_CTX_XP,            /* bf16  [T*k, d]   permuted tokens                          */
    MOE_CTX_AB,            /* bf16  [T*k, 2f]  FC1 output [a | b] (pre-activation)      */
    MOE_CTX_H,             /* bf16  [T*k, f]   silu(a) * b                              */
    MOE_CTX_YP,            /* bf16  [T*k, d]   FC2 output                               */
    MOE_CTX_AB_S,          /* bf16  [T, 2fs]   shared expert FC1 output (fs > 0)        */
    MOE_CTX_H_S,           /* bf16  [T, fs]                                             */
    MOE_CTX_YS,            /* bf16  [T, d]     shared expert output                     */
    MOE_CTX_NFIELDS
} moe_ctx_field_t;

/* floor(c * T * k / E): the per-expert capacity (max_token_count) for factor c
 * (X-MoE verdict page, referee minor comment on section 4.1.1 Listing 1).
 * Host-only.  Returns 0 (unlimited) for c <= 0 and -1 for invalid T, k, E. */
int32_t moe_capacity_from_factor(int64_t T, int32_t k, int32_t E, double c);

/* Bytes of the workspace `ws` (scratch + error word; one block serves every call)
 * and of the forward context `ctx` (tensors saved for the backward).  Host-only;
 * both out-pointers may be NULL. */
moe_status_t moe_workspace_size(const moe_config_t *cfg, size_t *ws_bytes, size_t *ctx_bytes);

/* Bytes of a workspace for the calls of single stages alone (route, permute, grouped FFN, combine
 * and their gradients, the norms' and checkpoints' error word): the part of moe_workspace_size's that
 * holds no whole intermediates.  Not for moe_layer_fwd, moe_layer_bwd, their MXFP8 forms and
 * moe_grouped_ffn_bwd_mx.  Host-only. */
moe_status_t moe_stage_workspace_size(const moe_config_t *cfg, size_t *ws_bytes);

/* Byte offset of every saved tensor inside `ctx`; offsets[MOE_CTX_NFIELDS]. Host-only. */
moe_status_t moe_ctx_offsets(const moe_config_t *cfg, size_t *offsets);

/* Clear the error word at the start of `ws` (enqueued on `stream`).  Call once on a
 * freshly allocated workspace. */
moe_status_t moe_ws_init(void *ws, void *stream);

/*
 * F1 + F2: route.  Primus MoE blog, Figure 7 dataflow (router top-k); X-MoE verdict
 * page, key machinery (padding-free buffer side arrays), referee comments on section
 * 4.1.1 Listing 1 and section 5.6 (capacity, drop only on overflow).
 *   logits   [T,E] fp32 in.
 *   topk_idx [T,k] out: the k best experts per token, by logit descending, ties to
 *            the lower id, NaN below -inf.  topk_w [T,k] out: gate weights computed
 *            over all k before any drop.
 *   counts [E] (assignments routed to e that were not dropped for a negative score),
 *            kept [E] = min(counts, capacity), offsets [E+1] = exclusive scan of
 *            kept; dest_row [T,k] = offsets[e] + (rank of t among e's tokens by
 *            ascending t), or -1 if that rank >= capacity; src_tok [T*k] / src_slot
 *            [T*k] (= t*k+j) invert dest_row (-1 past offsets[E]); drop_mask [T,k].
 *   Every integer output is deterministic (no atomics decide an order).
 */
moe_status_t moe_route(const moe_config_t *cfg, const float *logits, int32_t *topk_idx,
                       float *topk_w, int32_t *counts, int32_t *kept, int32_t *offsets,
                       int32_t *dest_row, int32_t *src_tok, int32_t *src_slot,
                       uint8_t *drop_mask, void *ws, void *stream);

/* Size of the fixed device scratch behind moe_route_noalloc (per GPU). */
#define MOE_NOALLOC_ROUTE_SCRATCH_BYTES (1u << 20)

/*
 * moe_route_noalloc -- the routing step (same outputs, same kernels as moe_route) for
 * callers that cannot allocate device memory, so cannot provide `ws`.  There is no
 * counterpart of this entry point in the paper; it exists for deployment reasons.
 *
 * Who needs it: a plugin running inside a host framework that owns all device memory
 * through its own pool and does not allow other code to call cudaMalloc, or a
 * latency-critical caller that cannot accept the device-wide synchronisation that
 * cudaMalloc / cudaFree may cause.  This call allocates nothing: the routing histogram
 * lives in a fixed __device__ array of MOE_NOALLOC_ROUTE_SCRATCH_BYTES compiled into
 * the library, which every GPU that loads the library holds until the process exits.
 *
 *   Arguments as for moe_route, except that `ws` is replaced by dev_flags_or_null: an
 *   optional device int32 that receives the MOE_DEVERR_* bits (NaN logits); with NULL
 *   those flags are dropped.
 *   Limit: the routing scratch must fit in MOE_NOALLOC_ROUTE_SCRATCH_BYTES.  With
 *   up(n) = n rounded up to a multiple of 256, it takes
 *       up(ceil(T/32) * E * 4)                                  bytes, plus, only when
 *       drop_by_score is set with a capacity,  up((E+1) * 4) + up(T * k * 4)  bytes
 *   (each expert's base and one 32-bit word per assignment for the score ranking).
 *   Examples that fit: plain or token-order capacity routing up to T = 32768 with
 *   E = 256 (exactly 1 MiB); drop-by-score routing with T = 16384, E = 64, k = 6
 *   (128 KiB + 512 B + 384 KiB).  T = 32768, E = 256 with drop_by_score does not fit.
 *   Larger shapes return MOE_ERR_UNSUPPORTED with nothing enqueued.
 *   Set-up: the first call on each device looks up the array's device address
 *   (cudaGetSymbolAddress) with that device current; make that first call before any
 *   stream capture.  Only a successful lookup is remembered: if it fails (the call
 *   returns MOE_ERR_CUDA, nothing enqueued), the next call on that device tries again.
 *   Sharing: every call on a device uses the same array and leaves its contents behind
 *   (the kernels overwrite every entry they read, so nothing has to be cleared between
 *   calls); calls whose execution overlaps on the GPU -- e.g. on two streams without an
 *   ordering between them -- race on it and must be serialised by the caller.
 */
moe_status_t moe_route_noalloc(const moe_config_t *cfg, const float *logits, int32_t *topk_idx,
                               float *topk_w, int32_t *counts, int32_t *kept, int32_t *offsets,
                               int32_t *dest_row, int32_t *src_tok, int32_t *src_slot,
                               uint8_t *drop_mask, int32_t *dev_flags_or_null, void *stream);

/*
 * F3: permute-gather into expert order (Primus MoE blog, Figure 7, the permutation step
 * before FC1; X-MoE padding-free buffer).
 *   xp[p] = x[src_tok[p]] for p < offsets[E]; rows past offsets[E] are not written.
 *   x [T,d] bf16 in, xp [T*k,d] bf16 out.  A pure bit copy.
 */
moe_status_t moe_permute(const moe_config_t *cfg, const void *x, const int32_t *src_tok,
                         const int32_t *offsets, void *xp, void *ws, void *stream);

/*
 * F4 + F5: grouped SwiGLU expert FFN over the ragged segments given by offsets
 * (Primus MoE blog, Figure 7 FC1 / SwiGLU / FC2; JAX section: one launch over
 * ragged variable-M groups).  For every row p of expert e:
 *   [a | b] = xp[p] W1[e]^T  -> ab[p] (bf16, saved for the backward)
 *   h[p]    = silu(a) * b    (from the bf16 a, b; bf16)
 *   yp[p]   = h[p] W2[e]^T   (bf16)
 *   xp [T*k,d], ab [T*k,2f], h [T*k,f], yp [T*k,d]; only rows < offsets[E] written.
 */
moe_status_t moe_grouped_ffn(const moe_config_t *cfg, const void *xp, const int32_t *offsets,
                             const void *W1, const void *W2, void *ab, void *h, void *yp,
                             void *ws, void *stream);

/*
 * F3 + F4 + F5 fused: moe_grouped_ffn with the permute folded into FC1's operand loads
 * (Primus MoE blog, MegaMoE section: the dispatch fused into the FC1 grouped GEMM, here
 * on one GPU: tensor-memory-accelerator gathers of the token rows, no xp buffer).
 *   Row p of expert e is computed from x[src_tok[p]]; outputs as moe_grouped_ffn.
 *   x [T,d] bf16, src_tok [T*k] int32 (entries < offsets[E] must lie in [0,T); a bad one
 *   sets MOE_DEVERR_BAD_INDEX and row 0 is read instead).
 */
moe_status_t moe_grouped_ffn_gather(const moe_config_t *cfg, const void *x,
                                    const int32_t *src_tok, const int32_t *offsets,
                                    const void *W1, const void *W2, void *ab, void *h, void *yp,
                                    void *ws, void *stream);

/*
 * F7: combine = unpermute and scale (Primus MoE blog, Figure 7, last step).
 *   y[t] = sum_{j = 0..k-1, dest_row[t,j] >= 0} topk_w[t,j] * yp[dest_row[t,j]]
 *          (+ ys[t] if ys_or_null is not NULL), fp32 accumulation, bf16 out [T,d].
 */
moe_status_t moe_combine(const moe_config_t *cfg, const void *yp, const int32_t *dest_row,
                         const float *topk_w, const void *ys_or_null, void *y, void *ws,
                         void *stream);

/*
 * B1: backward of combine and of the gate (Primus MoE blog, MegaMoE section: the
 * dispatch of the upstream gradient dy).  For each kept slot (t,j) with row p = dest_row[t,j]:
 *   dyp[p] = bf16(topk_w[t,j] * dy[t]);  dw[t,j] = <dy[t], yp[p]> (0 if dropped)
 *   softmax gate: dlogits[t,e_j] = w_j (dw_j - sum_i w_i dw_i)
 *   sigmoid gate: S = sum_i s_i, s_i = sigma(l_i):
 *                 dlogits[t,e_j] = scale (dw_j / S - sum_i s_i dw_i / S^2) s_j (1 - s_j)
 *   dlogits [T,E] fp32 out, zero for unselected experts.  Both are evaluated in the
 *   equal pairwise form sum_i u_i (dw_j - dw_i) (u_i the normalised scores, summing to 1),
 *   which keeps its precision when one score carries almost all the weight.
 */
moe_status_t moe_combine_bwd(const moe_config_t *cfg, const void *dy, const void *yp,
                             const float *logits, const int32_t *topk_idx, const float *topk_w,
                             const int32_t *dest_row, void *dyp, float *dlogits, void *ws,
                             void *stream);

/*
 * B2..B5: backward of the grouped SwiGLU FFN (Primus MoE blog, MegaMoE section and
 * JAX section: data-gradient grouped GEMMs plus the two variable-K weight-gradient
 * grouped GEMMs).  For the rows of expert e (K of the weight gradients = the
 * segment's row count, which may be 0):
 *   dh = dyp W2[e];  da = dh * b * silu'(a);  db = dh * silu(a)  -> dab [T*k,2f] bf16
 *   dW2[e] = dyp_e^T h_e  [d,f] bf16;   dxp = dab W1[e]  [T*k,d] bf16;
 *   dW1[e] = dab_e^T xp_e [2f,d] bf16  (all fp32-accumulated).
 */
moe_status_t moe_grouped_ffn_bwd(const moe_config_t *cfg, const void *dyp, const void *xp,
                                 const int32_t *offsets, const void *W1, const void *W2,
                                 const void *ab, const void *h, void *dab, void *dxp, void *dW1,
                                 void *dW2, void *ws, void *stream);

/*
 * B2..B5 with the FC1 weight gradient gathering its operand from x: as
 * moe_grouped_ffn_bwd with xp[p] = x[src_tok[p]] read straight from x
 * (dW1[e] = dab_e^T x[src_tok]_e); no xp buffer exists.  Same index rules as
 * moe_grouped_ffn_gather.
 */
moe_status_t moe_grouped_ffn_bwd_gather(const moe_config_t *cfg, const void *dyp, const void *x,
                                        const int32_t *src_tok, const int32_t *offsets,
                                        const void *W1, const void *W2, const void *ab,
                                        const void *h, void *dab, void *dxp, void *dW1,
                                        void *dW2, void *ws, void *stream);

/*
 * B1's dispatch of dy fused into B2 (Primus MoE blog, MegaMoE section: the dispatch of the
 * upstream gradient folded into the FC2 data-gradient grouped GEMM).  As
 * moe_grouped_ffn_bwd, except that the FC2 data-gradient takes its rows straight from dy:
 * for row p of expert e, t = src_tok[p], s = src_slot[p],
 *   dh = topk_w[s] * (dy[t] W2[e])      (fp32: the gate weight is applied to the product
 *                                         in the GEMM's epilogue, so w * dy is never rounded
 *                                         to bf16 on this path)
 *   da, db from dh as in moe_grouped_ffn_bwd -> dab [T*k,2f] bf16
 * dy [T,d] bf16 and topk_w [T,k] fp32 as moe_combine_bwd takes them; src_tok / src_slot
 * [T*k] int32 from moe_route (entries < offsets[E] must lie in [0,T) and [0,T*k); a bad
 * one sets MOE_DEVERR_BAD_INDEX, row 0 of dy / a weight of 0 is used instead).
 * The FC2 weight gradient still contracts the rows dyp = bf16(w dy) that moe_combine_bwd
 * writes, so dyp is an input here; dxp, dW1 and dW2 are as in moe_grouped_ffn_bwd.
 */
moe_status_t moe_grouped_ffn_bwd_dispatch(const moe_config_t *cfg, const void *dy,
                                          const float *topk_w, const int32_t *src_tok,
                                          const int32_t *src_slot, const void *dyp,
                                          const void *xp, const int32_t *offsets,
                                          const void *W1, const void *W2, const void *ab,
                                          const void *h, void *dab, void *dxp, void *dW1,
                                          void *dW2, void *ws, void *stream);

/*
 * B6: un-permute reduce (Primus MoE blog, MegaMoE section: the reduction of each
 * token's rows after the FC1 data gradient).
 *   dx[t] = sum_{j kept} dxp[dest_row[t,j]] (+ dxs[t] if dxs_or_null), fp32 accumulation,
 *   gathered per token (deterministic, no atomics); bf16 [T,d] out.
 */
moe_status_t moe_unpermute_reduce(const moe_config_t *cfg, const void *dxp,
                                  const int32_t *dest_row, const void *dxs_or_null, void *dx,
                                  void *ws, void *stream);

/*
 * ---- MXFP8 forward of the routed experts (Primus MoE blog, FP8 section: the MXFP8 recipe
 * with OCP E4M3 elements for the expert grouped GEMMs, weight-quantisation caching;
 * MegaMoE section: the SwiGLU step quantises its own output).  MX rule (OCP Microscaling
 * formats v1.0): blocks of 32 consecutive elements along the contraction axis share the
 * scale 2^X, X = floor(log2(max |v|)) - 8 clamped to [-127, 127] (-127 for an all-zero
 * block), stored as the E8M0 code X + 127; elements are E4M3(v / 2^X), rounded to
 * nearest (ties to even) and saturated at +-448.  d and ffn must be multiples of 128.
 */

/* Bytes of the quantised-weight blob for cfg's routed experts, and the byte offsets of its
 * eight parts: offsets[0] W1 codes [E][2f][d] E4M3, offsets[1] W1 scales, offsets[2] W2
 * codes [E][d][f], offsets[3] W2 scales (the forward's, quantised along d and f);
 * offsets[4] W2^T codes [E][f][d] quantised along d, offsets[5] their scales, offsets[6]
 * W1^T codes [E][d][2f] quantised along 2f, offsets[7] their scales (the backward's data
 * gradients).  The transposes' scale atoms ((e*ceil(C/256) + nt)*(K/128) + kb)*2 + half
 * cover rows e*C + nt*256 + half*128 + m of the transpose (C = f or d rows per expert,
 * K = d or 2f).  The scales are stored in 512-byte atoms: atom
 * ((e*(f/128) + nb)*(d/128) + kb)*2 + half holds, at byte 16*(m%32) + 4*(m/32) + j, the
 * scale of W1 row e*2f + half*f + nb*128 + m, elements 32*(4*kb + j) .. +31; W2 atom
 * ((e*ceil(d/256) + nt)*(f/128) + kb)*2 + half covers W2 row e*d + nt*256 + half*128 + m.
 * Atom bytes of rows past an expert's end hold 127.  Host-only; offsets (8 entries) may be
 * NULL. */
moe_status_t moe_mx_weights_size(const moe_config_t *cfg, size_t *bytes, size_t *offsets);

/* Bytes of an activation scale array for contraction length K (d for x, ffn for h).
 * Activation scales are stored in 512-byte atoms tiled by 128 rows inside each expert
 * segment: for row p of expert e, local row l = p - offsets[e], m = l % 128, the scale of
 * elements 32*(4*kb + j) .. +31 sits in atom ((offsets[e] >> 7) + e + l/128) * (K/128) + kb
 * at byte 16*(m%32) + 4*(m/32) + j; bytes of rows past a segment's end are unspecified.
 * Size: ((T*k >> 7) + E + 1) * (K/128) * 512.  Host-only. */
moe_status_t moe_mx_act_scales_size(const moe_config_t *cfg, int32_t K, size_t *bytes);

/* Quantise W1 [E,2f,d] and W2 [E,d,f] (bf16) into the blob (device, 256-byte aligned,
 * moe_mx_weights_size bytes).  The caller keeps the blob while the weights are unchanged
 * (weight-quantisation caching). */
moe_status_t moe_mx_quantize_weights(const moe_config_t *cfg, const void *W1, const void *W2,
                                     void *wq, void *stream);

/* F3 with MXFP8 output: for p < offsets[E], xq[p] = E4M3 codes of x[src_tok[p]] ([T*k][d]
 * bytes) and its E8M0 scales into x_sf (activation atoms, moe_mx_act_scales_size(cfg, d)
 * bytes); with xp_or_null also the bf16 copy xp[p] = x[src_tok[p]] (the backward's saved
 * input). */
moe_status_t moe_mx_permute_quant(const moe_config_t *cfg, const void *x,
                                  const int32_t *src_tok, const int32_t *offsets,
                                  void *xp_or_null, void *xq, uint8_t *x_sf, void *ws,
                                  void *stream);

/* F4 + F5 on MXFP8 operands (block-scaled tensor-core MMAs, fp32 accumulation):
 *   [a|b] = bf16(deq(xq) deq(W1q[e])^T) -> ab;  h = bf16(silu(a) b) -> h;
 *   hq, h_sf = MX(h) along f (the SwiGLU epilogue quantises its bf16 output);
 *   yp = bf16(deq(hq) deq(W2q[e])^T).
 * Shapes as moe_grouped_ffn; hq [T*k][f] bytes; x_sf and h_sf are activation atoms
 * (moe_mx_act_scales_size with K = d and K = ffn). */
moe_status_t moe_grouped_ffn_mx(const moe_config_t *cfg, const void *xq, const uint8_t *x_sf,
                                const int32_t *offsets, const void *wq, void *ab, void *h,
                                uint8_t *hq, uint8_t *h_sf, void *yp, void *ws, void *stream);

/* Whole forward with the routed experts in MXFP8 (cfg->mxfp8 = 1): route -> permute and
 * quantise -> MXFP8 grouped FFN -> (bf16 shared expert) -> combine.  ctx receives the same
 * tensors as moe_layer_fwd (xp, ab, h, yp in bf16), so moe_layer_bwd runs unchanged; the
 * quantised activations live in ws.  wq: the blob of moe_mx_quantize_weights. */
moe_status_t moe_layer_fwd_mx(const moe_config_t *cfg, const float *logits, const void *x,
                              const void *wq, const void *W1s, const void *W2s, void *y,
                              void *ctx, void *ws, void *stream);

/* B2..B5 with the data-gradient GEMMs on MXFP8 operands (cfg->mxfp8 = 1 or 2): dyp is
 * quantised along d; dh = deq(MX(dyp)) deq(W2^T codes), the SwiGLU backward gives dab
 * (bf16 out) which is quantised along 2f; dxp = bf16(deq(MX(dab)) deq(W1^T codes)).  With
 * cfg->mxfp8 = 1 the weight gradients dW1, dW2 are computed from the bf16 xp, h, dyp and
 * dab as in moe_grouped_ffn_bwd; with 2, dW2[e] = bf16(deq(Q(dyp_e))^T deq(Q(h_e))) and
 * dW1[e] = bf16(deq(Q(dab_e))^T deq(Q(xp_e))), Q quantising each column of the segment's
 * rows in 32-row blocks from its first row (an expert without rows gets zeros).
 * wq: the blob of moe_mx_quantize_weights.  The quantised operands live in ws. */
moe_status_t moe_grouped_ffn_bwd_mx(const moe_config_t *cfg, const void *dyp, const void *xp,
                                    const int32_t *offsets, const void *wq, const void *ab,
                                    const void *h, void *dab, void *dxp, void *dW1, void *dW2,
                                    void *ws, void *stream);

/* Whole backward with the routed experts' data gradients in MXFP8 (cfg->mxfp8 = 1; with 2
 * their weight gradients too, as in moe_grouped_ffn_bwd_mx); as moe_layer_bwd otherwise
 * (the shared expert stays bf16). */
moe_status_t moe_layer_bwd_mx(const moe_config_t *cfg, const void *ctx, const float *logits,
                              const void *x, const void *dy, const void *wq, const void *W1s,
                              const void *W2s, void *dx, void *dW1, void *dW2, void *dW1s,
                              void *dW2s, float *dlogits, void *ws, void *stream);

/*
 * ---- Group-limited routing.  For token t with logits l (NaN counts as -inf and sets
 * MOE_DEVERR_NAN_LOGIT, +inf as the largest finite value):
 *   score s_e = sigma(l_e), or exp(l_e) / sum_i exp(l_i) over all E experts
 *   key   c_e = s_e + bias_e with a bias (the choice alone sees it), else l_e
 *   The E experts form `groups` runs of E / groups consecutive ones.  A group is worth its
 *   largest c (group_top = 1) or the sum of its two largest (2; of the scores s when there is
 *   no bias; of one alone if only one is in service); the top_groups worthiest stay.
 *   The k largest keys of the groups that stay are chosen, in descending order.  Every tie
 *   goes to the lower index; keys and worths that include scores are compared in 64 bits.
 *   weight w_j = route_scale * s_j (renorm = 0), or route_scale * s_j / sum of the chosen s
 *   (renorm = 1; the quotient's limit where all of them underflow).
 * An expert whose logit is -inf is out of service for that token and never chosen.  A slot
 * for which nothing is left (a padding token: all its logits -inf) gets expert -1, weight 0
 * and dest_row -1, and takes no row.
 */
typedef enum {
    MOE_SCORE_SOFTMAX = 0,
    MOE_SCORE_SIGMOID = 1
} moe_score_t;

typedef struct {
    int32_t score;        /* moe_score_t                                                  */
    int32_t groups;       /* 1 <= groups <= 32, divides E; 1 = no groups                  */
    int32_t top_groups;   /* 1 <= top_groups <= groups, top_groups * (E / groups) >= k    */
    int32_t group_top;    /* 1 or 2 (2 needs groups of at least two experts)              */
    int32_t renorm;       /* 0 or 1                                                       */
    const float *bias;    /* [E] device fp32, finite, or NULL                             */
} moe_router_t;

/*
 * Route with `router`.  cfg gives T, E, k, route_scale and capacity (dropping by token order);
 * its gate is not used, and select_bias, drop_negative and drop_by_score must be unset
 * (MOE_ERR_INVALID_ARG).  Outputs, workspace and determinism as moe_route, except for slots
 * without an expert as described above; those are marked in drop_mask too.
 */
moe_status_t moe_route_groups(const moe_config_t *cfg, const moe_router_t *router,
                              const float *logits, int32_t *topk_idx, float *topk_w,
                              int32_t *counts, int32_t *kept, int32_t *offsets,
                              int32_t *dest_row, int32_t *src_tok, int32_t *src_slot,
                              uint8_t *drop_mask, void *ws, void *stream);

/*
 * Gradient of moe_route_groups' weights: dlogits [T,E] fp32 from dw [T,k] fp32, the gradient of
 * topk_w.  The choice is piecewise constant: with renorm, or sigmoid scores, only the chosen
 * experts' logits have a gradient; softmax scores without renorm reach every expert.  Slots
 * with topk_idx -1 are ignored; another index outside [0, E) sets MOE_DEVERR_BAD_INDEX and is
 * ignored too.
 */
moe_status_t moe_route_groups_bwd(const moe_config_t *cfg, const moe_router_t *router,
                                  const float *logits, const int32_t *topk_idx, const float *dw,
                                  float *dlogits, void *ws, void *stream);

/*
 * The combine's backward for a gate whose own backward is a separate call:
 *   dyp[p] = bf16(topk_w[t,j] * dy[t]), dw[t,j] = <dy[t], yp[p]> with p = dest_row[t,j]; dw is 0
 *   where dest_row is -1.  dw [T,k] fp32.
 */
moe_status_t moe_combine_bwd_dw(const moe_config_t *cfg, const void *dy, const void *yp,
                                const float *topk_w, const int32_t *dest_row, void *dyp,
                                float *dw, void *ws, void *stream);

/*
 * ---- 8-bit operands with one scale for each block of 128.
 * A block is 128 consecutive elements along the product's contraction axis (the last one of a
 * row may be shorter), or 128 x 128 elements of a weight.  With amax the block's largest
 * magnitude, held at or above 2^-110:
 *   scale  s = amax / 448, or (pow2) the smallest power of two >= amax / 448;   fp32
 *   code   E4M3(v * (448 / amax)), or E4M3(v / s) with pow2; nearest, ties to even,
 *          saturated at 448; quotients and products are single fp32 roundings
 * so that v is close to code * s.  A NaN makes its block NaN; an infinity has an infinite scale
 * (pow2 or not), its own code is NaN and the others' are 0.
 *
 * Along the row:    codes [rows][ld] bytes, scales [rows][ceil(C/128)].
 * Along the tokens: for a weight gradient, whose contraction runs over an expert's rows.  Each
 *   segment's rows form blocks of 128 from its first row; the segments' blocks follow one
 *   another, B = moe_fp8_token_blocks(rows, G) bounds their number.  codes_t [C][128 B]: column
 *   c of block i at codes_t[c][128 i ..], zero codes past the segment's end; scales_t [B][C].
 *   Blocks past the last segment's are not written.
 * ld is a multiple of 16 and at least the row's length; what lies past it may be written with
 * zeros and is never read.  offsets [G+1] (device) delimit the segments as in moe_route;
 * NULL with G = 1: one segment of `rows` rows.  G <= 256, C, N, K < 2^24, rows < 2^31 - 2^15.
 * `ws` is any workspace initialised by moe_ws_init (MOE_FP8_WS_BYTES suffice): it holds the
 * error word.
 */
#define MOE_FP8_WS_BYTES 256

/* ceil(rows / 128) + G: the number of token blocks to provide for.  -1 for invalid arguments.
 * Host-only. */
int64_t moe_fp8_token_blocks(int64_t rows, int32_t G);

typedef struct {
    int64_t rows;         /* rows of the outputs (offsets[G] <= rows of them live); >= 0  */
    int64_t src_rows;     /* rows of x when src_tok is given                              */
    int32_t G;            /* segments                                                     */
    int32_t C;            /* columns                                                      */
    int64_t ldx;          /* elements between rows of x, >= C                             */
    int64_t ld;           /* bytes between rows of codes                                  */
    int32_t pow2;         /* 0 or 1                                                       */
} moe_fp8_quant_t;

/*
 * Quantise bf16 rows: row p is x[p], or x[src_tok[p]] (entries outside [0, src_rows) set
 * MOE_DEVERR_BAD_INDEX; such a row is not written by the row form and read as row 0 by the
 * token form).  codes and scales, codes_t and scales_t, or all four are given; either pair may
 * be NULL.
 */
moe_status_t moe_fp8_quantize(const moe_fp8_quant_t *q, const void *x,
                              const int32_t *src_tok_or_null, const int32_t *offsets_or_null,
                              void *codes, float *scales, void *codes_t, float *scales_t, void *ws,
                              void *stream);

/*
 * Quantise weights W [G][N][K] bf16 in 128 x 128 blocks: codes [G][N][ld], scales
 * [G][ceil(N/128)][ceil(K/128)]; with codes_t also the transposes codes_t [G][K][ld_t] (the
 * same codes) and scales_t [G][ceil(K/128)][ceil(N/128)], the operand of the data gradient.
 */
moe_status_t moe_fp8_quantize_weights(const void *W, int32_t G, int32_t N, int32_t K, void *codes,
                                      int64_t ld, float *scales, void *codes_t_or_null,
                                      int64_t ld_t, float *scales_t_or_null, int32_t pow2,
                                      void *stream);

typedef struct {
    int64_t rows;
    int32_t G;
    int32_t f;            /* SwiGLU width; ab is [rows][2f] bf16, dense                   */
    int64_t ld;           /* bytes between rows of codes                                  */
    int32_t pow2;
} moe_fp8_act_t;

/* SwiGLU with quantised output: h = silu(a) * b of ab = [a | b], rounded to bf16 once from its
 * exact value, quantised as moe_fp8_quantize does with C = f (codes, scales and, or, codes_t,
 * scales_t). */
moe_status_t moe_fp8_swiglu(const moe_fp8_act_t *p, const void *ab, const int32_t *offsets_or_null,
                            void *codes, float *scales, void *codes_t, float *scales_t, void *ws,
                            void *stream);

/* Its backward from dh [rows][f] bf16: da = dh b silu'(a), db = dh silu(a), each rounded to bf16
 * once, [da | db] quantised with C = 2f; with h_codes_t, h_scales_t also h along the tokens
 * (C = f), recomputed from ab.  codes and scales are required; codes_t, scales_t and h_codes_t,
 * h_scales_t are optional pairs (the latter only with the former). */
moe_status_t moe_fp8_swiglu_bwd(const moe_fp8_act_t *p, const void *dh, const void *ab,
                                const int32_t *offsets_or_null, void *codes, float *scales,
                                void *codes_t, float *scales_t, void *h_codes_t,
                                float *h_scales_t, void *ws, void *stream);

typedef enum { MOE_OUT_BF16 = 0, MOE_OUT_FP32 = 1 } moe_out_t;

typedef struct {
    int64_t rows;         /* rows of a and out                                            */
    int32_t G, N, K;
    int64_t lda, ldb;     /* bytes between rows of a and b, multiples of 16, >= K         */
    int64_t ldo;          /* elements between rows of out, >= N                           */
    int32_t out_type;     /* moe_out_t                                                    */
} moe_fp8_gemm_t;

/*
 * Grouped product: for the rows p of segment g, out[p][n] = sum_k A[p][k] B[g][n][k] over the
 * values (codes times scales); a [rows][lda] with scales along the row, b [G][N][ldb] with
 * weight block scales.  Products over a block accumulate in the tensor core's fp32, blocks are
 * scaled and summed in fp32, one rounding to the output type.  Rows past offsets[G] are not
 * written.  The data gradient is the same call on the transposed weights.
 */
moe_status_t moe_fp8_gemm(const moe_fp8_gemm_t *g, const void *a, const float *a_scales,
                          const void *b, const float *b_scales, const int32_t *offsets_or_null,
                          void *out, void *ws, void *stream);

typedef struct {
    int64_t rows;
    int32_t G, M, N;
    int32_t out_type;
} moe_fp8_wgrad_t;

/*
 * Weight gradient: dW[g][m][n] = sum over the rows p of segment g of A[p][m] B[p][n], from
 * along-token operands a [M][128 B] and b [N][128 B] with their scales (the same segments in
 * both); zeros for an empty segment.  dW [G][M][N] dense, every element written.
 */
moe_status_t moe_fp8_wgrad(const moe_fp8_wgrad_t *g, const void *a, const float *a_scales,
                           const void *b, const float *b_scales, const int32_t *offsets_or_null,
                           void *dW, void *ws, void *stream);

/*
 * ---- Normalisation of rows, and activations held in 8 bits for the backward pass.
 *
 * Checkpoint of rows: codes [rows][ld] bytes and fp32 scales [rows][ceil(C/128)], one for each
 * block of 128 along the row (the last one may be shorter).  With amax the block's largest
 * magnitude, held at or above 2^-110:
 *   MOE_CKPT_INT8  scale amax / 127, code = the whole number nearest to v * (127 / amax), ties to
 *                  even, the product rounded once: a value is off by at most half a scale (and the
 *                  largest fp32 number itself may be restored as infinity)
 *   MOE_CKPT_E4M3  scale and code as moe_fp8_quantize's along the row (pow2 = 0), so that the row
 *                  codes of a product's operand are its checkpoint
 * with quotients correctly rounded in fp32.  A value is restored as code * scale in fp32, and
 * rounded once more where it is stored as bf16; where a mean is taken from it, code * scale - mean is
 * rounded once.  A block that holds a NaN or an infinity restores
 * as NaN throughout.  ld is a multiple of 16 and at least C; nothing is written past C, and
 * what lies there does not count.
 *
 * `live` (device, one int32, 4-byte aligned; NULL: all rows): the number of rows that hold
 * something, &offsets[E] for the rows of the expert segments.  Rows behind it are neither read nor
 * written.  A number outside [0, rows] is held to that range and sets MOE_DEVERR_BAD_OFFSETS.
 * rows < 2^31 - 2^15, C < 2^24.  `ws` as for the 8-bit operands: it holds the error word.
 */
typedef enum { MOE_CKPT_INT8 = 0, MOE_CKPT_E4M3 = 1 } moe_ckpt_t;
typedef enum { MOE_NORM_LAYER = 0, MOE_NORM_RMS = 1 } moe_norm_kind_t;

typedef struct {
    int64_t rows;
    int32_t C;            /* columns                                                      */
    int32_t kind;         /* moe_norm_kind_t                                              */
    float eps;            /* finite, >= 0; forward only                                   */
    int32_t x_type;       /* moe_out_t of x, residual and total; of add and dx            */
    int32_t y_type;       /* of y; of dy                                                  */
    int32_t p_type;       /* of gamma and beta                                            */
    int32_t g_type;       /* of dgamma and dbeta                                          */
    int32_t format;       /* moe_ckpt_t                                                   */
    int64_t ldx;          /* elements between rows of x, >= C                             */
    int64_t ld_add;       /* of residual; of add                                          */
    int64_t ld_y;         /* of y; of dy                                                  */
    int64_t ld_out;       /* of total; of dx                                              */
    int64_t ld_codes;     /* bytes between rows of codes                                  */
} moe_norm_t;

/*
 * Normalise rows.  v = x, or x + residual (summed in fp32, rounded to x_type); m = mean of v, 0
 * with MOE_NORM_RMS; rstd = 1 / sqrt(mean of (v - m)^2 + eps):
 *   y = (v - m) * rstd * gamma + beta        (gamma or beta NULL: 1 or 0; fp32, rounded once)
 *   total = v (only with residual), mean = m [rows] (not with MOE_NORM_RMS), rstd [rows], and the
 *   checkpoint of v (codes, scales); each of these may be NULL.
 * Statistics are fp32: squares of magnitudes above 2^63 overflow.  A constant row has no answer with
 * eps = 0: NaN where the sum of its values is exact, else what the sum's rounding leaves.  Rows of x,
 * residual, y and total may be strided and need only their elements' alignment (off 16 bytes, or with
 * a width off 8, accesses are narrower); gamma, beta, mean, rstd, codes and scales are dense and start
 * at 16 bytes, as pointers do elsewhere.  total may be x or residual itself, and so may y if it is of
 * their type and has their distance.
 */
moe_status_t moe_norm(const moe_norm_t *p, const void *x, const void *residual_or_null,
                      const void *gamma_or_null, const void *beta_or_null, void *y,
                      void *total_or_null, float *mean_or_null, float *rstd_or_null,
                      void *codes_or_null, float *scales_or_null, void *stream);

/* Bytes of moe_norm_bwd's ws: the error word and the partial sums over the rows.  -1 for invalid
 * or unsupported sizes.  Host-only. */
int64_t moe_norm_ws_size(int64_t rows, int32_t C);

/*
 * Gradient of moe_norm.  With xhat = (v - mean) * rstd and G = dy * gamma:
 *   dx = rstd * (G - mean(G) - xhat * mean(G * xhat)) + add      (no mean(G) with MOE_NORM_RMS)
 *   dgamma = sum over the rows of dy * xhat, dbeta = sum over the rows of dy
 * v: rows of x_type at x, or with x_scales their checkpoint, whose codes are at x (ld_codes).  mean
 * and rstd are moe_norm's, of v itself; mean is NULL with MOE_NORM_RMS.  dx is the gradient of x
 * and of residual alike; add (NULL: none) is the gradient that reaches v by another way, the
 * stream's own.  dgamma and dbeta may be NULL; with rows = 0 they are zeros.  Sums over the rows
 * are fp32, in an order that rows, C, the types, the alignment and the device decide: the same bits
 * every time.  dx may be add itself, or dy if that is of its type and has its distance.  ws:
 * moe_norm_ws_size bytes, whose contents need not be kept: the calls of a stream may share it.
 */
moe_status_t moe_norm_bwd(const moe_norm_t *p, const void *dy, const void *x,
                          const float *x_scales_or_null, const float *mean, const float *rstd,
                          const void *gamma_or_null, const void *add_or_null, void *dx,
                          void *dgamma_or_null, void *dbeta_or_null, void *ws, void *stream);

/* y of moe_norm again, from the checkpoint of v and v's statistics. */
moe_status_t moe_ckpt_norm(const moe_norm_t *p, const void *codes, const float *scales,
                           const float *mean, const float *rstd, const void *gamma_or_null,
                           const void *beta_or_null, void *y, void *stream);

typedef struct {
    int64_t rows;
    int32_t C;            /* columns; [a | b]: 2f                                         */
    int32_t format;       /* moe_ckpt_t                                                   */
    int32_t x_type;       /* moe_out_t of x (SwiGLU: not used)                            */
    int64_t ldx;          /* elements between rows of x, >= C (SwiGLU: not used)          */
    int64_t ld;           /* bytes between rows of codes                                  */
} moe_ckpt_rows_t;

/* Rows x into their checkpoint, and back. */
moe_status_t moe_ckpt_save(const moe_ckpt_rows_t *p, const void *x, const int32_t *live_or_null,
                           void *codes, float *scales, void *ws, void *stream);
moe_status_t moe_ckpt_load(const moe_ckpt_rows_t *p, const void *codes, const float *scales,
                           const int32_t *live_or_null, void *x, void *ws, void *stream);

/* From the checkpoint of [a | b] (C = 2f): ab [rows][2f] bf16 and h = silu(a) * b [rows][f] bf16,
 * h from the fp32 values that the codes stand for.  Either may be NULL.  ab and h are what
 * moe_grouped_ffn_bwd and its variants read. */
moe_status_t moe_ckpt_swiglu(const moe_ckpt_rows_t *p, const void *codes, const float *scales,
                             const int32_t *live_or_null, void *ab_or_null, void *h_or_null,
                             void *ws, void *stream);

/* Backward of h = silu(a) * b from dh [rows][f] bf16 and the checkpoint of [a | b]:
 * da = dh b silu'(a), db = dh silu(a) -> dab [rows][2f] bf16, and h (NULL: not wanted). */
moe_status_t moe_ckpt_swiglu_bwd(const moe_ckpt_rows_t *p, const void *dh, const void *codes,
                                 const float *scales, const int32_t *live_or_null, void *dab,
                                 void *h_or_null, void *ws, void *stream);

/* moe_combine_bwd_dw with yp [T*k][d] from its checkpoint. */
moe_status_t moe_ckpt_combine_bwd(const moe_config_t *cfg, const void *dy, const void *codes,
                                  int64_t ld, const float *scales, int32_t format,
                                  const float *topk_w, const int32_t *dest_row, void *dyp,
                                  float *dw, void *ws, void *stream);

/*
 * Whole forward: route -> permute -> grouped FFN -> (shared expert) -> combine.
 *   logits [T,E] fp32, x [T,d], W1, W2 (W1s, W2s if ffn_shared > 0, else may be NULL)
 *   y [T,d] out.  ctx (moe_workspace_size bytes) receives the saved tensors listed in
 *   moe_ctx_field_t; ws is scratch.  No host synchronisation.
 */
moe_status_t moe_layer_fwd(const moe_config_t *cfg, const float *logits, const void *x,
                           const void *W1, const void *W2, const void *W1s, const void *W2s,
                           void *y, void *ctx, void *ws, void *stream);

/*
 * Whole backward from the forward's ctx and the upstream gradient dy [T,d]:
 *   dx [T,d], dW1 [E,2f,d], dW2 [E,d,f] (dW1s, dW2s if ffn_shared > 0), dlogits [T,E].
 *   x and logits are the forward's inputs (not copied into ctx).
 */
moe_status_t moe_layer_bwd(const moe_config_t *cfg, const void *ctx, const float *logits,
                           const void *x, const void *dy, const void *W1, const void *W2,
                           const void *W1s, const void *W2s, void *dx, void *dW1, void *dW2,
                           void *dW1s, void *dW2s, float *dlogits, void *ws, void *stream);

/*
 * Diagnostics: exercises the device-side failure path without a GPU fault.  Enqueues one
 * small kernel that waits on an mbarrier nothing will ever complete, with the same bounded
 * wait the grouped GEMM uses, limited to `budget_cycles` SM clock cycles (clamped to
 * 2e9, about one second).  When the wait gives up it sets MOE_DEVERR_TIMEOUT in the error
 * word of `ws` and returns normally, so moe_status() then reports MOE_ERR_TIMEOUT and
 * the context stays usable.  (Not part of the layer; there is no counterpart on the
 * pages.)
 */
moe_status_t moe_selftest_wait_timeout(void *ws, int64_t budget_cycles, void *stream);

/*
 * Diagnostics: the SM clock the grouped GEMMs' mainloops ran at.  Under the power cap the
 * clock that sampling tools report between samples can differ from the one the tensor-core
 * loops see, which decides the peak their throughput is measured against.  While tracing
 * is on, the MMA-issuing warp of every bf16 and MXFP8 grouped-GEMM CTA (the leader of a
 * CTA pair) adds, once per launch, the SM cycles (clock64) and the nanoseconds
 * (%globaltimer) of its tile loop to device-side sums; cycles / ns is that loop's clock.
 * The cost is a flag load and two timer reads per CTA and launch, plus three atomics per
 * CTA and launch while on.  (Not part of the layer; there is no counterpart on the pages.)
 *
 * moe_gemm_clock_trace(1) zeroes the sums and turns tracing on; moe_gemm_clock_trace(0)
 * turns it off and keeps them.  moe_gemm_clock_read() returns the sums: *cycles and *ns
 * over *loops loops (NULL pointers: MOE_ERR_INVALID_ARG).  Both are synchronous host
 * calls on the current device, ordered with the legacy default stream only: call them
 * with no grouped GEMM in flight (after a device or stream synchronisation).  Tracing
 * state is per device and shared by every caller in the process.
 */
moe_status_t moe_gemm_clock_trace(int enable);
moe_status_t moe_gemm_clock_read(uint64_t *cycles, uint64_t *ns, uint64_t *loops);

/* Synchronise `stream`, then read and clear the device error word in `ws`.
 * Returns MOE_OK, MOE_ERR_DEVICE_FLAG or MOE_ERR_TIMEOUT (MOE_DEVERR_TIMEOUT set),
 * or MOE_ERR_CUDA; *flags (may be NULL) receives the MOE_DEVERR_* bits. */
moe_status_t moe_status(void *ws, void *stream, int32_t *flags);

/* Human-readable name of a status code.  Host-only; never NULL. */
const char *moe_status_string(moe_status_t s);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GB300_H */
