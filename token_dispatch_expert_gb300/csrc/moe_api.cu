// moe_api.cu -- the C ABI declared in include/moe.h: host-side validation, the layout of
// the caller-owned workspace and forward context, and the order in which the layer's
// kernels are enqueued.  Nothing here allocates device memory or waits for the device
// (except moe_status).
#include <cmath>
#include <cstring>

#include "common.cuh"
#include "internal.h"
#include "rows8.cuh"

using namespace moe;

namespace {

constexpr size_t ALIGN = 256;

size_t align_up(size_t x) { return (x + ALIGN - 1) / ALIGN * ALIGN; }

moe_status_t validate(const moe_config_t* c) {
  if (!c) return MOE_ERR_INVALID_ARG;
  if (c->T <= 0 || c->E <= 0 || c->k <= 0 || c->k > c->E || c->d <= 0 || c->ffn <= 0 ||
      c->ffn_shared < 0 || c->capacity < 0)
    return MOE_ERR_INVALID_ARG;
  if (c->gate != MOE_GATE_SOFTMAX_TOPK && c->gate != MOE_GATE_SIGMOID_TOPK)
    return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(c->route_scale)) return MOE_ERR_INVALID_ARG;
  if ((c->drop_negative != 0 && c->drop_negative != 1) ||
      (c->recompute != 0 && c->recompute != 1) ||
      (c->drop_by_score != 0 && c->drop_by_score != 1) || (c->mxfp8 < 0 || c->mxfp8 > 2))
    return MOE_ERR_INVALID_ARG;
  if (c->select_bias && (reinterpret_cast<uintptr_t>(c->select_bias) & 3u))
    return MOE_ERR_INVALID_ARG;
  if (c->E > 256 || c->k > 8) return MOE_ERR_UNSUPPORTED;
  if (c->d % 64 || c->ffn % 64 || c->ffn_shared % 64) return MOE_ERR_UNSUPPORTED;
  // MXFP8: K blocks of 128 elements; the backward's FC1 rerun would be bf16, not MXFP8
  if (c->mxfp8 && (c->d % 128 || c->ffn % 128 || c->recompute)) return MOE_ERR_UNSUPPORTED;
  if (c->T * static_cast<int64_t>(c->k) >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;
  // 2f rows x d of one expert must be addressable with int32 tile coordinates
  if (static_cast<int64_t>(c->E) * 2 * c->ffn >= (int64_t(1) << 31) ||
      static_cast<int64_t>(c->E) * c->d >= (int64_t(1) << 31))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// every pointer must be non-null and 16-byte aligned
template <typename... P>
bool ptrs_ok(P... ps) {
  const void* arr[] = {static_cast<const void*>(ps)...};
  for (const void* p : arr)
    if (!p || !aligned16(p)) return false;
  return true;
}

struct CtxLayout {
  size_t off[MOE_CTX_NFIELDS];
  size_t total;
};

CtxLayout ctx_layout(const moe_config_t* c) {
  const size_t T = static_cast<size_t>(c->T), k = c->k, E = c->E, d = c->d, f = c->ffn,
               fs = c->ffn_shared;
  const size_t R = T * k;
  size_t sz[MOE_CTX_NFIELDS];
  sz[MOE_CTX_TOPK_IDX] = R * 4;
  sz[MOE_CTX_TOPK_W] = R * 4;
  sz[MOE_CTX_COUNTS] = E * 4;
  sz[MOE_CTX_KEPT] = E * 4;
  sz[MOE_CTX_OFFSETS] = (E + 1) * 4;
  sz[MOE_CTX_DEST_ROW] = R * 4;
  sz[MOE_CTX_SRC_TOK] = R * 4;
  sz[MOE_CTX_SRC_SLOT] = R * 4;
  sz[MOE_CTX_DROP_MASK] = R;
  sz[MOE_CTX_XP] = R * d * 2;
  const bool keep_act = !c->recompute;   // with recompute, FC1's outputs live in ws
  sz[MOE_CTX_AB] = keep_act ? R * 2 * f * 2 : 0;
  sz[MOE_CTX_H] = keep_act ? R * f * 2 : 0;
  sz[MOE_CTX_YP] = R * d * 2;
  sz[MOE_CTX_AB_S] = keep_act ? T * 2 * fs * 2 : 0;
  sz[MOE_CTX_H_S] = keep_act ? T * fs * 2 : 0;
  sz[MOE_CTX_YS] = fs ? T * d * 2 : 0;
  CtxLayout L;
  size_t o = 0;
  for (int i = 0; i < MOE_CTX_NFIELDS; ++i) {
    L.off[i] = o;
    o += align_up(sz[i]);
  }
  L.total = o;
  return L;
}

struct WsLayout {
  size_t route, maps, dyp, dab, dxp, dab_s, dx_s, ab, h, ab_s, h_s, xq, x_sf, hq, h_sf, dyq,
      dy_sf, dabq, dab_sf, dyT, dyT_sf, hT, hT_sf, dabT, dabT_sf, xpT, xpT_sf, total;
};

WsLayout ws_layout(const moe_config_t* c) {
  const size_t T = static_cast<size_t>(c->T), k = c->k, d = c->d, f = c->ffn,
               fs = c->ffn_shared;
  const size_t R = T * k;
  WsLayout L;
  size_t o = WS_HEADER_BYTES;
  L.route = o; o += align_up(route_scratch_bytes(c));
  L.maps = o;  o += align_up(2 * static_cast<size_t>(c->E) * SEG_MAP_BYTES);
  // (moe_stage_workspace_size ends here: what follows is the whole layer's alone)
  L.dyp = o;   o += align_up(R * d * 2);
  L.dab = o;   o += align_up(R * 2 * f * 2);
  L.dxp = o;   o += align_up(R * d * 2);
  L.dab_s = o; o += align_up(T * 2 * fs * 2);
  L.dx_s = o;  o += align_up(fs ? T * d * 2 : 0);
  // selective rematerialisation: FC1's outputs are scratch, recomputed by the backward
  const bool rc = c->recompute != 0;
  L.ab = o;    o += align_up(rc ? R * 2 * f * 2 : 0);
  L.h = o;     o += align_up(rc ? R * f * 2 : 0);
  L.ab_s = o;  o += align_up(rc ? T * 2 * fs * 2 : 0);
  L.h_s = o;   o += align_up(rc ? T * fs * 2 : 0);
  // MXFP8 forward: the quantised activations and their scales
  const bool mx = c->mxfp8 != 0;
  L.xq = o;    o += align_up(mx ? R * d : 0);
  L.x_sf = o;  o += align_up(mx ? mx_act_scale_bytes(c->T * c->k, c->E, c->d) : 0);
  L.hq = o;    o += align_up(mx ? R * f : 0);
  L.h_sf = o;  o += align_up(mx ? mx_act_scale_bytes(c->T * c->k, c->E, c->ffn) : 0);
  // ... and the backward's: dyp and dab in MXFP8
  L.dyq = o;   o += align_up(mx ? R * d : 0);
  L.dy_sf = o; o += align_up(mx ? mx_act_scale_bytes(c->T * c->k, c->E, c->d) : 0);
  L.dabq = o;  o += align_up(mx ? R * 2 * f : 0);
  L.dab_sf = o; o += align_up(mx ? mx_act_scale_bytes(c->T * c->k, c->E, 2 * c->ffn) : 0);
  // ... and with mxfp8 = 2 the weight gradients' operands, quantised along the tokens:
  // dW2 = dyp^T h (dyp the M operand, h the N operand), dW1 = dab^T xp
  const bool mw = c->mxfp8 == 2;
  const int64_t Rc = c->T * c->k;
  const int E = c->E, D = c->d, F = c->ffn;
  L.dyT = o;     o += align_up(mw ? mx_tok_codes_bytes(Rc, E, D) : 0);
  L.dyT_sf = o;  o += align_up(mw ? mx_tok_scale_bytes(Rc, E, D, false) : 0);
  L.hT = o;      o += align_up(mw ? mx_tok_codes_bytes(Rc, E, F) : 0);
  L.hT_sf = o;   o += align_up(mw ? mx_tok_scale_bytes(Rc, E, F, true) : 0);
  L.dabT = o;    o += align_up(mw ? mx_tok_codes_bytes(Rc, E, 2 * F) : 0);
  L.dabT_sf = o; o += align_up(mw ? mx_tok_scale_bytes(Rc, E, 2 * F, false) : 0);
  L.xpT = o;     o += align_up(mw ? mx_tok_codes_bytes(Rc, E, D) : 0);
  L.xpT_sf = o;  o += align_up(mw ? mx_tok_scale_bytes(Rc, E, D, true) : 0);
  L.total = o;
  return L;
}

template <typename T>
T* at(void* base, size_t off) {
  return reinterpret_cast<T*>(static_cast<uint8_t*>(base) + off);
}
template <typename T>
const T* at(const void* base, size_t off) {
  return reinterpret_cast<const T*>(static_cast<const uint8_t*>(base) + off);
}

moe_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

#define MOE_TRY(expr)                                        \
  do {                                                       \
    cudaError_t e_ = (expr);                                 \
    if (e_ != cudaSuccess) return MOE_ERR_CUDA;              \
  } while (0)

GroupedGemmArgs gemm_args(int mode, const moe_config_t* c, const int32_t* offsets,
                          int64_t uniform_rows, int d, int f, const void* A, const void* B,
                          void* out0, void* out1, const void* aux, int* err) {
  GroupedGemmArgs a{};
  a.mode = mode;
  a.offsets = offsets;
  a.G = uniform_rows > 0 ? 1 : c->E;
  a.uniform_rows = uniform_rows;
  a.rows_cap = uniform_rows > 0 ? uniform_rows : c->T * c->k;
  a.d = d;
  a.f = f;
  a.A = A;
  a.B = B;
  a.out0 = out0;
  a.out1 = out1;
  a.aux = aux;
  a.err = err;
  return a;
}

// Rows of the FC1 input taken from x through src_tok (the fused permute), or none.
struct Gather {
  const int32_t* idx = nullptr;
  const void* src = nullptr;
  int64_t rows = 0;
};

void set_gather(GroupedGemmArgs& a, const Gather& gx) {
  a.gather_idx = gx.idx;
  a.gather_src = gx.src;
  a.gather_rows = gx.rows;
}

moe_status_t ffn_fwd(const moe_config_t* c, const void* xp, const int32_t* offsets,
                     int64_t uniform_rows, int f, const void* W1, const void* W2, void* ab,
                     void* h, void* yp, int* err, cudaStream_t st, Gather gx = {}) {
  GroupedGemmArgs a1 = gemm_args(GEMM_FC1_SWIGLU, c, offsets, uniform_rows, c->d, f, xp, W1, ab,
                                 h, nullptr, err);
  set_gather(a1, gx);
  MOE_TRY(launch_grouped_gemm(a1, st));
  GroupedGemmArgs a2 =
      gemm_args(GEMM_FC2, c, offsets, uniform_rows, c->d, f, h, W2, yp, nullptr, nullptr, err);
  MOE_TRY(launch_grouped_gemm(a2, st));
  return MOE_OK;
}

// The FC2 data-gradient's rows taken from dy through src_tok, each scaled by its slot's
// gate weight in the epilogue (the dispatch of dy fused into that GEMM), or none.
struct DyDispatch {
  Gather rows;
  const float* topk_w = nullptr;
  const int32_t* src_slot = nullptr;
  int64_t n_slots = 0;
};

moe_status_t ffn_bwd(const moe_config_t* c, const void* dyp, const void* xp,
                     const int32_t* offsets, int64_t uniform_rows, int f, const void* W1,
                     const void* W2, const void* ab, const void* h, void* dab, void* dxp,
                     void* dW1, void* dW2, void* seg_maps, int* err, cudaStream_t st,
                     Gather gx = {}, DyDispatch gd = {}) {
  GroupedGemmArgs g2 = gemm_args(GEMM_DGRAD2_SWIGLU, c, offsets, uniform_rows, c->d, f, dyp, W2,
                                 dab, nullptr, ab, err);
  if (gd.rows.idx) {
    set_gather(g2, gd.rows);
    g2.gate_w = gd.topk_w;
    g2.gate_slot = gd.src_slot;
    g2.n_slots = gd.n_slots;
  }
  MOE_TRY(launch_grouped_gemm(g2, st));
  GroupedGemmArgs w2 = gemm_args(GEMM_WGRAD, c, offsets, uniform_rows, c->d, f, dyp, h, dW2,
                                 nullptr, nullptr, err);
  w2.wg_M = c->d;
  w2.wg_N = f;
  w2.seg_maps = seg_maps;
  MOE_TRY(launch_grouped_gemm(w2, st));
  GroupedGemmArgs g1 = gemm_args(GEMM_DGRAD1, c, offsets, uniform_rows, c->d, f, dab, W1, dxp,
                                 nullptr, nullptr, err);
  MOE_TRY(launch_grouped_gemm(g1, st));
  GroupedGemmArgs w1 = gemm_args(GEMM_WGRAD, c, offsets, uniform_rows, c->d, f, dab, xp, dW1,
                                 nullptr, nullptr, err);
  w1.wg_M = 2 * f;
  w1.wg_N = c->d;
  w1.seg_maps = seg_maps;
  set_gather(w1, gx);
  MOE_TRY(launch_grouped_gemm(w1, st));
  return MOE_OK;
}

// A wait that nothing will complete: the bounded wait gives up, flags the timeout and the
// kernel returns (the path every pipeline wait of the grouped GEMM takes on a stall).
__global__ void selftest_wait_kernel(int* err, long long budget) {
  __shared__ uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bar), 1);
    fence_mbar_init();
    abort_flag = 0;
  }
  __syncthreads();
  if (threadIdx.x == 0) mbar_wait_bounded(smem_u32(&bar), 0, &abort_flag, err, budget);
}

// ----------------------------------------------------------------- routers and 8-bit operands
moe_status_t validate_router(const moe_config_t* c, const moe_router_t* r) {
  const moe_status_t s = validate(c);
  if (s != MOE_OK) return s;
  if (!r || c->select_bias || c->drop_negative || c->drop_by_score) return MOE_ERR_INVALID_ARG;
  if (r->score != MOE_SCORE_SOFTMAX && r->score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (r->groups < 1 || c->E % r->groups || r->top_groups < 1 || r->top_groups > r->groups ||
      (r->group_top != 1 && r->group_top != 2) || (r->renorm != 0 && r->renorm != 1))
    return MOE_ERR_INVALID_ARG;
  const int per = c->E / r->groups;
  if (r->top_groups * per < c->k || (r->groups > 1 && r->group_top > per))
    return MOE_ERR_INVALID_ARG;
  if (r->bias && (reinterpret_cast<uintptr_t>(r->bias) & 3u)) return MOE_ERR_INVALID_ARG;
  return r->groups > 32 ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

constexpr int32_t FP8_MAX_DIM = 1 << 24;
constexpr int64_t FP8_MAX_ROWS = (int64_t(1) << 31) - (1 << 15);

moe_status_t validate_segments(int64_t rows, int32_t G, const int32_t* offsets) {
  if (rows < 0 || G < 1 || (!offsets && G != 1)) return MOE_ERR_INVALID_ARG;
  if (offsets && !aligned16(offsets)) return MOE_ERR_INVALID_ARG;
  return (rows >= FP8_MAX_ROWS || G > 256) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}
moe_status_t validate_dim(int64_t n) {
  if (n < 1) return MOE_ERR_INVALID_ARG;
  return n >= FP8_MAX_DIM ? MOE_ERR_UNSUPPORTED : MOE_OK;
}
bool ld_ok(int64_t ld, int64_t n) { return ld >= n && ld % 16 == 0; }
// codes and their scales: both given, or (optional) neither
bool pair_ok(const void* codes, const void* scales, bool optional) {
  return (optional && !codes && !scales) || ptrs_ok(codes, scales);
}

// What every quantiser checks of its outputs; `cols` columns.
moe_status_t validate_quant_out(int64_t rows, int32_t G, const int32_t* offsets, int64_t cols,
                                int64_t ld, int32_t pow2, const void* codes, const void* scales,
                                const void* codes_t, const void* scales_t, const void* ws) {
  moe_status_t s = validate_segments(rows, G, offsets);
  if (s == MOE_OK) s = validate_dim(cols);
  if (s != MOE_OK) return s;
  if (pow2 != 0 && pow2 != 1) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;   // empty buffers may have no address
  if (!pair_ok(codes, scales, true) ||
      !pair_ok(codes_t, scales_t, true) || (!codes && !codes_t) || !ptrs_ok(ws) ||
      (codes && !ld_ok(ld, cols)))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

}  // namespace

extern "C" {

int32_t moe_capacity_from_factor(int64_t T, int32_t k, int32_t E, double c) {
  if (T <= 0 || k <= 0 || E <= 0) return -1;
  if (!(c > 0.0)) return 0;
  const long double v = static_cast<long double>(c) * static_cast<long double>(T) *
                        static_cast<long double>(k) / static_cast<long double>(E);
  // absorb binary representation error of c (e.g. 1.25 is exact, 0.1 is not)
  const long double fl = std::floor(v + 1e-9L);
  if (fl > 2147483647.0L) return 2147483647;
  return static_cast<int32_t>(fl);
}

moe_status_t moe_workspace_size(const moe_config_t* cfg, size_t* ws_bytes, size_t* ctx_bytes) {
  moe_status_t s = validate(cfg);
  if (s != MOE_OK) return s;
  if (ws_bytes) *ws_bytes = ws_layout(cfg).total;
  if (ctx_bytes) *ctx_bytes = ctx_layout(cfg).total;
  return MOE_OK;
}

moe_status_t moe_stage_workspace_size(const moe_config_t* cfg, size_t* ws_bytes) {
  const moe_status_t s = validate(cfg);
  if (s != MOE_OK) return s;
  if (!ws_bytes) return MOE_ERR_INVALID_ARG;
  *ws_bytes = ws_layout(cfg).dyp;
  return MOE_OK;
}

moe_status_t moe_ctx_offsets(const moe_config_t* cfg, size_t* offsets) {
  moe_status_t s = validate(cfg);
  if (s != MOE_OK) return s;
  if (!offsets) return MOE_ERR_INVALID_ARG;
  CtxLayout L = ctx_layout(cfg);
  for (int i = 0; i < MOE_CTX_NFIELDS; ++i) offsets[i] = L.off[i];
  return MOE_OK;
}

moe_status_t moe_ws_init(void* ws, void* stream) {
  if (!ptrs_ok(ws)) return MOE_ERR_INVALID_ARG;
  return cuda_status(cudaMemsetAsync(ws, 0, WS_HEADER_BYTES, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_route(const moe_config_t* cfg, const float* logits, int32_t* topk_idx,
                       float* topk_w, int32_t* counts, int32_t* kept, int32_t* offsets,
                       int32_t* dest_row, int32_t* src_tok, int32_t* src_slot,
                       uint8_t* drop_mask, void* ws, void* stream) {
  moe_status_t s = validate(cfg);
  if (s != MOE_OK) return s;
  if (!ptrs_ok(logits, topk_idx, topk_w, counts, kept, offsets, dest_row, src_tok, src_slot,
               drop_mask, ws))
    return MOE_ERR_INVALID_ARG;
  WsLayout W = ws_layout(cfg);
  return cuda_status(launch_route(cfg, logits, topk_idx, topk_w, counts, kept, offsets,
                                  dest_row, src_tok, src_slot, drop_mask, at<uint8_t>(ws, W.route),
                                  static_cast<int*>(ws), static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_permute(const moe_config_t* cfg, const void* x, const int32_t* src_tok,
                         const int32_t* offsets, void* xp, void* ws, void* stream) {
  moe_status_t s = validate(cfg);
  if (s != MOE_OK) return s;
  if (!ptrs_ok(x, src_tok, offsets, xp, ws)) return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_permute(x, src_tok, offsets, cfg->E, cfg->T, cfg->T * cfg->k, cfg->d,
                                    xp, static_cast<int*>(ws),
                                    static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_grouped_ffn(const moe_config_t* cfg, const void* xp, const int32_t* offsets,
                             const void* W1, const void* W2, void* ab, void* h, void* yp,
                             void* ws, void* stream) {
  moe_status_t s = validate(cfg);
  if (s != MOE_OK) return s;
  if (!ptrs_ok(xp, offsets, W1, W2, ab, h, yp, ws)) return MOE_ERR_INVALID_ARG;
  return ffn_fwd(cfg, xp, offsets, 0, cfg->ffn, W1, W2, ab, h, yp, static_cast<int*>(ws),
                 static_cast<cudaStream_t>(stream));
}

moe_status_t moe_grouped_ffn_gather(const moe_config_t* cfg, const void* x,
                                    const int32_t* src_tok, const int32_t* offsets,
                                    const void* W1, const void* W2, void* ab, void* h, void* yp,
                                    void* ws, void* stream) {
  moe_status_t s = validate(cfg);
  if (s != MOE_OK) return s;
  if (!ptrs_ok(x, src_tok, offsets, W1, W2, ab, h, yp, ws)) return MOE_ERR_INVALID_ARG;
  Gather gx;
  gx.idx = src_tok;
  gx.src = x;
  gx.rows = cfg->T;
  return ffn_fwd(cfg, nullptr, offsets, 0, cfg->ffn, W1, W2, ab, h, yp, static_cast<int*>(ws),
                 static_cast<cudaStream_t>(stream), gx);
}

moe_status_t moe_combine(const moe_config_t* cfg, const void* yp, const int32_t* dest_row,
                         const float* topk_w, const void* ys_or_null, void* y, void* ws,
                         void* stream) {
  moe_status_t s = validate(cfg);
  if (s != MOE_OK) return s;
  if (!ptrs_ok(yp, dest_row, topk_w, y, ws)) return MOE_ERR_INVALID_ARG;
  if (ys_or_null && !aligned16(ys_or_null)) return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_combine(yp, dest_row, topk_w, ys_or_null, cfg->T, cfg->k, cfg->d,
                                    cfg->T * cfg->k, y, static_cast<int*>(ws),
                                    static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_combine_bwd(const moe_config_t* cfg, const void* dy, const void* yp,
                             const float* logits, const int32_t* topk_idx, const float* topk_w,
                             const int32_t* dest_row, void* dyp, float* dlogits, void* ws,
                             void* stream) {
  moe_status_t s = validate(cfg);
  if (s != MOE_OK) return s;
  if (!ptrs_ok(dy, yp, logits, topk_idx, topk_w, dest_row, dyp, dlogits, ws))
    return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_combine_bwd(dy, yp, logits, topk_idx, topk_w, dest_row, cfg->T,
                                        cfg->E, cfg->k, cfg->d, cfg->gate, cfg->route_scale,
                                        cfg->T * cfg->k, dyp, dlogits, static_cast<int*>(ws),
                                        static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_grouped_ffn_bwd(const moe_config_t* cfg, const void* dyp, const void* xp,
                                 const int32_t* offsets, const void* W1, const void* W2,
                                 const void* ab, const void* h, void* dab, void* dxp, void* dW1,
                                 void* dW2, void* ws, void* stream) {
  moe_status_t s = validate(cfg);
  if (s != MOE_OK) return s;
  if (!ptrs_ok(dyp, xp, offsets, W1, W2, ab, h, dab, dxp, dW1, dW2, ws))
    return MOE_ERR_INVALID_ARG;
  return ffn_bwd(cfg, dyp, xp, offsets, 0, cfg->ffn, W1, W2, ab, h, dab, dxp, dW1, dW2,
                 at<uint8_t>(ws, ws_layout(cfg).maps), static_cast<int*>(ws),
                 static_cast<cudaStream_t>(stream));
}

moe_status_t moe_grouped_ffn_bwd_gather(const moe_config_t* cfg, const void* dyp, const void* x,
                                        const int32_t* src_tok, const int32_t* offsets,
                                        const void* W1, const void* W2, const void* ab,
                                        const void* h, void* dab, void* dxp, void* dW1,
                                        void* dW2, void* ws, void* stream) {
  moe_status_t s = validate(cfg);
  if (s != MOE_OK) return s;
  if (!ptrs_ok(dyp, x, src_tok, offsets, W1, W2, ab, h, dab, dxp, dW1, dW2, ws))
    return MOE_ERR_INVALID_ARG;
  Gather gx;
  gx.idx = src_tok;
  gx.src = x;
  gx.rows = cfg->T;
  return ffn_bwd(cfg, dyp, nullptr, offsets, 0, cfg->ffn, W1, W2, ab, h, dab, dxp, dW1, dW2,
                 at<uint8_t>(ws, ws_layout(cfg).maps), static_cast<int*>(ws),
                 static_cast<cudaStream_t>(stream), gx);
}

moe_status_t moe_grouped_ffn_bwd_dispatch(const moe_config_t* cfg, const void* dy,
                                          const float* topk_w, const int32_t* src_tok,
                                          const int32_t* src_slot, const void* dyp,
                                          const void* xp, const int32_t* offsets,
                                          const void* W1, const void* W2, const void* ab,
                                          const void* h, void* dab, void* dxp, void* dW1,
                                          void* dW2, void* ws, void* stream) {
  moe_status_t s = validate(cfg);
  if (s != MOE_OK) return s;
  if (!ptrs_ok(dy, topk_w, src_tok, src_slot, dyp, xp, offsets, W1, W2, ab, h, dab, dxp, dW1,
               dW2, ws))
    return MOE_ERR_INVALID_ARG;
  DyDispatch gd;
  gd.rows.idx = src_tok;
  gd.rows.src = dy;
  gd.rows.rows = cfg->T;
  gd.topk_w = topk_w;
  gd.src_slot = src_slot;
  gd.n_slots = cfg->T * cfg->k;
  return ffn_bwd(cfg, dyp, xp, offsets, 0, cfg->ffn, W1, W2, ab, h, dab, dxp, dW1, dW2,
                 at<uint8_t>(ws, ws_layout(cfg).maps), static_cast<int*>(ws),
                 static_cast<cudaStream_t>(stream), Gather{}, gd);
}

moe_status_t moe_unpermute_reduce(const moe_config_t* cfg, const void* dxp,
                                  const int32_t* dest_row, const void* dxs_or_null, void* dx,
                                  void* ws, void* stream) {
  moe_status_t s = validate(cfg);
  if (s != MOE_OK) return s;
  if (!ptrs_ok(dxp, dest_row, dx, ws)) return MOE_ERR_INVALID_ARG;
  if (dxs_or_null && !aligned16(dxs_or_null)) return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_combine(dxp, dest_row, nullptr, dxs_or_null, cfg->T, cfg->k, cfg->d,
                                    cfg->T * cfg->k, dx, static_cast<int*>(ws),
                                    static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_layer_fwd(const moe_config_t* cfg, const float* logits, const void* x,
                           const void* W1, const void* W2, const void* W1s, const void* W2s,
                           void* y, void* ctx, void* ws, void* stream) {
  moe_status_t s = validate(cfg);
  if (s != MOE_OK) return s;
  if (!ptrs_ok(logits, x, W1, W2, y, ctx, ws)) return MOE_ERR_INVALID_ARG;
  if (cfg->ffn_shared && !ptrs_ok(W1s, W2s)) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int* err = static_cast<int*>(ws);
  CtxLayout C = ctx_layout(cfg);
  WsLayout W = ws_layout(cfg);
  int32_t* offsets = at<int32_t>(ctx, C.off[MOE_CTX_OFFSETS]);
  MOE_TRY(launch_route(cfg, logits, at<int32_t>(ctx, C.off[MOE_CTX_TOPK_IDX]),
                       at<float>(ctx, C.off[MOE_CTX_TOPK_W]),
                       at<int32_t>(ctx, C.off[MOE_CTX_COUNTS]),
                       at<int32_t>(ctx, C.off[MOE_CTX_KEPT]), offsets,
                       at<int32_t>(ctx, C.off[MOE_CTX_DEST_ROW]),
                       at<int32_t>(ctx, C.off[MOE_CTX_SRC_TOK]),
                       at<int32_t>(ctx, C.off[MOE_CTX_SRC_SLOT]),
                       at<uint8_t>(ctx, C.off[MOE_CTX_DROP_MASK]), at<uint8_t>(ws, W.route), err,
                       st));
  void* xp = at<uint8_t>(ctx, C.off[MOE_CTX_XP]);
  MOE_TRY(launch_permute(x, at<int32_t>(ctx, C.off[MOE_CTX_SRC_TOK]), offsets, cfg->E, cfg->T,
                         cfg->T * cfg->k, cfg->d, xp, err, st));
  void* yp = at<uint8_t>(ctx, C.off[MOE_CTX_YP]);
  const bool rc = cfg->recompute != 0;
  void* ab = rc ? at<uint8_t>(ws, W.ab) : at<uint8_t>(ctx, C.off[MOE_CTX_AB]);
  void* h = rc ? at<uint8_t>(ws, W.h) : at<uint8_t>(ctx, C.off[MOE_CTX_H]);
  s = ffn_fwd(cfg, xp, offsets, 0, cfg->ffn, W1, W2, ab, h, yp, err, st);
  if (s != MOE_OK) return s;
  const void* ys = nullptr;
  if (cfg->ffn_shared) {
    void* ysw = at<uint8_t>(ctx, C.off[MOE_CTX_YS]);
    void* ab_s = rc ? at<uint8_t>(ws, W.ab_s) : at<uint8_t>(ctx, C.off[MOE_CTX_AB_S]);
    void* h_s = rc ? at<uint8_t>(ws, W.h_s) : at<uint8_t>(ctx, C.off[MOE_CTX_H_S]);
    s = ffn_fwd(cfg, x, nullptr, cfg->T, cfg->ffn_shared, W1s, W2s, ab_s, h_s, ysw, err, st);
    if (s != MOE_OK) return s;
    ys = ysw;
  }
  MOE_TRY(launch_combine(yp, at<int32_t>(ctx, C.off[MOE_CTX_DEST_ROW]),
                         at<float>(ctx, C.off[MOE_CTX_TOPK_W]), ys, cfg->T, cfg->k, cfg->d,
                         cfg->T * cfg->k, y, err, st));
  return MOE_OK;
}

moe_status_t moe_mx_weights_size(const moe_config_t* cfg, size_t* bytes, size_t* offsets) {
  moe_status_t s = validate(cfg);
  if (s != MOE_OK) return s;
  if (cfg->d % 128 || cfg->ffn % 128) return MOE_ERR_UNSUPPORTED;
  const MxWeightLayout L = mx_weight_layout(cfg->E, cfg->d, cfg->ffn);
  if (bytes) *bytes = L.total;
  if (offsets) {
    offsets[0] = L.w1q;
    offsets[1] = L.w1sf;
    offsets[2] = L.w2q;
    offsets[3] = L.w2sf;
    offsets[4] = L.w2tq;
    offsets[5] = L.w2tsf;
    offsets[6] = L.w1tq;
    offsets[7] = L.w1tsf;
  }
  return MOE_OK;
}

moe_status_t moe_mx_act_scales_size(const moe_config_t* cfg, int32_t K, size_t* bytes) {
  moe_status_t s = validate(cfg);
  if (s != MOE_OK) return s;
  if (K <= 0 || K % 128 || !bytes) return MOE_ERR_INVALID_ARG;
  *bytes = mx_act_scale_bytes(cfg->T * cfg->k, cfg->E, K);
  return MOE_OK;
}

moe_status_t moe_mx_quantize_weights(const moe_config_t* cfg, const void* W1, const void* W2,
                                     void* wq, void* stream) {
  size_t bytes = 0;
  moe_status_t s = moe_mx_weights_size(cfg, &bytes, nullptr);
  if (s != MOE_OK) return s;
  if (!ptrs_ok(W1, W2, wq) || (reinterpret_cast<uintptr_t>(wq) & 255u)) return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_mx_quant_weights(W1, W2, cfg->E, cfg->d, cfg->ffn, wq,
                                             static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_mx_permute_quant(const moe_config_t* cfg, const void* x, const int32_t* src_tok,
                                  const int32_t* offsets, void* xp_or_null, void* xq,
                                  uint8_t* x_sf, void* ws, void* stream) {
  moe_status_t s = validate(cfg);
  if (s != MOE_OK) return s;
  if (cfg->d % 128) return MOE_ERR_UNSUPPORTED;
  if (!ptrs_ok(x, src_tok, offsets, xq, x_sf, ws)) return MOE_ERR_INVALID_ARG;
  if (xp_or_null && !aligned16(xp_or_null)) return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_mx_permute_quant(x, src_tok, offsets, cfg->E, cfg->T,
                                             cfg->T * cfg->k, cfg->d, xp_or_null, xq, x_sf,
                                             static_cast<int*>(ws),
                                             static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_grouped_ffn_mx(const moe_config_t* cfg, const void* xq, const uint8_t* x_sf,
                                const int32_t* offsets, const void* wq, void* ab, void* h,
                                uint8_t* hq, uint8_t* h_sf, void* yp, void* ws, void* stream) {
  moe_status_t s = validate(cfg);
  if (s != MOE_OK) return s;
  if (cfg->d % 128 || cfg->ffn % 128) return MOE_ERR_UNSUPPORTED;
  if (!ptrs_ok(xq, x_sf, offsets, wq, ab, h, hq, h_sf, yp, ws)) return MOE_ERR_INVALID_ARG;
  MxFfnArgs a{};
  a.E = cfg->E;
  a.d = cfg->d;
  a.f = cfg->ffn;
  a.rows_cap = cfg->T * cfg->k;
  a.offsets = offsets;
  a.xq = xq;
  a.x_sf = x_sf;
  a.wq = wq;
  a.ab = ab;
  a.h = h;
  a.hq = hq;
  a.h_sf = h_sf;
  a.yp = yp;
  a.err = static_cast<int*>(ws);
  return cuda_status(launch_mx_ffn(a, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_layer_fwd_mx(const moe_config_t* cfg, const float* logits, const void* x,
                              const void* wq, const void* W1s, const void* W2s, void* y,
                              void* ctx, void* ws, void* stream) {
  moe_status_t s = validate(cfg);
  if (s != MOE_OK) return s;
  if (!cfg->mxfp8) return MOE_ERR_INVALID_ARG;
  if (!ptrs_ok(logits, x, wq, y, ctx, ws)) return MOE_ERR_INVALID_ARG;
  if (cfg->ffn_shared && !ptrs_ok(W1s, W2s)) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int* err = static_cast<int*>(ws);
  CtxLayout C = ctx_layout(cfg);
  WsLayout W = ws_layout(cfg);
  int32_t* offsets = at<int32_t>(ctx, C.off[MOE_CTX_OFFSETS]);
  const int32_t* src_tok = at<int32_t>(ctx, C.off[MOE_CTX_SRC_TOK]);
  MOE_TRY(launch_route(cfg, logits, at<int32_t>(ctx, C.off[MOE_CTX_TOPK_IDX]),
                       at<float>(ctx, C.off[MOE_CTX_TOPK_W]),
                       at<int32_t>(ctx, C.off[MOE_CTX_COUNTS]),
                       at<int32_t>(ctx, C.off[MOE_CTX_KEPT]), offsets,
                       at<int32_t>(ctx, C.off[MOE_CTX_DEST_ROW]),
                       at<int32_t>(ctx, C.off[MOE_CTX_SRC_TOK]),
                       at<int32_t>(ctx, C.off[MOE_CTX_SRC_SLOT]),
                       at<uint8_t>(ctx, C.off[MOE_CTX_DROP_MASK]), at<uint8_t>(ws, W.route), err,
                       st));
  void* xp = at<uint8_t>(ctx, C.off[MOE_CTX_XP]);
  MOE_TRY(launch_mx_permute_quant(x, src_tok, offsets, cfg->E, cfg->T, cfg->T * cfg->k, cfg->d,
                                  xp, at<uint8_t>(ws, W.xq), at<uint8_t>(ws, W.x_sf), err, st));
  MxFfnArgs a{};
  a.E = cfg->E;
  a.d = cfg->d;
  a.f = cfg->ffn;
  a.rows_cap = cfg->T * cfg->k;
  a.offsets = offsets;
  a.xq = at<uint8_t>(ws, W.xq);
  a.x_sf = at<uint8_t>(ws, W.x_sf);
  a.wq = wq;
  a.ab = at<uint8_t>(ctx, C.off[MOE_CTX_AB]);
  a.h = at<uint8_t>(ctx, C.off[MOE_CTX_H]);
  a.hq = at<uint8_t>(ws, W.hq);
  a.h_sf = at<uint8_t>(ws, W.h_sf);
  void* yp = at<uint8_t>(ctx, C.off[MOE_CTX_YP]);
  a.yp = yp;
  a.err = err;
  MOE_TRY(launch_mx_ffn(a, st));
  const void* ys = nullptr;
  if (cfg->ffn_shared) {   // the shared expert stays bf16
    void* ysw = at<uint8_t>(ctx, C.off[MOE_CTX_YS]);
    s = ffn_fwd(cfg, x, nullptr, cfg->T, cfg->ffn_shared, W1s, W2s,
                at<uint8_t>(ctx, C.off[MOE_CTX_AB_S]), at<uint8_t>(ctx, C.off[MOE_CTX_H_S]), ysw,
                err, st);
    if (s != MOE_OK) return s;
    ys = ysw;
  }
  MOE_TRY(launch_combine(yp, at<int32_t>(ctx, C.off[MOE_CTX_DEST_ROW]),
                         at<float>(ctx, C.off[MOE_CTX_TOPK_W]), ys, cfg->T, cfg->k, cfg->d,
                         cfg->T * cfg->k, y, err, st));
  return MOE_OK;
}

namespace {
// The MXFP8 backward of the routed experts' FFN: quantise dyp, DGRAD2 and DGRAD1 on MXFP8
// operands, then the two weight gradients: bf16 (mxfp8 = 1), or (mxfp8 = 2) on operands
// quantised along each segment's tokens.
moe_status_t ffn_bwd_mx(const moe_config_t* c, const void* dyp, const void* xp,
                        const int32_t* offsets, const void* wq, const void* ab, const void* h,
                        void* dab, void* dxp, void* dW1, void* dW2, void* ws, cudaStream_t st) {
  const WsLayout W = ws_layout(c);
  int* err = static_cast<int*>(ws);
  const int64_t R = c->T * c->k;
  MOE_TRY(launch_mx_permute_quant(dyp, nullptr, offsets, c->E, R, R, c->d, nullptr,
                                  at<uint8_t>(ws, W.dyq), at<uint8_t>(ws, W.dy_sf), err, st));
  MxDgradArgs a{};
  a.E = c->E;
  a.d = c->d;
  a.f = c->ffn;
  a.rows_cap = R;
  a.offsets = offsets;
  a.dyq = at<uint8_t>(ws, W.dyq);
  a.dy_sf = at<uint8_t>(ws, W.dy_sf);
  a.wq = wq;
  a.ab = ab;
  a.dab = dab;
  a.dabq = at<uint8_t>(ws, W.dabq);
  a.dab_sf = at<uint8_t>(ws, W.dab_sf);
  a.dxp = dxp;
  a.err = err;
  MOE_TRY(launch_mx_ffn_dgrad(a, st));
  if (c->mxfp8 == 2) {
    auto quant = [&](const void* X, int C, bool role_n, size_t q, size_t sf) {
      return launch_mx_quant_tok(X, offsets, c->E, R, C, role_n, at<uint8_t>(ws, q),
                                 at<uint8_t>(ws, sf), err, st);
    };
    MxWgradArgs g{};
    g.E = c->E;
    g.rows_cap = R;
    g.offsets = offsets;
    g.err = err;
    // dW2 [E][d][f] = dyp^T h
    MOE_TRY(quant(dyp, c->d, false, W.dyT, W.dyT_sf));
    MOE_TRY(quant(h, c->ffn, true, W.hT, W.hT_sf));
    g.M = c->d;
    g.N = c->ffn;
    g.aq = at<uint8_t>(ws, W.dyT);
    g.a_sf = at<uint8_t>(ws, W.dyT_sf);
    g.bq = at<uint8_t>(ws, W.hT);
    g.b_sf = at<uint8_t>(ws, W.hT_sf);
    g.dW = dW2;
    MOE_TRY(launch_mx_wgrad(g, st));
    // dW1 [E][2f][d] = dab^T xp
    MOE_TRY(quant(dab, 2 * c->ffn, false, W.dabT, W.dabT_sf));
    MOE_TRY(quant(xp, c->d, true, W.xpT, W.xpT_sf));
    g.M = 2 * c->ffn;
    g.N = c->d;
    g.aq = at<uint8_t>(ws, W.dabT);
    g.a_sf = at<uint8_t>(ws, W.dabT_sf);
    g.bq = at<uint8_t>(ws, W.xpT);
    g.b_sf = at<uint8_t>(ws, W.xpT_sf);
    g.dW = dW1;
    MOE_TRY(launch_mx_wgrad(g, st));
    return MOE_OK;
  }
  void* maps = at<uint8_t>(ws, W.maps);
  GroupedGemmArgs w2 = gemm_args(GEMM_WGRAD, c, offsets, 0, c->d, c->ffn, dyp, h, dW2, nullptr,
                                 nullptr, err);
  w2.wg_M = c->d;
  w2.wg_N = c->ffn;
  w2.seg_maps = maps;
  MOE_TRY(launch_grouped_gemm(w2, st));
  GroupedGemmArgs w1 = gemm_args(GEMM_WGRAD, c, offsets, 0, c->d, c->ffn, dab, xp, dW1, nullptr,
                                 nullptr, err);
  w1.wg_M = 2 * c->ffn;
  w1.wg_N = c->d;
  w1.seg_maps = maps;
  MOE_TRY(launch_grouped_gemm(w1, st));
  return MOE_OK;
}
}  // namespace

moe_status_t moe_grouped_ffn_bwd_mx(const moe_config_t* cfg, const void* dyp, const void* xp,
                                    const int32_t* offsets, const void* wq, const void* ab,
                                    const void* h, void* dab, void* dxp, void* dW1, void* dW2,
                                    void* ws, void* stream) {
  moe_status_t s = validate(cfg);
  if (s != MOE_OK) return s;
  if (!cfg->mxfp8) return MOE_ERR_INVALID_ARG;
  if (!ptrs_ok(dyp, xp, offsets, wq, ab, h, dab, dxp, dW1, dW2, ws)) return MOE_ERR_INVALID_ARG;
  return ffn_bwd_mx(cfg, dyp, xp, offsets, wq, ab, h, dab, dxp, dW1, dW2, ws,
                    static_cast<cudaStream_t>(stream));
}

namespace {
// The whole backward; wq != null runs the routed experts' data gradients on MXFP8 operands.
moe_status_t layer_bwd(const moe_config_t* cfg, const void* ctx, const float* logits,
                       const void* x, const void* dy, const void* W1, const void* W2,
                       const void* wq, const void* W1s, const void* W2s, void* dx, void* dW1,
                       void* dW2, void* dW1s, void* dW2s, float* dlogits, void* ws,
                       void* stream) {
  moe_status_t s = MOE_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int* err = static_cast<int*>(ws);
  CtxLayout C = ctx_layout(cfg);
  WsLayout W = ws_layout(cfg);
  const int32_t* offsets = at<int32_t>(ctx, C.off[MOE_CTX_OFFSETS]);
  const int32_t* dest_row = at<int32_t>(ctx, C.off[MOE_CTX_DEST_ROW]);
  void* dyp = at<uint8_t>(ws, W.dyp);
  void* dab = at<uint8_t>(ws, W.dab);
  void* dxp = at<uint8_t>(ws, W.dxp);
  const bool rc = cfg->recompute != 0;
  const void* xp_saved = at<uint8_t>(ctx, C.off[MOE_CTX_XP]);
  const void* ab = at<uint8_t>(ctx, C.off[MOE_CTX_AB]);
  const void* h = at<uint8_t>(ctx, C.off[MOE_CTX_H]);
  const void* ab_s = at<uint8_t>(ctx, C.off[MOE_CTX_AB_S]);
  const void* h_s = at<uint8_t>(ctx, C.off[MOE_CTX_H_S]);
  if (rc) {
    // selective rematerialisation: rerun FC1 (+ SwiGLU) from the saved permuted tokens;
    // the grouped GEMM is deterministic, so ab and h equal the forward's bit for bit
    GroupedGemmArgs a1 = gemm_args(GEMM_FC1_SWIGLU, cfg, offsets, 0, cfg->d, cfg->ffn, xp_saved,
                                   W1, at<uint8_t>(ws, W.ab), at<uint8_t>(ws, W.h), nullptr, err);
    MOE_TRY(launch_grouped_gemm(a1, st));
    ab = at<uint8_t>(ws, W.ab);
    h = at<uint8_t>(ws, W.h);
    if (cfg->ffn_shared) {
      GroupedGemmArgs a2 = gemm_args(GEMM_FC1_SWIGLU, cfg, nullptr, cfg->T, cfg->d,
                                     cfg->ffn_shared, x, W1s, at<uint8_t>(ws, W.ab_s),
                                     at<uint8_t>(ws, W.h_s), nullptr, err);
      MOE_TRY(launch_grouped_gemm(a2, st));
      ab_s = at<uint8_t>(ws, W.ab_s);
      h_s = at<uint8_t>(ws, W.h_s);
    }
  }
  MOE_TRY(launch_combine_bwd(dy, at<uint8_t>(ctx, C.off[MOE_CTX_YP]), logits,
                             at<int32_t>(ctx, C.off[MOE_CTX_TOPK_IDX]),
                             at<float>(ctx, C.off[MOE_CTX_TOPK_W]), dest_row, cfg->T, cfg->E,
                             cfg->k, cfg->d, cfg->gate, cfg->route_scale, cfg->T * cfg->k, dyp,
                             dlogits, err, st));
  if (wq)
    s = ffn_bwd_mx(cfg, dyp, xp_saved, offsets, wq, ab, h, dab, dxp, dW1, dW2, ws, st);
  else
    s = ffn_bwd(cfg, dyp, xp_saved, offsets, 0, cfg->ffn, W1, W2, ab, h, dab, dxp, dW1, dW2,
                at<uint8_t>(ws, W.maps), err, st);
  if (s != MOE_OK) return s;
  const void* dxs = nullptr;
  if (cfg->ffn_shared) {
    void* dxsw = at<uint8_t>(ws, W.dx_s);
    s = ffn_bwd(cfg, dy, x, nullptr, cfg->T, cfg->ffn_shared, W1s, W2s, ab_s, h_s,
                at<uint8_t>(ws, W.dab_s), dxsw, dW1s, dW2s, nullptr, err, st);
    if (s != MOE_OK) return s;
    dxs = dxsw;
  }
  MOE_TRY(launch_combine(dxp, dest_row, nullptr, dxs, cfg->T, cfg->k, cfg->d, cfg->T * cfg->k,
                         dx, err, st));
  return MOE_OK;
}
}  // namespace

moe_status_t moe_layer_bwd(const moe_config_t* cfg, const void* ctx, const float* logits,
                           const void* x, const void* dy, const void* W1, const void* W2,
                           const void* W1s, const void* W2s, void* dx, void* dW1, void* dW2,
                           void* dW1s, void* dW2s, float* dlogits, void* ws, void* stream) {
  moe_status_t s = validate(cfg);
  if (s != MOE_OK) return s;
  if (!ptrs_ok(ctx, logits, x, dy, W1, W2, dx, dW1, dW2, dlogits, ws)) return MOE_ERR_INVALID_ARG;
  if (cfg->ffn_shared && !ptrs_ok(W1s, W2s, dW1s, dW2s)) return MOE_ERR_INVALID_ARG;
  return layer_bwd(cfg, ctx, logits, x, dy, W1, W2, nullptr, W1s, W2s, dx, dW1, dW2, dW1s, dW2s,
                   dlogits, ws, stream);
}

moe_status_t moe_layer_bwd_mx(const moe_config_t* cfg, const void* ctx, const float* logits,
                              const void* x, const void* dy, const void* wq, const void* W1s,
                              const void* W2s, void* dx, void* dW1, void* dW2, void* dW1s,
                              void* dW2s, float* dlogits, void* ws, void* stream) {
  moe_status_t s = validate(cfg);
  if (s != MOE_OK) return s;
  if (!cfg->mxfp8) return MOE_ERR_INVALID_ARG;
  if (!ptrs_ok(ctx, logits, x, dy, wq, dx, dW1, dW2, dlogits, ws)) return MOE_ERR_INVALID_ARG;
  if (cfg->ffn_shared && !ptrs_ok(W1s, W2s, dW1s, dW2s)) return MOE_ERR_INVALID_ARG;
  return layer_bwd(cfg, ctx, logits, x, dy, nullptr, nullptr, wq, W1s, W2s, dx, dW1, dW2, dW1s,
                   dW2s, dlogits, ws, stream);
}

moe_status_t moe_selftest_wait_timeout(void* ws, int64_t budget_cycles, void* stream) {
  if (!ptrs_ok(ws) || budget_cycles <= 0) return MOE_ERR_INVALID_ARG;
  const long long budget = budget_cycles > 2000000000LL ? 2000000000LL : budget_cycles;
  selftest_wait_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(static_cast<int*>(ws),
                                                                        budget);
  return cuda_status(cudaGetLastError());
}

moe_status_t moe_gemm_clock_trace(int enable) {
  if (moe::gemm_clock_trace_set(enable != 0) != cudaSuccess ||
      moe::mx_clock_trace_set(enable != 0) != cudaSuccess)
    return MOE_ERR_CUDA;
  return MOE_OK;
}

moe_status_t moe_gemm_clock_read(uint64_t* cycles, uint64_t* ns, uint64_t* loops) {
  if (!cycles || !ns || !loops) return MOE_ERR_INVALID_ARG;
  unsigned long long sum[3] = {0, 0, 0};
  if (moe::gemm_clock_trace_add(sum) != cudaSuccess ||
      moe::mx_clock_trace_add(sum) != cudaSuccess)
    return MOE_ERR_CUDA;
  *cycles = sum[0];
  *ns = sum[1];
  *loops = sum[2];
  return MOE_OK;
}

moe_status_t moe_status(void* ws, void* stream, int32_t* flags) {
  if (!ptrs_ok(ws)) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int32_t h = 0;
  if (cudaMemcpyAsync(&h, ws, sizeof(h), cudaMemcpyDeviceToHost, st) != cudaSuccess)
    return MOE_ERR_CUDA;
  if (cudaStreamSynchronize(st) != cudaSuccess) return MOE_ERR_CUDA;
  if (h) {
    if (cudaMemsetAsync(ws, 0, sizeof(int32_t), st) != cudaSuccess) return MOE_ERR_CUDA;
    if (cudaStreamSynchronize(st) != cudaSuccess) return MOE_ERR_CUDA;
  }
  if (flags) *flags = h;
  if (h & MOE_DEVERR_TIMEOUT) return MOE_ERR_TIMEOUT;
  return h ? MOE_ERR_DEVICE_FLAG : MOE_OK;
}

const char* moe_status_string(moe_status_t s) {
  switch (s) {
    case MOE_OK: return "MOE_OK";
    case MOE_ERR_INVALID_ARG: return "MOE_ERR_INVALID_ARG";
    case MOE_ERR_UNSUPPORTED: return "MOE_ERR_UNSUPPORTED";
    case MOE_ERR_CUDA: return "MOE_ERR_CUDA";
    case MOE_ERR_DEVICE_FLAG: return "MOE_ERR_DEVICE_FLAG";
    case MOE_ERR_TIMEOUT: return "MOE_ERR_TIMEOUT";
  }
  return "MOE_ERR_UNKNOWN";
}

moe_status_t moe_route_groups(const moe_config_t* cfg, const moe_router_t* router,
                              const float* logits, int32_t* topk_idx, float* topk_w,
                              int32_t* counts, int32_t* kept, int32_t* offsets, int32_t* dest_row,
                              int32_t* src_tok, int32_t* src_slot, uint8_t* drop_mask, void* ws,
                              void* stream) {
  moe_status_t s = validate_router(cfg, router);
  if (s != MOE_OK) return s;
  if (!ptrs_ok(logits, topk_idx, topk_w, counts, kept, offsets, dest_row, src_tok, src_slot,
               drop_mask, ws))
    return MOE_ERR_INVALID_ARG;
  const WsLayout W = ws_layout(cfg);
  return cuda_status(launch_route_groups(cfg, router, logits, topk_idx, topk_w, counts, kept,
                                         offsets, dest_row, src_tok, src_slot, drop_mask,
                                         at<uint8_t>(ws, W.route), static_cast<int*>(ws),
                                         static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_route_groups_bwd(const moe_config_t* cfg, const moe_router_t* router,
                                  const float* logits, const int32_t* topk_idx, const float* dw,
                                  float* dlogits, void* ws, void* stream) {
  moe_status_t s = validate_router(cfg, router);
  if (s != MOE_OK) return s;
  if (!ptrs_ok(logits, topk_idx, dw, dlogits, ws)) return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_route_groups_bwd(cfg, router, logits, topk_idx, dw, dlogits,
                                             static_cast<int*>(ws),
                                             static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_combine_bwd_dw(const moe_config_t* cfg, const void* dy, const void* yp,
                                const float* topk_w, const int32_t* dest_row, void* dyp, float* dw,
                                void* ws, void* stream) {
  moe_status_t s = validate(cfg);
  if (s != MOE_OK) return s;
  if (!ptrs_ok(dy, yp, topk_w, dest_row, dyp, dw, ws)) return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_combine_bwd_dw(dy, yp, topk_w, dest_row, cfg->T, cfg->k, cfg->d,
                                           cfg->T * cfg->k, dyp, dw, static_cast<int*>(ws),
                                           static_cast<cudaStream_t>(stream)));
}

int64_t moe_fp8_token_blocks(int64_t rows, int32_t G) {
  return rows < 0 || G < 1 ? -1 : fp8_token_blocks(rows, G);
}

moe_status_t moe_fp8_quantize(const moe_fp8_quant_t* q, const void* x, const int32_t* src_tok,
                              const int32_t* offsets, void* codes, float* scales, void* codes_t,
                              float* scales_t, void* ws, void* stream) {
  if (!q) return MOE_ERR_INVALID_ARG;
  moe_status_t s = validate_quant_out(q->rows, q->G, offsets, q->C, q->ld, q->pow2, codes, scales,
                                      codes_t, scales_t, ws);
  if (s != MOE_OK) return s;
  if (q->rows == 0) return MOE_OK;
  // x: any bf16 address and row distance (rows that start off 16 bytes are read by the element)
  if (!x || (reinterpret_cast<uintptr_t>(x) & 1u) || q->ldx < q->C ||
      (src_tok && (!aligned16(src_tok) || q->src_rows < 1)))
    return MOE_ERR_INVALID_ARG;
  Fp8QuantArgs a{};
  a.src = FP8_SRC_ROWS;
  a.x = x;
  a.ldx = q->ldx;
  a.src_rows = q->src_rows;
  a.src_tok = src_tok;
  a.C = q->C;
  a.rows = q->rows;
  a.offsets = offsets;
  a.G = q->G;
  a.codes = codes;
  a.scales = scales;
  a.ld = q->ld;
  a.codes_t = codes_t;
  a.scales_t = scales_t;
  a.pow2 = q->pow2;
  a.err = static_cast<int*>(ws);
  return cuda_status(launch_fp8_quant(a, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_fp8_quantize_weights(const void* W, int32_t G, int32_t N, int32_t K, void* codes,
                                      int64_t ld, float* scales, void* codes_t, int64_t ld_t,
                                      float* scales_t, int32_t pow2, void* stream) {
  if (G < 1 || (pow2 != 0 && pow2 != 1)) return MOE_ERR_INVALID_ARG;
  moe_status_t s = validate_dim(N);
  if (s == MOE_OK) s = validate_dim(K);
  if (s != MOE_OK) return s;
  if (!W || (reinterpret_cast<uintptr_t>(W) & 1u) || !ptrs_ok(codes, scales) || !ld_ok(ld, K) ||
      !pair_ok(codes_t, scales_t, true) || (codes_t && !ld_ok(ld_t, N)))
    return MOE_ERR_INVALID_ARG;
  const int64_t blocks = ((N + 127) / 128) * static_cast<int64_t>((K + 127) / 128);
  if (G > 256 || G * blocks >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;
  return cuda_status(launch_fp8_weights(W, G, N, K, codes, ld, scales, codes_t, ld_t, scales_t,
                                        pow2, static_cast<cudaStream_t>(stream)));
}

static Fp8QuantArgs act_args(int src, const moe_fp8_act_t* p, const void* dh, const void* ab,
                             const int32_t* offsets, void* codes, float* scales, void* codes_t,
                             float* scales_t, void* ws) {
  Fp8QuantArgs a{};
  a.src = src;
  a.x = ab;
  a.dh = dh;
  a.f = p->f;
  a.rows = p->rows;
  a.offsets = offsets;
  a.G = p->G;
  a.codes = codes;
  a.scales = scales;
  a.ld = p->ld;
  a.codes_t = codes_t;
  a.scales_t = scales_t;
  a.pow2 = p->pow2;
  a.err = static_cast<int*>(ws);
  return a;
}

moe_status_t moe_fp8_swiglu(const moe_fp8_act_t* p, const void* ab, const int32_t* offsets,
                            void* codes, float* scales, void* codes_t, float* scales_t, void* ws,
                            void* stream) {
  if (!p) return MOE_ERR_INVALID_ARG;
  moe_status_t s = validate_quant_out(p->rows, p->G, offsets, p->f, p->ld, p->pow2, codes, scales,
                                      codes_t, scales_t, ws);
  if (s != MOE_OK) return s;
  if (p->rows == 0) return MOE_OK;
  if (!ptrs_ok(ab)) return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_fp8_quant(act_args(FP8_SRC_SWIGLU, p, nullptr, ab, offsets, codes,
                                               scales, codes_t, scales_t, ws),
                                      static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_fp8_swiglu_bwd(const moe_fp8_act_t* p, const void* dh, const void* ab,
                                const int32_t* offsets, void* codes, float* scales, void* codes_t,
                                float* scales_t, void* h_codes_t, float* h_scales_t, void* ws,
                                void* stream) {
  if (!p) return MOE_ERR_INVALID_ARG;
  moe_status_t s = validate_dim(p->f);
  if (s == MOE_OK)
    s = validate_quant_out(p->rows, p->G, offsets, 2 * static_cast<int64_t>(p->f), p->ld, p->pow2,
                           codes, scales, codes_t, scales_t, ws);
  if (s != MOE_OK) return s;
  if (p->rows == 0) return MOE_OK;
  if (!ptrs_ok(dh, ab, codes) || !pair_ok(h_codes_t, h_scales_t, true) || (h_codes_t && !codes_t))
    return MOE_ERR_INVALID_ARG;
  Fp8QuantArgs a = act_args(FP8_SRC_SWIGLU_BWD, p, dh, ab, offsets, codes, scales, codes_t,
                            scales_t, ws);
  a.h_codes_t = h_codes_t;
  a.h_scales_t = h_scales_t;
  return cuda_status(launch_fp8_quant(a, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_fp8_gemm(const moe_fp8_gemm_t* g, const void* a, const float* a_scales,
                          const void* b, const float* b_scales, const int32_t* offsets, void* out,
                          void* ws, void* stream) {
  if (!g) return MOE_ERR_INVALID_ARG;
  moe_status_t s = validate_segments(g->rows, g->G, offsets);
  if (s == MOE_OK) s = validate_dim(g->N);
  if (s == MOE_OK) s = validate_dim(g->K);
  if (s != MOE_OK) return s;
  const bool fp32 = g->out_type == MOE_OUT_FP32;
  if ((!fp32 && g->out_type != MOE_OUT_BF16) || !ld_ok(g->lda, g->K) || !ld_ok(g->ldb, g->K) ||
      g->ldo < g->N)
    return MOE_ERR_INVALID_ARG;
  if (g->rows == 0) return MOE_OK;
  if (!ptrs_ok(a, a_scales, b, b_scales, ws) || !out ||
      (reinterpret_cast<uintptr_t>(out) & (fp32 ? 3u : 1u)))
    return MOE_ERR_INVALID_ARG;
  // tile coordinates are 32-bit: every tile's first weight row
  if (static_cast<int64_t>(g->G) * g->N >= FP8_MAX_ROWS) return MOE_ERR_UNSUPPORTED;
  const int64_t tiles = (g->rows / 128 + g->G) * ((g->N + 127) / 128);
  if (tiles >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;
  Fp8GemmArgs x{};
  x.rows = g->rows;
  x.G = g->G;
  x.N = g->N;
  x.K = g->K;
  x.a = a;
  x.a_scales = a_scales;
  x.lda = g->lda;
  x.b = b;
  x.b_scales = b_scales;
  x.ldb = g->ldb;
  x.offsets = offsets;
  x.out = out;
  x.ldo = g->ldo;
  x.out_fp32 = fp32;
  x.err = static_cast<int*>(ws);
  return cuda_status(launch_fp8_gemm(x, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_fp8_wgrad(const moe_fp8_wgrad_t* g, const void* a, const float* a_scales,
                           const void* b, const float* b_scales, const int32_t* offsets, void* dW,
                           void* ws, void* stream) {
  if (!g) return MOE_ERR_INVALID_ARG;
  moe_status_t s = validate_segments(g->rows, g->G, offsets);
  if (s == MOE_OK) s = validate_dim(g->M);
  if (s == MOE_OK) s = validate_dim(g->N);
  if (s != MOE_OK) return s;
  const bool fp32 = g->out_type == MOE_OUT_FP32;
  if ((!fp32 && g->out_type != MOE_OUT_BF16) || !ptrs_ok(a, a_scales, b, b_scales, dW, ws))
    return MOE_ERR_INVALID_ARG;
  const int64_t tiles = static_cast<int64_t>(g->G) * ((g->M + 127) / 128) * ((g->N + 127) / 128);
  // 32-bit tile counts and positions along the tokens
  if (tiles >= (int64_t(1) << 31) || 128 * fp8_token_blocks(g->rows, g->G) >= (int64_t(1) << 31))
    return MOE_ERR_UNSUPPORTED;
  Fp8GemmArgs x{};
  x.wgrad = true;
  x.rows = g->rows;
  x.G = g->G;
  x.N = g->N;
  x.K = g->M;
  x.a = a;
  x.a_scales = a_scales;
  x.b = b;
  x.b_scales = b_scales;
  x.offsets = offsets;
  x.out = dW;
  x.ldo = g->N;
  x.out_fp32 = fp32;
  x.err = static_cast<int*>(ws);
  return cuda_status(launch_fp8_gemm(x, static_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------- normalisation and 8-bit checkpoints of rows
static bool row_type_ok(int32_t t) { return t == MOE_OUT_BF16 || t == MOE_OUT_FP32; }
static bool format_ok(int32_t f) { return f == MOE_CKPT_INT8 || f == MOE_CKPT_E4M3; }
// rows that may be strided: aligned to their elements
static bool rows_ok(const void* p, int64_t ld, int64_t C, int32_t type) {
  return p && reinterpret_cast<uintptr_t>(p) % (type == MOE_OUT_FP32 ? 4 : 2) == 0 && ld >= C;
}
static bool opt_ok(const void* p) { return !p || aligned16(p); }

// what every call checks of its sizes; rows = 0 passes
static moe_status_t validate_rows(int64_t rows, int64_t C) {
  if (rows < 0 || C < 1) return MOE_ERR_INVALID_ARG;
  return rows >= FP8_MAX_ROWS || C >= FP8_MAX_DIM ? MOE_ERR_UNSUPPORTED : MOE_OK;
}
static moe_status_t validate_norm(const moe_norm_t* p) {
  if (!p) return MOE_ERR_INVALID_ARG;
  const moe_status_t s = validate_rows(p->rows, p->C);
  if (s != MOE_OK) return s;
  if ((p->kind != MOE_NORM_LAYER && p->kind != MOE_NORM_RMS) || !row_type_ok(p->x_type) ||
      !row_type_ok(p->y_type) || !row_type_ok(p->p_type) || !row_type_ok(p->g_type) ||
      !format_ok(p->format))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}
static NormArgs norm_args(const moe_norm_t* p) {
  NormArgs a{};
  a.rows = p->rows;
  a.ldx = p->ldx;
  a.ld_add = p->ld_add;
  a.ld_y = p->ld_y;
  a.ld_out = p->ld_out;
  a.ld_codes = p->ld_codes;
  a.C = p->C;
  a.blocks = (p->C + 127) / 128;
  a.kind = p->kind;
  a.format = p->format;
  a.src_type = a.x_type = p->x_type;
  a.y_type = p->y_type;
  a.p_type = p->p_type;
  a.g_type = p->g_type;
  a.eps = p->eps;
  return a;
}

moe_status_t moe_norm(const moe_norm_t* p, const void* x, const void* residual, const void* gamma,
                      const void* beta, void* y, void* total, float* mean, float* rstd, void* codes,
                      float* scales, void* stream) {
  const moe_status_t s = validate_norm(p);
  if (s != MOE_OK) return s;
  if (!std::isfinite(p->eps) || p->eps < 0.0f) return MOE_ERR_INVALID_ARG;
  if (p->rows == 0) return MOE_OK;
  if (!rows_ok(x, p->ldx, p->C, p->x_type) || !rows_ok(y, p->ld_y, p->C, p->y_type) ||
      (residual && !rows_ok(residual, p->ld_add, p->C, p->x_type)) ||
      (total && (!residual || !rows_ok(total, p->ld_out, p->C, p->x_type))) || !opt_ok(gamma) ||
      !opt_ok(beta) || !opt_ok(mean) || !opt_ok(rstd) || (mean && p->kind == MOE_NORM_RMS) ||
      !pair_ok(codes, scales, true) || (codes && !ld_ok(p->ld_codes, p->C)))
    return MOE_ERR_INVALID_ARG;
  NormArgs a = norm_args(p);
  a.x = x;
  a.add = residual;
  a.gamma = gamma;
  a.beta = beta;
  a.y = y;
  a.out = total;
  a.mean = mean;
  a.rstd = rstd;
  a.codes = codes;
  a.scales = scales;
  return cuda_status(launch_norm(a, static_cast<cudaStream_t>(stream)));
}

int64_t moe_norm_ws_size(int64_t rows, int32_t C) {
  if (validate_rows(rows, C) != MOE_OK) return -1;
  const int64_t parts = rows < NORM_PARTS ? rows : NORM_PARTS;
  return static_cast<int64_t>(WS_HEADER_BYTES) + parts * norm_part_floats(C) * 4;
}

moe_status_t moe_norm_bwd(const moe_norm_t* p, const void* dy, const void* x, const float* x_scales,
                          const float* mean, const float* rstd, const void* gamma, const void* add,
                          void* dx, void* dgamma, void* dbeta, void* ws, void* stream) {
  const moe_status_t s = validate_norm(p);
  if (s != MOE_OK) return s;
  if (!opt_ok(dgamma) || !opt_ok(dbeta)) return MOE_ERR_INVALID_ARG;
  const bool layer = p->kind == MOE_NORM_LAYER;
  if (p->rows > 0) {
    if (!rows_ok(dy, p->ld_y, p->C, p->y_type) || !rows_ok(dx, p->ld_out, p->C, p->x_type) ||
        (add && !rows_ok(add, p->ld_add, p->C, p->x_type)) || !opt_ok(gamma) || !ptrs_ok(rstd, ws) ||
        (layer ? !ptrs_ok(mean) : mean != nullptr))
      return MOE_ERR_INVALID_ARG;
    if (x_scales ? !ptrs_ok(x, x_scales) || !ld_ok(p->ld_codes, p->C)
                 : !rows_ok(x, p->ldx, p->C, p->x_type))
      return MOE_ERR_INVALID_ARG;
  } else if (!dgamma && !dbeta) {
    return MOE_OK;
  }
  NormArgs a = norm_args(p);
  a.x = x;
  if (x_scales) {
    a.src_type = code_type(p->format);
    a.ldx = p->ld_codes;
    a.x_scales = x_scales;
  }
  a.y = const_cast<void*>(dy);
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.gamma = gamma;
  a.add = add;
  a.out = dx;
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  a.part = ws ? at<float>(ws, WS_HEADER_BYTES) : nullptr;
  a.err = static_cast<int*>(ws);
  return cuda_status(launch_norm_bwd(a, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_ckpt_norm(const moe_norm_t* p, const void* codes, const float* scales,
                           const float* mean, const float* rstd, const void* gamma,
                           const void* beta, void* y, void* stream) {
  const moe_status_t s = validate_norm(p);
  if (s != MOE_OK) return s;
  if (p->rows == 0) return MOE_OK;
  if (!ptrs_ok(codes, scales, rstd) || !ld_ok(p->ld_codes, p->C) ||
      (p->kind == MOE_NORM_LAYER ? !ptrs_ok(mean) : mean != nullptr) || !opt_ok(gamma) ||
      !opt_ok(beta) || !rows_ok(y, p->ld_y, p->C, p->y_type))
    return MOE_ERR_INVALID_ARG;
  NormArgs a = norm_args(p);
  a.x = codes;
  a.src_type = code_type(p->format);
  a.ldx = p->ld_codes;
  a.x_scales = scales;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.gamma = gamma;
  a.beta = beta;
  a.y = y;
  return cuda_status(launch_ckpt_norm(a, static_cast<cudaStream_t>(stream)));
}

static moe_status_t validate_ckpt(const moe_ckpt_rows_t* p, const int32_t* live) {
  if (!p) return MOE_ERR_INVALID_ARG;
  const moe_status_t s = validate_rows(p->rows, p->C);
  if (s != MOE_OK) return s;
  if (!format_ok(p->format) || !row_type_ok(p->x_type) ||
      (reinterpret_cast<uintptr_t>(live) & 3u) || !ld_ok(p->ld, p->C))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}
static CkptArgs ckpt_args(const moe_ckpt_rows_t* p, const int32_t* live, void* ws) {
  CkptArgs a{};
  a.live = live;
  a.rows = p->rows;
  a.ldx = p->ldx;
  a.ld = p->ld;
  a.C = p->C;
  a.blocks = (p->C + 127) / 128;
  a.format = p->format;
  a.x_type = p->x_type;
  a.err = static_cast<int*>(ws);
  return a;
}

moe_status_t moe_ckpt_save(const moe_ckpt_rows_t* p, const void* x, const int32_t* live, void* codes,
                           float* scales, void* ws, void* stream) {
  const moe_status_t s = validate_ckpt(p, live);
  if (s != MOE_OK || p->rows == 0) return s;
  if (!rows_ok(x, p->ldx, p->C, p->x_type) || !ptrs_ok(codes, scales, ws))
    return MOE_ERR_INVALID_ARG;
  CkptArgs a = ckpt_args(p, live, ws);
  a.x = x;
  a.codes = codes;
  a.scales = scales;
  return cuda_status(launch_ckpt_save(a, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_ckpt_load(const moe_ckpt_rows_t* p, const void* codes, const float* scales,
                           const int32_t* live, void* x, void* ws, void* stream) {
  const moe_status_t s = validate_ckpt(p, live);
  if (s != MOE_OK || p->rows == 0) return s;
  if (!rows_ok(x, p->ldx, p->C, p->x_type) || !ptrs_ok(codes, scales, ws))
    return MOE_ERR_INVALID_ARG;
  CkptArgs a = ckpt_args(p, live, ws);
  a.codes_in = codes;
  a.scales_in = scales;
  a.out = x;
  return cuda_status(launch_ckpt_load(a, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_ckpt_swiglu(const moe_ckpt_rows_t* p, const void* codes, const float* scales,
                             const int32_t* live, void* ab, void* h, void* ws, void* stream) {
  const moe_status_t s = validate_ckpt(p, live);
  if (s != MOE_OK) return s;
  if (p->C % 2) return MOE_ERR_INVALID_ARG;
  if (p->rows == 0) return MOE_OK;
  if (!ptrs_ok(codes, scales, ws) || (!ab && !h) || !opt_ok(ab) || !opt_ok(h))
    return MOE_ERR_INVALID_ARG;
  CkptArgs a = ckpt_args(p, live, ws);
  a.codes_in = codes;
  a.scales_in = scales;
  a.out = ab;
  a.h = h;
  return cuda_status(launch_ckpt_swiglu(a, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_ckpt_swiglu_bwd(const moe_ckpt_rows_t* p, const void* dh, const void* codes,
                                 const float* scales, const int32_t* live, void* dab, void* h,
                                 void* ws, void* stream) {
  const moe_status_t s = validate_ckpt(p, live);
  if (s != MOE_OK) return s;
  if (p->C % 2) return MOE_ERR_INVALID_ARG;
  if (p->rows == 0) return MOE_OK;
  if (!ptrs_ok(dh, codes, scales, dab, ws) || !opt_ok(h)) return MOE_ERR_INVALID_ARG;
  CkptArgs a = ckpt_args(p, live, ws);
  a.dh = dh;
  a.codes_in = codes;
  a.scales_in = scales;
  a.out = dab;
  a.h = h;
  return cuda_status(launch_ckpt_swiglu(a, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_ckpt_combine_bwd(const moe_config_t* cfg, const void* dy, const void* codes,
                                  int64_t ld, const float* scales, int32_t format,
                                  const float* topk_w, const int32_t* dest_row, void* dyp, float* dw,
                                  void* ws, void* stream) {
  const moe_status_t s = validate(cfg);
  if (s != MOE_OK) return s;
  if (!format_ok(format) || !ld_ok(ld, cfg->d) ||
      !ptrs_ok(dy, codes, scales, topk_w, dest_row, dyp, dw, ws))
    return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_ckpt_combine_bwd(dy, codes, ld, scales, format, topk_w, dest_row, cfg->T,
                                             cfg->k, cfg->d, cfg->T * cfg->k, dyp, dw,
                                             static_cast<int*>(ws),
                                             static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
