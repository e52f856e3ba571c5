// ckpt.cu -- activations held in 8 bits from the forward to the backward pass: saving rows,
// restoring them, the SwiGLU's gradient and the combine's gradient from them.
//
// A checkpoint is one code a value and one fp32 scale for each block of 128 along the row
// (rows8.cuh).  Everything here is memory's: 3 bytes a value to save bf16 rows or to restore them,
// 10 a column of the SwiGLU's gradient, 3 a value of the combine's.
#include <type_traits>

#include "rows8.cuh"

namespace moe {
namespace {

constexpr int THREADS = 256, WARPS = THREADS / 32;

__device__ __forceinline__ int64_t live_rows(const CkptArgs& a) {
  if (!a.live) return a.rows;
  const int64_t n = *a.live;
  if (n < 0 || n > a.rows) {
    if (blockIdx.x == 0 && threadIdx.x == 0) flag_error(a.err, MOE_DEVERR_BAD_OFFSETS);
    return n < 0 ? 0 : a.rows;
  }
  return n;
}

// Save: a warp takes N chunks of 256 columns, going on over the rows' ends.
template <int V, int N, int X, int FORMAT>
__global__ void __launch_bounds__(THREADS)
save_kernel(const __grid_constant__ CkptArgs a, RowDiv div) {
  griddep_wait();   // see common.cuh: dependent launches
  const int lane = threadIdx.x & 31;
  const int64_t items = live_rows(a) * div.per;
  const int64_t step = static_cast<int64_t>(gridDim.x) * WARPS * N;
  constexpr int XS = X == ROW_BF16 ? 2 : 4;
  for (int64_t i0 = (static_cast<int64_t>(blockIdx.x) * WARPS + (threadIdx.x >> 5)) * N; i0 < items;
       i0 += step) {
    int64_t row = div.row(i0);
    int k = static_cast<int>(i0 - row * div.per);
    Raw8 raw[N];
    void* codes[N];
    float* scales[N];
    int chunk[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      chunk[i] = i0 + i < items ? k * CHUNK : a.C;   // (a chunk that starts at C has no columns)
      load_raw<V>(raw[i], static_cast<const uint8_t*>(a.x) + row * a.ldx * XS, X, chunk[i], a.C, lane);
      codes[i] = static_cast<uint8_t*>(a.codes) + row * a.ld;
      scales[i] = a.scales + row * a.blocks;
      if (++k == div.per) { k = 0; ++row; }
    }
    float f[N][8];
#pragma unroll
    for (int i = 0; i < N; ++i) unpack_raw<V>(raw[i], X, f[i]);
    save_chunks<V, N>(codes, scales, FORMAT, chunk, a.C, lane, f);
  }
  griddep_launch();
}

template <int V, int N, int X, int FORMAT>
__global__ void __launch_bounds__(THREADS)
load_kernel(const __grid_constant__ CkptArgs a, RowDiv div) {
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t items = live_rows(a) * div.per;
  const int64_t step = static_cast<int64_t>(gridDim.x) * WARPS * N;
  constexpr int XS = X == ROW_BF16 ? 2 : 4, TYPE = FORMAT == MOE_CKPT_INT8 ? ROW_INT8 : ROW_E4M3;
  for (int64_t i0 = (static_cast<int64_t>(blockIdx.x) * WARPS + (threadIdx.x >> 5)) * N; i0 < items;
       i0 += step) {
    int64_t row = div.row(i0);
    int k = static_cast<int>(i0 - row * div.per);
    Raw8 raw[N];
    float sc[N][8 / V];
    uint8_t* out[N];
    int chunk[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      out[i] = static_cast<uint8_t*>(a.out) + row * a.ldx * XS;
      chunk[i] = i0 + i < items ? k * CHUNK : a.C;
      load_raw<V>(raw[i], static_cast<const uint8_t*>(a.codes_in) + row * a.ld, TYPE, chunk[i], a.C,
                  lane);
      load_scales<V>(sc[i], a.scales_in + row * a.blocks, 0, chunk[i], a.C, lane);
      if (++k == div.per) { k = 0; ++row; }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float f[8];
      unpack_raw<V>(raw[i], TYPE, f);
      scale_values<V>(f, sc[i]);
      store_values<V>(out[i], X, chunk[i], a.C, lane, f);
    }
  }
  griddep_launch();
}

// [a | b] and h, or with BACK [da | db] and h from dh: f = C / 2 columns, a warp takes N chunks of
// 256 of them.  With s = sigma(a): h = a s b, da = dh b s (1 + a (1 - s)), db = dh a s, from the
// 32-bit restored values, each rounded once.
template <int V, int N, bool BACK, int TYPE>
__global__ void __launch_bounds__(THREADS)
swiglu_kernel(const __grid_constant__ CkptArgs p, RowDiv div) {
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int f = p.C / 2;
  const int64_t items = live_rows(p) * div.per;
  const int64_t step = static_cast<int64_t>(gridDim.x) * WARPS * N;
  for (int64_t i0 = (static_cast<int64_t>(blockIdx.x) * WARPS + (threadIdx.x >> 5)) * N; i0 < items;
       i0 += step) {
    int64_t row = div.row(i0);
    int k = static_cast<int>(i0 - row * div.per);
    Raw8 ra[N], rb[N], rd[N];
    float sa[N][8 / V], sb[N][8 / V];
    int64_t at[N];
    int chunk[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      at[i] = row;
      chunk[i] = k * CHUNK;
      if (i0 + i < items) {
        const uint8_t* codes = static_cast<const uint8_t*>(p.codes_in) + row * p.ld;
        const float* scales = p.scales_in + row * p.blocks;
        load_raw<V>(ra[i], codes, TYPE, chunk[i], f, lane);
        load_raw<V>(rb[i], codes + f, TYPE, chunk[i], f, lane);
        if (BACK)
          load_raw<V>(rd[i], static_cast<const __nv_bfloat16*>(p.dh) + row * f, ROW_BF16, chunk[i],
                      f, lane);
        load_scales<V>(sa[i], scales, 0, chunk[i], f, lane);
        load_scales<V>(sb[i], scales, f, chunk[i], f, lane);
      }
      if (++k == div.per) { k = 0; ++row; }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i0 + i >= items) break;
      float a[8], b[8], h[8];
      unpack_raw<V>(ra[i], TYPE, a);
      unpack_raw<V>(rb[i], TYPE, b);
      scale_values<V>(a, sa[i]);
      scale_values<V>(b, sb[i]);
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + at[i] * p.C;
      if (BACK) {
        float d[8];
        unpack_raw<V>(rd[i], ROW_BF16, d);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float s = sigmoid_fast(a[j]), as = a[j] * s;
          const float da = d[j] * b[j] * fmaf(as, 1.0f - s, s);
          h[j] = as * b[j];
          b[j] = d[j] * as;
          a[j] = da;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = a[j] * sigmoid_fast(a[j]) * b[j];
      }
      if (p.out) {
        store_values<V>(out, ROW_BF16, chunk[i], f, lane, a);
        store_values<V>(out + f, ROW_BF16, chunk[i], f, lane, b);
      }
      if (p.h)
        store_values<V>(static_cast<__nv_bfloat16*>(p.h) + at[i] * f, ROW_BF16, chunk[i], f, lane, h);
    }
  }
  griddep_launch();
}

// One warp per token: dyp[p_j] = w_j dy[t], dw_j = <dy[t], codes * scales of row p_j>; 0 for a
// dropped slot.  The codes of a lane's eight columns are summed before the block's scale
// multiplies them.
template <int KMAX, int TYPE>
__global__ void __launch_bounds__(THREADS)
combine_bwd_kernel(const uint4* __restrict__ dy, const uint8_t* __restrict__ codes, int64_t ld,
                   const float* __restrict__ scales, int blocks, const float* __restrict__ topk_w,
                   const int32_t* __restrict__ dest_row, int64_t T, int k, int d, int64_t rows_cap,
                   uint4* __restrict__ dyp, float* __restrict__ dw, int* err) {
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int nvec = d / 8;
  const int64_t gw = (static_cast<int64_t>(blockIdx.x) * THREADS + threadIdx.x) >> 5;
  const int64_t nw = (static_cast<int64_t>(gridDim.x) * THREADS) >> 5;
  for (int64_t t = gw; t < T; t += nw) {
    int my_p = -1;
    float my_w = 0.0f;
    if (lane < k) {
      my_p = dest_row[t * k + lane];
      my_w = topk_w[t * k + lane];
      if (my_p >= rows_cap || my_p < -1) {
        flag_error(err, MOE_DEVERR_BAD_INDEX);
        my_p = -1;
      }
    }
    int64_t p[KMAX];
    float wt[KMAX], dot[KMAX];
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
      p[j] = __shfl_sync(FULL_MASK, my_p, j);
      wt[j] = __shfl_sync(FULL_MASK, my_w, j);
      if (j >= k) p[j] = -1;
      dot[j] = 0.0f;
    }
    for (int c = lane; c < nvec; c += 32) {
      const uint4 g = dy[t * nvec + c];
      uint2 v[KMAX];
      float sc[KMAX];
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if (p[j] >= 0) {
          v[j] = *reinterpret_cast<const uint2*>(codes + p[j] * ld + 8 * c);
          sc[j] = scales[p[j] * blocks + (c >> 4)];
        }
      float gf[8];
      unpack8(g, gf);
#pragma unroll
      for (int j = 0; j < KMAX; ++j)
        if (p[j] >= 0) {
          Raw8 raw;
          raw.w[0] = v[j].x;
          raw.w[1] = v[j].y;
          float f[8], o[8], s = 0.0f;
          unpack_raw<8>(raw, TYPE, f);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            s = fmaf(gf[q], f[q], s);
            o[q] = wt[j] * gf[q];
          }
          dot[j] = fmaf(s, sc[j], dot[j]);
          dyp[p[j] * nvec + c] = pack8(o);
        }
    }
    float mine = 0.0f;
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
      dot[j] = warp_sum(dot[j]);
      if (j == lane) mine = dot[j];
    }
    if (lane < k) dw[t * k + lane] = mine;
  }
  griddep_launch();
}

int sm_count() {
  int dev = 0, sms = 152;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

// f(the rows' type, the format) as constants
template <typename F>
cudaError_t by_types(const CkptArgs& a, F f) {
  using Bf16 = std::integral_constant<int, ROW_BF16>;
  using Fp32 = std::integral_constant<int, ROW_FP32>;
  using Int8 = std::integral_constant<int, MOE_CKPT_INT8>;
  using E4m3 = std::integral_constant<int, MOE_CKPT_E4M3>;
  if (a.x_type == ROW_BF16) return a.format == MOE_CKPT_INT8 ? f(Bf16(), Int8()) : f(Bf16(), E4m3());
  return a.format == MOE_CKPT_INT8 ? f(Fp32(), Int8()) : f(Fp32(), E4m3());
}

dim3 item_grid(int64_t rows, int per, int n) {
  const int64_t need = (rows * per + WARPS * n - 1) / (WARPS * n);
  const int64_t most = static_cast<int64_t>(1) << 30;
  return dim3(static_cast<unsigned>(need < most ? need : most));
}

}  // namespace

cudaError_t launch_ckpt_save(const CkptArgs& a, cudaStream_t st) {
  const RowDiv div((a.C + CHUNK - 1) / CHUNK);
  const int xs = row_size(a.x_type);
  auto go = [&](auto kern, int n) {
    return launch_pdl(kern, item_grid(a.rows, div.per, n), dim3(THREADS), 0, st, 1, a, div);
  };
  auto pick = [&](auto x, auto format) {
    constexpr int X = decltype(x)::value, F = decltype(format)::value;
    if (a.C % 8 == 0 && rows_fit(a.x, a.ldx, xs, 8)) return go(save_kernel<8, 4, X, F>, 4);
    if (a.C % 2 == 0 && rows_fit(a.x, a.ldx, xs, 2)) return go(save_kernel<2, 2, X, F>, 2);
    return go(save_kernel<1, 2, X, F>, 2);
  };
  return by_types(a, pick);
}

cudaError_t launch_ckpt_load(const CkptArgs& a, cudaStream_t st) {
  const RowDiv div((a.C + CHUNK - 1) / CHUNK);
  const int xs = row_size(a.x_type);
  auto go = [&](auto kern, int n) {
    return launch_pdl(kern, item_grid(a.rows, div.per, n), dim3(THREADS), 0, st, 1, a, div);
  };
  auto pick = [&](auto x, auto format) {
    constexpr int X = decltype(x)::value, F = decltype(format)::value;
    if (a.C % 8 == 0 && rows_fit(a.out, a.ldx, xs, 8)) return go(load_kernel<8, 4, X, F>, 4);
    if (a.C % 2 == 0 && rows_fit(a.out, a.ldx, xs, 2)) return go(load_kernel<2, 2, X, F>, 2);
    return go(load_kernel<1, 2, X, F>, 2);
  };
  return by_types(a, pick);
}

cudaError_t launch_ckpt_swiglu(const CkptArgs& a, cudaStream_t st) {
  const int f = a.C / 2;
  const RowDiv div((f + CHUNK - 1) / CHUNK);
  auto go = [&](auto kern, int n) {
    return launch_pdl(kern, item_grid(a.rows, div.per, n), dim3(THREADS), 0, st, 1, a, div);
  };
  auto pick = [&](auto back, auto format) {
    constexpr bool B = decltype(back)::value;
    constexpr int T = decltype(format)::value == MOE_CKPT_INT8 ? ROW_INT8 : ROW_E4M3;
    // (dh, [a | b] and h are dense from 16-byte addresses: the width alone decides)
    if (f % 8 == 0) return go(swiglu_kernel<8, 2, B, T>, 2);
    if (f % 2 == 0) return go(swiglu_kernel<2, 1, B, T>, 1);
    return go(swiglu_kernel<1, 1, B, T>, 1);
  };
  using Int8 = std::integral_constant<int, MOE_CKPT_INT8>;
  using E4m3 = std::integral_constant<int, MOE_CKPT_E4M3>;
  if (a.dh)
    return a.format == MOE_CKPT_INT8 ? pick(std::true_type(), Int8()) : pick(std::true_type(), E4m3());
  return a.format == MOE_CKPT_INT8 ? pick(std::false_type(), Int8()) : pick(std::false_type(), E4m3());
}

cudaError_t launch_ckpt_combine_bwd(const void* dy, const void* codes, int64_t ld,
                                    const float* scales, int format, const float* topk_w,
                                    const int32_t* dest_row, int64_t T, int k, int d,
                                    int64_t rows_cap, void* dyp, float* dw, int* err,
                                    cudaStream_t st) {
  const int64_t need = (T + WARPS - 1) / WARPS, cap = static_cast<int64_t>(sm_count()) * 8;
  const dim3 grid(static_cast<unsigned>(need < cap ? need : cap));
#define MOE_COMBINE_T(KM, TY)                                                                   \
  launch_pdl(combine_bwd_kernel<KM, TY>, grid, dim3(THREADS), 0, st, 1,                         \
             static_cast<const uint4*>(dy), static_cast<const uint8_t*>(codes), ld, scales,      \
             (d + 127) / 128, topk_w, dest_row, T, k, d, rows_cap, static_cast<uint4*>(dyp), dw, \
             err)
#define MOE_COMBINE(KM) \
  (format == MOE_CKPT_INT8 ? MOE_COMBINE_T(KM, ROW_INT8) : MOE_COMBINE_T(KM, ROW_E4M3))
  if (k <= 2) return MOE_COMBINE(2);
  if (k <= 4) return MOE_COMBINE(4);
  if (k <= 6) return MOE_COMBINE(6);
  return MOE_COMBINE(8);
#undef MOE_COMBINE
#undef MOE_COMBINE_T
}

}  // namespace moe
