// norm_bwd.cu -- gradient of the layer norm and the root-mean-square norm (formulas: norm.cu),
// from the rows or from their 8-bit checkpoint.
//
// A row is read once (dy and v), its two sums are taken over the threads that hold it, and dv is
// written.  Every thread keeps the same columns for all the rows of its CTA, so the sums over the
// rows for dgamma and dbeta stay in its registers until the end; the CTAs' sums go to the
// workspace and a second launch adds them in a fixed order: no atomics, the same bits every time.
#include "rows8.cuh"

namespace moe {
namespace {

constexpr int MAX_WARPS = 16;

struct Shared {
  float2 part[2][MAX_WARPS];
};

__device__ __forceinline__ const void* row_at(const void* p, int64_t row, int64_t ld, int size) {
  return static_cast<const uint8_t*>(p) + row * ld * size;
}
__device__ __forceinline__ void* row_at(void* p, int64_t row, int64_t ld, int size) {
  return static_cast<uint8_t*>(p) + row * ld * size;
}

// Sums over the warps of a row; one barrier, `turn` alternates from row to row.
__device__ __forceinline__ float2 row_sum(float a, float b, Shared& sh, int turn, int warp, int nw) {
  a = warp_sum(a);
  b = warp_sum(b);
  if (nw == 1) return make_float2(a, b);
  if ((threadIdx.x & 31) == 0) sh.part[turn][warp] = make_float2(a, b);
  __syncthreads();
  float sa = 0.0f, sb = 0.0f;
  for (int i = 0; i < nw; ++i) {
    const float2 p = sh.part[turn][i];
    sa += p.x;
    sb += p.y;
  }
  return make_float2(sa, sb);
}

// v -> xhat of a chunk
template <int V>
__device__ __forceinline__ void xhat_values(float* x, const Raw8& raw, const float* sc,
                                            const NormArgs& a, float mean, float rstd) {
  unpack_raw<V>(raw, a.src_type, x);
  if (a.x_scales) scale_values<V>(x, sc);
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = (x[j] - mean) * rstd;
}

// nw warps share a row, N chunks to a warp; with nw = 1 the CTA's warps have rows of their own.
template <int V, int N>
__global__ void __launch_bounds__(32 * MAX_WARPS)
norm_bwd_kernel(const __grid_constant__ NormArgs a, int nw) {
  griddep_wait();   // see common.cuh: dependent launches
  __shared__ Shared sh;
  extern __shared__ float columns[];   // with nw = 1: the warps' sums over the rows
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int w = nw == 1 ? 0 : warp;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (nw == 1 ? blockDim.x >> 5 : 1);
  const int xs = row_size(a.x_type), ys = row_size(a.y_type), ss = row_size(a.src_type);
  const float over = 1.0f / static_cast<float>(a.C);
  float dg[N][8], db[N][8];
  int chunk[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    chunk[i] = (i * nw + w) * CHUNK;
#pragma unroll
    for (int j = 0; j < 8; ++j) dg[i][j] = db[i][j] = 0.0f;
  }
  int turn = 0;
  for (int64_t row = nw == 1 ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + warp : blockIdx.x;
       row < a.rows; row += step) {
    const void* xr = row_at(a.x, row, a.ldx, ss);
    const void* yr = row_at(static_cast<const void*>(a.y), row, a.ld_y, ys);
    const void* ar = a.add ? row_at(a.add, row, a.ld_add, xs) : nullptr;
    Raw8 x[N], y[N], ad[N];
    float sc[N][8 / V];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      load_raw<V>(y[i], yr, a.y_type, chunk[i], a.C, lane);
      load_raw<V>(x[i], xr, a.src_type, chunk[i], a.C, lane);
      if (a.x_scales) load_scales<V>(sc[i], a.x_scales + row * a.blocks, 0, chunk[i], a.C, lane);
    }
    if (ar) {
#pragma unroll
      for (int i = 0; i < N; ++i) load_raw<V>(ad[i], ar, a.x_type, chunk[i], a.C, lane);
    }
    const float mean = a.kind == MOE_NORM_LAYER ? a.mean[row] : 0.0f;
    const float rstd = a.rstd[row];
    float c1 = 0.0f, c2 = 0.0f;
    float xh[N][8], g[N][8];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      unpack_raw<V>(y[i], a.y_type, g[i]);
      xhat_values<V>(xh[i], x[i], sc[i], a, mean, rstd);
      float p[8];
      if (a.gamma) load_values<V>(p, a.gamma, a.p_type, chunk[i], a.C, lane);
      float s = 0.0f, t = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // (past the row's end dy is 0, and so is everything that it multiplies)
        dg[i][j] = fmaf(g[i][j], xh[i][j], dg[i][j]);
        db[i][j] += g[i][j];
        if (a.gamma) g[i][j] *= p[j];
        s += g[i][j];
        t = fmaf(g[i][j], xh[i][j], t);
      }
      c1 += s;
      c2 += t;
    }
    const float2 c = row_sum(c1, c2, sh, turn, w, nw);
    turn ^= 1;
    c1 = a.kind == MOE_NORM_LAYER ? c.x * over : 0.0f;
    c2 = c.y * over;
    void* dr = row_at(a.out, row, a.ld_out, xs);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float d[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = rstd * (g[i][j] - c1 - xh[i][j] * c2);
      if (ar) {
        float p[8];
        unpack_raw<V>(ad[i], a.x_type, p);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] += p[j];
      }
      store_values<V>(dr, a.x_type, chunk[i], a.C, lane, d);
    }
  }
  griddep_launch();
  if (!a.part) return;
  const int64_t wide = norm_part_floats(a.C) / 2;
  float* mine = a.part + 2 * wide * blockIdx.x;
  if (nw == 1) {
    // the warps' sums one after another, so that their order is fixed
    for (int k = 0; k < static_cast<int>(blockDim.x >> 5); ++k) {
      if (warp == k) {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int c = i * CHUNK + 32 * j + lane;
            if (k > 0) {
              dg[i][j] += columns[c];
              db[i][j] += columns[N * CHUNK + c];
            }
            columns[c] = dg[i][j];
            columns[N * CHUNK + c] = db[i][j];
          }
      }
      __syncthreads();
    }
    if (warp + 1 != static_cast<int>(blockDim.x >> 5)) return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    store_values<V>(mine, ROW_FP32, chunk[i], a.C, lane, dg[i]);
    store_values<V>(mine + wide, ROW_FP32, chunk[i], a.C, lane, db[i]);
  }
}

// Rows of more columns than stay in registers: two passes over the row, and the sums over the
// CTA's rows in its part of the workspace.
template <int V>
__global__ void __launch_bounds__(32 * MAX_WARPS)
norm_bwd_wide_kernel(const __grid_constant__ NormArgs a) {
  griddep_wait();
  __shared__ Shared sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int xs = row_size(a.x_type), ys = row_size(a.y_type), ss = row_size(a.src_type);
  const float over = 1.0f / static_cast<float>(a.C);
  const int64_t wide = norm_part_floats(a.C) / 2;
  float* mine = a.part ? a.part + 2 * wide * blockIdx.x : nullptr;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const void* xr = row_at(a.x, row, a.ldx, ss);
    const void* yr = row_at(static_cast<const void*>(a.y), row, a.ld_y, ys);
    const float mean = a.kind == MOE_NORM_LAYER ? a.mean[row] : 0.0f;
    const float rstd = a.rstd[row];
    float c1 = 0.0f, c2 = 0.0f;
    float2 c;
    for (int pass = 0; pass < 2; ++pass) {
      for (int k = warp * CHUNK; k < a.C; k += nw * CHUNK) {
        Raw8 x, y;
        float sc[8 / V], g[8], xh[8], p[8];
        load_raw<V>(y, yr, a.y_type, k, a.C, lane);
        load_raw<V>(x, xr, a.src_type, k, a.C, lane);
        if (a.x_scales) load_scales<V>(sc, a.x_scales + row * a.blocks, 0, k, a.C, lane);
        unpack_raw<V>(y, a.y_type, g);
        xhat_values<V>(xh, x, sc, a, mean, rstd);
        if (pass == 0 && mine) {
          float s[8], t[8];
          const bool first = row == blockIdx.x;
          load_values<V>(s, mine, ROW_FP32, k, a.C, lane);
          load_values<V>(t, mine + wide, ROW_FP32, k, a.C, lane);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            s[j] = first ? g[j] * xh[j] : fmaf(g[j], xh[j], s[j]);
            t[j] = first ? g[j] : t[j] + g[j];
          }
          store_values<V>(mine, ROW_FP32, k, a.C, lane, s);
          store_values<V>(mine + wide, ROW_FP32, k, a.C, lane, t);
        }
        if (a.gamma) {
          load_values<V>(p, a.gamma, a.p_type, k, a.C, lane);
#pragma unroll
          for (int j = 0; j < 8; ++j) g[j] *= p[j];
        }
        if (pass == 0) {
          float s = 0.0f, t = 0.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            s += g[j];
            t = fmaf(g[j], xh[j], t);
          }
          c1 += s;
          c2 += t;
          continue;
        }
        float d[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = rstd * (g[j] - c.x - xh[j] * c.y);
        if (a.add) {
          load_values<V>(p, row_at(a.add, row, a.ld_add, xs), a.x_type, k, a.C, lane);
#pragma unroll
          for (int j = 0; j < 8; ++j) d[j] += p[j];
        }
        store_values<V>(row_at(a.out, row, a.ld_out, xs), a.x_type, k, a.C, lane, d);
      }
      if (pass == 0) {
        c = row_sum(c1, c2, sh, turn, warp, nw);
        turn ^= 1;
        c.x = a.kind == MOE_NORM_LAYER ? c.x * over : 0.0f;
        c.y *= over;
      }
    }
  }
  griddep_launch();
}

// dgamma and dbeta from the CTAs' sums: 32 columns to a CTA, blockIdx.y says which of the two.
constexpr int SUM_ROWS = 16;
__global__ void __launch_bounds__(32 * SUM_ROWS)
norm_sum_kernel(const float* part, int parts, int64_t wide, int C, void* dgamma, void* dbeta,
                int type) {
  griddep_wait();
  __shared__ float sh[SUM_ROWS][33];
  void* out = blockIdx.y ? dbeta : dgamma;
  const int c = blockIdx.x * 32 + threadIdx.x;
  float s = 0.0f;
  if (out && c < C) {
    const float* p = part + (blockIdx.y ? wide : 0) + c;
#pragma unroll 4
    for (int i = threadIdx.y; i < parts; i += SUM_ROWS) s += p[2 * wide * i];
  }
  sh[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && out && c < C) {
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < SUM_ROWS; ++i) s += sh[i][threadIdx.x];
    if (type == ROW_FP32) static_cast<float*>(out)[c] = s;
    else static_cast<__nv_bfloat16*>(out)[c] = __float2bfloat16_rn(s);
  }
  griddep_launch();
}

int sm_count() {
  int dev = 0, sms = 152;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

}  // namespace

cudaError_t launch_norm_bwd(const NormArgs& in, cudaStream_t st) {
  NormArgs a = in;
  const bool sums = a.dgamma || a.dbeta;
  if (!sums) a.part = nullptr;
  const int chunks = (a.C + CHUNK - 1) / CHUNK;
  const int v = norm_vector(a);
  cudaError_t e = cudaSuccess;
  int parts = 0;
  if (a.rows > 0) {
    const bool wide = chunks > 4 * MAX_WARPS;
    const int n = chunks == 1 ? 1 : chunks <= 2 * MAX_WARPS ? 2 : 4;
    const int nw = chunks <= 2 ? 1 : (chunks + n - 1) / n;
    const int warps = wide ? MAX_WARPS : nw == 1 ? 4 : nw;
    const int64_t ctas = nw == 1 ? (a.rows + 3) / 4 : a.rows;
    int64_t cap = static_cast<int64_t>(sm_count()) * (warps > 8 ? 1 : 16 / warps);
    if (cap > NORM_PARTS) cap = NORM_PARTS;
    parts = static_cast<int>(ctas < cap ? ctas : cap);
    const dim3 grid(parts), block(32 * warps);
    const size_t smem = nw == 1 ? static_cast<size_t>(2) * n * CHUNK * 4 : 0;
#define MOE_NORM(V, N) launch_pdl(norm_bwd_kernel<V, N>, grid, block, smem, st, 1, a, nw)
#define MOE_NORM_N(V)                                                                \
  (wide ? launch_pdl(norm_bwd_wide_kernel<V>, grid, block, 0, st, 1, a)              \
        : n == 1 ? MOE_NORM(V, 1) : n == 2 ? MOE_NORM(V, 2) : MOE_NORM(V, 4))
    e = v == 8 ? MOE_NORM_N(8) : v == 2 ? MOE_NORM_N(2) : MOE_NORM_N(1);
#undef MOE_NORM_N
#undef MOE_NORM
    if (e != cudaSuccess) return e;
  }
  if (!sums) return e;
  return launch_pdl(norm_sum_kernel, dim3((a.C + 31) / 32, 2), dim3(32, SUM_ROWS), 0, st, 1, a.part,
                    parts, norm_part_floats(a.C) / 2, a.C, a.dgamma, a.dbeta, a.g_type);
}

}  // namespace moe
