// norm_bwd.cu -- gradient of the layer norm and the root-mean-square norm (formulas: norm.cu),
// from the rows or from their 8-bit checkpoint.
//
// A row is read once (dy and v), its two sums are taken over the threads that hold it, and dv is
// written.  Every thread keeps the same columns for all the rows of its CTA, so the sums over the
// rows for dgamma and dbeta stay in its registers until the end; the CTAs' sums go to the
// workspace and a second launch adds them in a fixed order: no atomics, the same bits every time.
// Where a copy reaches 6.79 TB/s:
//   16,384 x 4096 bf16, with add                 5.9 TB/s, 90 us: about 5 of it the sums' launch; sixteen
//                                                warps to an SM, which the sums' registers hold, wait for
//                                                shared memory and one another
//   the same from int8 codes                     4.9 TB/s, 96 us: as above, and the codes' conversion
//   8191 x 1413, E4M3 codes, fp32 stream         3.6 TB/s, 35 us: instructions, an element at a time
#include "rows8.cuh"

namespace moe {
namespace {

// v -> xhat of a chunk
template <int V>
__device__ __forceinline__ void xhat_values(float* x, const Raw8& raw, const float* sc,
                                            const NormArgs& a, float mean, float rstd) {
  unpack_raw<V>(raw, a.src_type, x);
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = (a.x_scales ? fmaf(x[j], sc[j / V], -mean) : x[j] - mean) * rstd;
}

// Rows of more columns than stay in registers, and bf16 rows with fp32 gradients: two passes over the
// row, and the sums over the CTA's rows in its part of the workspace.
template <int V>
__global__ void __launch_bounds__(32 * MAX_WARPS)
norm_bwd_wide_kernel(const __grid_constant__ NormArgs a) {
  griddep_wait();
  __shared__ RowSums sh;
  row_sum_init(sh);
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
        c = row_sum2(c1, c2, sh, turn, warp, nw);
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
    // (a bf16 stream with fp32 gradients, which no layer here makes, goes the wide rows' way at any width:
    // two passes over a row and the sums through memory, 383 us for 16,384 x 4096 where bf16 gradients
    // take 91, and 1276 us for 40 M elements of 256 columns, where an fp32 stream takes 101)
    if (chunks <= 4 * MAX_WARPS && (a.x_type == ROW_FP32 || a.y_type == ROW_BF16)) {
      e = a.x_type == ROW_BF16 ? launch_norm_bwd_bf16(a, v, chunks, st, &parts)
          : v == 8             ? launch_norm_bwd_fp32(a, chunks, st, &parts)
                               : launch_norm_bwd_fp32_odd(a, chunks, st, &parts);
    } else {
      parts = static_cast<int>(a.rows < 2 * row_sms() ? a.rows : 2 * row_sms());
      if (parts > NORM_PARTS) parts = NORM_PARTS;
      const dim3 grid(parts), block(32 * (chunks < MAX_WARPS ? chunks : MAX_WARPS));
      e = v == 8   ? launch_pdl(norm_bwd_wide_kernel<8>, grid, block, 0, st, 1, a)
          : v == 2 ? launch_pdl(norm_bwd_wide_kernel<2>, grid, block, 0, st, 1, a)
                   : launch_pdl(norm_bwd_wide_kernel<1>, grid, block, 0, st, 1, a);
    }
    if (e != cudaSuccess) return e;
  }
  if (!sums) return e;
  return launch_pdl(norm_sum_kernel, dim3((a.C + 31) / 32, 2), dim3(32, SUM_ROWS), 0, st, 1, a.part,
                    parts, norm_part_floats(a.C) / 2, a.C, a.dgamma, a.dbeta, a.g_type);
}

}  // namespace moe
