// fp8.cu -- 8-bit operands with one scale for each block of 128: quantising rows (along the
// row, and along the tokens of each expert's segment), weights (128 x 128 blocks), and the
// SwiGLU and its backward, which quantise their own output.
//
// A block's scale is s = amax / 448 with amax = max(max |v|, 2^-110) (448: the largest E4M3
// number; the floor keeps s a normal number and an all-zero block finite), or with pow2 the
// next power of two at or above it; its codes are E4M3(v * r), r = 448 / amax (or 1 / s, exact
// with pow2), rounded to nearest, ties to even, saturated at 448.  Both quotients and the
// product are single correctly rounded fp32 operations, so the codes are the same bits
// whatever kernel writes them: the rounding to 4 significant bits is the only one that
// matters.  A NaN in a block makes the whole block NaN, an infinity makes the others 0.
//
// All kernels are bound by memory: a bf16 value is read once (2 bytes) and one byte or, with
// both orientations, two bytes are written.
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int FQ_THREADS = 256;
constexpr int FQ_MAX_G = 256;
constexpr float E4M3_TOP = 448.0f;
constexpr float AMAX_FLOOR = 0x1p-110f;

__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {   // a in the low byte
  return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE,
                                                        __NV_E4M3));
}

// Scale and factor of a block from the bits of its largest magnitude (bf16, so that NaN > inf
// > every number in the bits' order).
__device__ __forceinline__ void block_scale(uint32_t amax_bf16, int pow2, float& s, float& r) {
  float a = __uint_as_float(amax_bf16 << 16);
  if (a < AMAX_FLOOR) a = AMAX_FLOOR;
  if (!pow2 || !(a < INFINITY)) {
    s = __fdiv_rn(a, E4M3_TOP);
    r = __fdiv_rn(E4M3_TOP, a);
  } else {
    // 448 = 1.75 * 2^8: the exponent of a less 8, and one more where a's fraction is above
    const uint32_t u = __float_as_uint(a);
    const int n = static_cast<int>(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    s = __uint_as_float(static_cast<uint32_t>(n) << 23);
    r = __uint_as_float(static_cast<uint32_t>(254 - n) << 23);
  }
}

__device__ __forceinline__ uint32_t max_mag2(uint32_t m, uint32_t w) {
  return __vmaxu2(m, w & 0x7fff7fffu);
}
__device__ __forceinline__ uint32_t max_mag8(const uint4& v) {
  uint32_t m = max_mag2(v.x & 0x7fff7fffu, v.y);
  m = max_mag2(m, v.z);
  return max_mag2(m, v.w);
}
__device__ __forceinline__ uint32_t fold2(uint32_t m) {   // the larger of the two halves
  const uint32_t hi = m >> 16, lo = m & 0xffffu;
  return hi > lo ? hi : lo;
}
__device__ __forceinline__ uint2 codes8(const uint4& v, float r) {
  float f[8];
  unpack8(v, f);
  return make_uint2(e4m3x2(f[0] * r, f[1] * r) | (e4m3x2(f[2] * r, f[3] * r) << 16),
                    e4m3x2(f[4] * r, f[5] * r) | (e4m3x2(f[6] * r, f[7] * r) << 16));
}

// ------------------------------------------------------------------ SwiGLU values
// h = silu(a) b and its derivatives are rounded to bf16 once from their exact value, so that
// codes and scales do not depend on how a kernel groups the arithmetic: the fp32 value is
// computed with a known error bound, and where both ends of the bound do not round to the same
// bf16 number (1 value in about 6000) it is computed again in 64 bits.
__device__ __noinline__ float silu_mul_exact(float a, float b) {
  const double x = static_cast<double>(a);
  return __double2float_rn(x * (1.0 / (1.0 + exp(-x))) * static_cast<double>(b));
}
__device__ __noinline__ float dsilu_mul_exact(float a, float b, float dh) {
  const double x = static_cast<double>(a);
  const double sg = 1.0 / (1.0 + exp(-x));
  return __double2float_rn(static_cast<double>(dh) * static_cast<double>(b) * sg *
                           (1.0 + x * (1.0 / (1.0 + exp(x)))));
}

// Two values and the bounds of their errors -> packed bf16; bit i of `open` set where value i
// is not settled (its bound crosses a rounding border, it is tiny, infinite or NaN).
__device__ __forceinline__ uint32_t settle2(float v0, float e0, float v1, float e1, int& open) {
  const uint32_t hi = pack_bf16x2(v0 + e0, v1 + e1), lo = pack_bf16x2(v0 - e0, v1 - e1);
  const uint32_t d = (hi ^ lo) & 0x7fff7fffu;   // an exact zero may change its sign in v + 0
  auto fits = [](float v, float e) { return (e >= 0x1p-120f && e < INFINITY) || v == 0.0f; };
  open = ((d & 0xffffu) || !fits(v0, e0) ? 1 : 0) | ((d >> 16) || !fits(v1, e1) ? 2 : 0);
  return lo;
}

// silu(a) b = a b / (1 + e^-a): a b is exact (two 8-bit significands), expf is off by at most
// one ulp (2^-23), the sum by 2^-24, the fast quotient by two ulp (2^-22): 1.75 * 2^-22.
constexpr float SILU_ERR = 0x1p-21f;
// silu'(a) = s (1 + a (1 - s)), s = 1 / (1 + t), 1 - s = t s: with u = a t s and g = 1 + u the
// error is below |s| (|u| + |g|) 2.75 * 2^-22 (t 2^-23; s 1.75 * 2^-22; four roundings).
constexpr float DSILU_ERR = 0x1.8p-21f;

__device__ __forceinline__ uint32_t silu_mul2(uint32_t a, uint32_t b) {
  const float a0 = bf16_lo(a), a1 = bf16_hi(a), b0 = bf16_lo(b), b1 = bf16_hi(b);
  const float v0 = __fdividef(a0 * b0, 1.0f + expf(-a0));
  const float v1 = __fdividef(a1 * b1, 1.0f + expf(-a1));
  int open;
  uint32_t w = settle2(v0, fabsf(v0) * SILU_ERR, v1, fabsf(v1) * SILU_ERR, open);
  if (a0 < -80.0f) open |= 1;   // the exponential's and the quotient's range
  if (a1 < -80.0f) open |= 2;
  if (open) {
    const float x0 = (open & 1) ? silu_mul_exact(a0, b0) : bf16_lo(w);
    const float x1 = (open & 2) ? silu_mul_exact(a1, b1) : bf16_hi(w);
    w = pack_bf16x2(x0, x1);
  }
  return w;
}
__device__ __forceinline__ uint4 silu_mul8(const uint4& a, const uint4& b) {
  return make_uint4(silu_mul2(a.x, b.x), silu_mul2(a.y, b.y), silu_mul2(a.z, b.z),
                    silu_mul2(a.w, b.w));
}
__device__ __forceinline__ uint32_t dsilu_mul2(uint32_t a, uint32_t b, uint32_t dh) {
  float v[2], e[2], fa[2], fb[2], fd[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    fa[i] = i ? bf16_hi(a) : bf16_lo(a);
    fb[i] = i ? bf16_hi(b) : bf16_lo(b);
    fd[i] = i ? bf16_hi(dh) : bf16_lo(dh);
    const float t = expf(-fa[i]);
    const float s = __fdividef(1.0f, 1.0f + t);
    const float u = fa[i] * t * s;
    const float g = 1.0f + u;
    const float qs = fd[i] * fb[i] * s;
    v[i] = qs * g;
    e[i] = fabsf(qs) * (fabsf(u) + fabsf(g)) * DSILU_ERR;
  }
  int open;
  uint32_t w = settle2(v[0], e[0], v[1], e[1], open);
  if (fa[0] < -80.0f) open |= 1;
  if (fa[1] < -80.0f) open |= 2;
  if (open) {
    const float x0 = (open & 1) ? dsilu_mul_exact(fa[0], fb[0], fd[0]) : bf16_lo(w);
    const float x1 = (open & 2) ? dsilu_mul_exact(fa[1], fb[1], fd[1]) : bf16_hi(w);
    w = pack_bf16x2(x0, x1);
  }
  return w;
}
__device__ __forceinline__ uint4 dsilu_mul8(const uint4& a, const uint4& b, const uint4& d) {
  return make_uint4(dsilu_mul2(a.x, b.x, d.x), dsilu_mul2(a.y, b.y, d.y),
                    dsilu_mul2(a.z, b.z, d.z), dsilu_mul2(a.w, b.w, d.w));
}

// ------------------------------------------------------------------ sources
// What a quantiser reads: eight consecutive values of a row, as packed bf16; columns at or past
// `cols` are 0.  VEC: every row starts on 16 bytes and a chunk never crosses an end.
enum { SRC_ROWS, SRC_SWIGLU, SRC_SWIGLU_BWD };

struct Source {
  const __nv_bfloat16* x;    // rows: [src_rows][ld]; SwiGLU: ab [rows][2f]
  const __nv_bfloat16* dh;   // backward: [rows][f]
  long long ld;
  int f;
  int cols;                  // columns quantised: C, f, or 2f
  bool h_only;               // backward: the columns are those of h
};

template <bool VEC>
__device__ __forceinline__ uint4 load8(const __nv_bfloat16* p, int n) {
  if constexpr (VEC) {
    return __ldg(reinterpret_cast<const uint4*>(p));
  } else {
    const uint16_t* u = reinterpret_cast<const uint16_t*>(p);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = 2 * i < n ? __ldg(u + 2 * i) : 0u;
      const uint32_t hi = 2 * i + 1 < n ? __ldg(u + 2 * i + 1) : 0u;
      w[i] = lo | (hi << 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <int SRC, bool VEC>
__device__ __forceinline__ uint4 value8(const Source& s, long long row, int c) {
  const int n = s.cols - c;
  if (n <= 0) return make_uint4(0u, 0u, 0u, 0u);
  if constexpr (SRC == SRC_ROWS) {
    return load8<VEC>(s.x + row * s.ld + c, n);
  } else {
    const __nv_bfloat16* ab = s.x + row * 2 * s.f;
    if (SRC == SRC_SWIGLU || s.h_only)
      return silu_mul8(load8<VEC>(ab + c, n), load8<VEC>(ab + s.f + c, n));
    const __nv_bfloat16* dh = s.dh + row * s.f;
    if constexpr (VEC) {
      const bool up = c >= s.f;
      const int k = up ? c - s.f : c;
      const uint4 a = load8<VEC>(ab + k, 8), d = load8<VEC>(dh + k, 8);
      return up ? silu_mul8(a, d) : dsilu_mul8(a, load8<VEC>(ab + s.f + k, 8), d);
    } else {
      // odd widths: the gate's and the up projection's columns may meet inside a chunk
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[i] = 0u;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int cc = c + 2 * i + j;
          if (cc >= s.cols) continue;
          const int k = cc < s.f ? cc : cc - s.f;
          auto bits = [](const __nv_bfloat16* p) {
            return static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(p)));
          };
          const uint32_t a = bits(ab + k), d = bits(dh + k);
          const uint32_t r = cc < s.f ? dsilu_mul2(a, bits(ab + s.f + k), d) : silu_mul2(a, d);
          w[i] |= (r & 0xffffu) << (16 * j);
        }
      }
      return make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

struct QuantOut {
  uint8_t* codes;      // [rows][ld]
  float* scales;       // [rows][kb]
  long long ld;
  int kb;
  uint8_t* codes_t;    // [cols][128 * kb_cap]
  float* scales_t;     // [kb_cap][cols]
  int kb_cap;
  int pow2;
};

__device__ __forceinline__ long long live_rows(const int32_t* offsets, int G, long long rows,
                                               int* err, bool first) {
  if (!offsets) return rows;
  const long long n = offsets[G];
  if (n < 0 || n > rows) {
    if (first) flag_error(err, MOE_DEVERR_BAD_OFFSETS);
    return n < 0 ? 0 : rows;
  }
  return n;
}

// ------------------------------------------------------------------ along the rows
// One warp per row; a lane takes eight values (16 bytes), half a warp a block.  ROW_BATCH
// chunks' loads are issued before any is used.
constexpr int ROW_BATCH = 4;

template <int SRC, bool VEC>
__global__ void __launch_bounds__(FQ_THREADS)
fp8_rows_kernel(const Source src, const int32_t* __restrict__ src_tok, long long src_rows,
                const int32_t* __restrict__ offsets, int G, long long rows, const QuantOut out,
                int* err) {
  griddep_wait();   // see common.cuh: dependent launches
  const int lane = threadIdx.x & 31;
  const long long gw = (static_cast<long long>(blockIdx.x) * FQ_THREADS + threadIdx.x) >> 5;
  const long long nw = (static_cast<long long>(gridDim.x) * FQ_THREADS) >> 5;
  const long long n_rows = live_rows(offsets, G, rows, err, gw == 0 && lane == 0);
  for (long long p = gw; p < n_rows; p += nw) {
    long long t = p;
    if (src_tok) {
      t = __ldg(src_tok + p);
      if (t < 0 || t >= src_rows) {
        if (lane == 0) flag_error(err, MOE_DEVERR_BAD_INDEX);
        continue;
      }
    }
    for (int c0 = 8 * lane; c0 - 8 * lane < src.cols; c0 += 256 * ROW_BATCH) {
      uint4 v[ROW_BATCH];
#pragma unroll
      for (int b = 0; b < ROW_BATCH; ++b) v[b] = value8<SRC, VEC>(src, t, c0 + 256 * b);
#pragma unroll
      for (int b = 0; b < ROW_BATCH; ++b) {
        const int c = c0 + 256 * b;
        uint32_t m = max_mag8(v[b]);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(FULL_MASK, m, o));
        float s, r;
        block_scale(fold2(m), out.pow2, s, r);
        if (c >= src.cols) continue;
        *reinterpret_cast<uint2*>(out.codes + p * out.ld + c) = codes8(v[b], r);
        if ((lane & 15) == 0) out.scales[p * out.kb + (c >> 7)] = s;
      }
    }
  }
  griddep_launch();
}

// ------------------------------------------------------------------ along the tokens (and rows)
// One CTA per 128 columns and 128-row block of a segment (blocks are counted from the
// segment's first row).  The tile goes through shared memory once: its rows are quantised from
// the registers that loaded them, its columns from shared memory, two columns and a quarter of
// the rows per thread, which then owns 32 consecutive codes of each column.
__device__ __forceinline__ uint32_t col_code(const uint32_t* w, int i, bool hi, float r) {
  float f[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = (hi ? bf16_hi(w[4 * i + j]) : bf16_lo(w[4 * i + j])) * r;
  return e4m3x2(f[0], f[1]) | (e4m3x2(f[2], f[3]) << 16);
}

template <int SRC, bool VEC>
__global__ void __launch_bounds__(FQ_THREADS)
fp8_tokens_kernel(const Source src, const int32_t* __restrict__ src_tok, long long src_rows,
                  const int32_t* __restrict__ offsets, int G, long long rows, const QuantOut out,
                  int* err) {
  griddep_wait();   // see common.cuh: dependent launches
  __shared__ uint4 tile[128][16];
  __shared__ uint32_t s_max[4][64];
  __shared__ int s_first[FQ_MAX_G + 1];
  __shared__ int s_sum[8];
  __shared__ int s_bad;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool first = blockIdx.x == 0 && blockIdx.y == 0;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  auto start_of = [&](int g) {
    return offsets ? static_cast<long long>(offsets[g]) : (g ? rows : 0LL);
  };
  // first block of every segment (G <= 256: one per thread)
  int nb = 0;
  if (tid < G) {
    const long long a = start_of(tid), b = start_of(tid + 1);
    if (a < 0 || b < a || b > rows || (tid == 0 && a != 0)) s_bad = 1;
    else nb = static_cast<int>((b - a + 127) / 128);
  }
  const int incl = warp_incl_scan(nb);
  if (lane == 31) s_sum[warp] = incl;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < warp; ++w) before += s_sum[w];
  if (tid < G) s_first[tid] = before + incl - nb;
  if (tid == G - 1) s_first[G] = before + incl;
  __syncthreads();
  if (s_bad) {
    if (first && tid == 0) flag_error(err, MOE_DEVERR_BAD_OFFSETS);
    return;
  }
  const int total = s_first[G];
  const int c0 = blockIdx.x * 128;
  for (int kb = blockIdx.y; kb < total; kb += gridDim.y) {
    int lo = 0, hi = G;   // s_first[lo] <= kb < s_first[lo + 1]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_first[mid] <= kb) lo = mid;
      else hi = mid;
    }
    const long long r0 = start_of(lo) + 128LL * (kb - s_first[lo]);
    const long long left = start_of(lo + 1) - r0;
    const int nr = left < 128 ? static_cast<int>(left) : 128;
    uint4 v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int r = (tid >> 4) + 16 * u, c = c0 + 8 * (tid & 15);
      v[u] = make_uint4(0u, 0u, 0u, 0u);
      if (r < nr) {
        long long t = r0 + r;
        if (src_tok) {
          t = __ldg(src_tok + t);
          if (t < 0 || t >= src_rows) {
            flag_error(err, MOE_DEVERR_BAD_INDEX);
            t = 0;
          }
        }
        v[u] = value8<SRC, VEC>(src, t, c);
      }
    }
    __syncthreads();   // the previous block's tile is consumed
#pragma unroll
    for (int u = 0; u < 8; ++u) tile[(tid >> 4) + 16 * u][tid & 15] = v[u];
    if (out.codes && !src.h_only) {
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int r = (tid >> 4) + 16 * u, c = c0 + 8 * (tid & 15);
        uint32_t m = max_mag8(v[u]);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(FULL_MASK, m, o));
        float s, f;
        block_scale(fold2(m), out.pow2, s, f);
        if (r < nr && c < src.cols) {
          *reinterpret_cast<uint2*>(out.codes + (r0 + r) * out.ld + c) = codes8(v[u], f);
          if ((tid & 15) == 0) out.scales[(r0 + r) * out.kb + (c >> 7)] = s;
        }
      }
    }
    __syncthreads();
    // columns c0 + 2 cp, + 1; rows 32 q .. 32 q + 31
    const int cp = tid & 63, q = tid >> 6;
    const uint32_t* words = reinterpret_cast<const uint32_t*>(tile);
    uint32_t w[32];
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      w[i] = words[(32 * q + i) * 64 + cp];
      m = max_mag2(m, w[i]);
    }
    s_max[q][cp] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __vmaxu2(m, s_max[i][cp]);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int c = c0 + 2 * cp + j;
      if (c >= src.cols) continue;
      float s, r;
      block_scale(j ? m >> 16 : m & 0xffffu, out.pow2, s, r);
      uint32_t code[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) code[i] = col_code(w, i, j != 0, r);
      uint4* dst = reinterpret_cast<uint4*>(
          out.codes_t + (static_cast<long long>(c) * out.kb_cap + kb) * 128 + 32 * q);
      dst[0] = make_uint4(code[0], code[1], code[2], code[3]);
      dst[1] = make_uint4(code[4], code[5], code[6], code[7]);
      if (q == 0) out.scales_t[static_cast<long long>(kb) * src.cols + c] = s;
    }
  }
  griddep_launch();
}

// ------------------------------------------------------------------ weights
// One CTA per 128 x 128 block of W [G][N][K]: one scale, the codes row-major and, for the data
// gradient's product, transposed (its block scales transposed with them).
template <bool VEC>
__global__ void __launch_bounds__(FQ_THREADS)
fp8_weights_kernel(const __nv_bfloat16* __restrict__ W, int N, int K, int nb, int kb,
                   uint8_t* __restrict__ codes, long long ld, float* __restrict__ scales,
                   uint8_t* __restrict__ codes_t, long long ld_t, float* __restrict__ scales_t,
                   int pow2) {
  griddep_wait();   // see common.cuh: dependent launches
  __shared__ uint32_t tile[128][33];
  __shared__ uint32_t s_max[8];
  const int tid = threadIdx.x;
  const int kbi = static_cast<int>(blockIdx.x % kb);
  const int k0 = kbi * 128;
  const long long gb = blockIdx.x / kb;       // group * nb + row block
  const long long g = gb / nb;
  const int n0 = static_cast<int>(gb - g * nb) * 128;
  uint4 v[8];
  uint32_t m = 0u;
  const int c = k0 + 8 * (tid & 15);
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int n = n0 + (tid >> 4) + 16 * u;
    v[u] = make_uint4(0u, 0u, 0u, 0u);
    if (n < N && c < K) v[u] = load8<VEC>(W + (g * N + n) * K + c, K - c);
    m = __vmaxu2(m, max_mag8(v[u]));
  }
  m = fold2(m);
  m = __reduce_max_sync(FULL_MASK, m);
  if ((tid & 31) == 0) s_max[tid >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, s_max[i]);
  float s, r;
  block_scale(m, pow2, s, r);
  if (tid == 0) {
    scales[gb * kb + kbi] = s;
    if (codes_t) scales_t[(g * kb + kbi) * nb + n0 / 128] = s;
  }
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int rr = (tid >> 4) + 16 * u;
    const uint2 q = codes8(v[u], r);
    if (n0 + rr < N && c < K)
      *reinterpret_cast<uint2*>(codes + (g * N + n0 + rr) * ld + c) = q;
    tile[rr][2 * (tid & 15)] = q.x;
    tile[rr][2 * (tid & 15) + 1] = q.y;
  }
  if (codes_t) {
    __syncthreads();
    // four columns and sixteen rows a thread: 4 x 4 byte transposes
    const int cq = tid & 31, rg = tid >> 5;
    uint32_t t[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = tile[16 * rg + 4 * i + j][cq];
      const uint32_t a = __byte_perm(w[0], w[1], 0x5140), b = __byte_perm(w[2], w[3], 0x5140);
      const uint32_t d = __byte_perm(w[0], w[1], 0x7362), e = __byte_perm(w[2], w[3], 0x7362);
      t[0][i] = __byte_perm(a, b, 0x5410);
      t[1][i] = __byte_perm(a, b, 0x7632);
      t[2][i] = __byte_perm(d, e, 0x5410);
      t[3][i] = __byte_perm(d, e, 0x7632);
    }
    const int n = n0 + 16 * rg;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = k0 + 4 * cq + j;
      // the padding up to ld_t takes the zero codes of rows past N
      if (k < K && n < N)
        *reinterpret_cast<uint4*>(codes_t + (g * K + k) * ld_t + n) =
            make_uint4(t[j][0], t[j][1], t[j][2], t[j][3]);
    }
  }
  griddep_launch();
}

int fq_sms() {
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <int SRC, bool VEC>
cudaError_t launch_quant(const Source& s, const Fp8QuantArgs& a, const QuantOut& o, bool tokens,
                         cudaStream_t st) {
  if (!tokens) {
    const long long want = (a.rows + FQ_THREADS / 32 - 1) / (FQ_THREADS / 32);
    const long long most = static_cast<long long>(fq_sms()) * 8;
    return launch_pdl(fp8_rows_kernel<SRC, VEC>, dim3(static_cast<unsigned>(want < most ? want : most)),
                      dim3(FQ_THREADS), 0, st, 1, s, a.src_tok, a.src_rows, a.offsets, a.G, a.rows,
                      o, a.err);
  }
  const unsigned gx = static_cast<unsigned>((s.cols + 127) / 128);
  const long long most = (static_cast<long long>(fq_sms()) * 8 + gx - 1) / gx;
  const long long blocks = fp8_token_blocks(a.rows, a.G);
  return launch_pdl(fp8_tokens_kernel<SRC, VEC>,
                    dim3(gx, static_cast<unsigned>(blocks < most ? blocks : most)),
                    dim3(FQ_THREADS), 0, st, 1, s, a.src_tok, a.src_rows, a.offsets, a.G, a.rows, o,
                    a.err);
}

}  // namespace

cudaError_t launch_fp8_quant(const Fp8QuantArgs& a, cudaStream_t st) {
  Source s{};
  s.x = static_cast<const __nv_bfloat16*>(a.x);
  s.dh = static_cast<const __nv_bfloat16*>(a.dh);
  s.ld = a.ldx;
  s.f = a.f;
  s.cols = a.src == FP8_SRC_ROWS ? a.C : a.src == FP8_SRC_SWIGLU ? a.f : 2 * a.f;
  QuantOut o{};
  o.codes = static_cast<uint8_t*>(a.codes);
  o.scales = a.scales;
  o.ld = a.ld;
  o.kb = (s.cols + 127) / 128;
  o.codes_t = static_cast<uint8_t*>(a.codes_t);
  o.scales_t = a.scales_t;
  o.kb_cap = static_cast<int>(fp8_token_blocks(a.rows, a.G));
  o.pow2 = a.pow2;
  const bool tokens = a.codes_t != nullptr;
  if (a.src == FP8_SRC_ROWS) {
    const bool vec = on16(a.x) && a.ldx % 8 == 0 && a.C % 8 == 0;
    return vec ? launch_quant<SRC_ROWS, true>(s, a, o, tokens, st)
               : launch_quant<SRC_ROWS, false>(s, a, o, tokens, st);
  }
  const bool vec = a.f % 8 == 0;
  if (a.src == FP8_SRC_SWIGLU)
    return vec ? launch_quant<SRC_SWIGLU, true>(s, a, o, tokens, st)
               : launch_quant<SRC_SWIGLU, false>(s, a, o, tokens, st);
  const cudaError_t e = vec ? launch_quant<SRC_SWIGLU_BWD, true>(s, a, o, tokens, st)
                            : launch_quant<SRC_SWIGLU_BWD, false>(s, a, o, tokens, st);
  if (e != cudaSuccess || !a.h_codes_t) return e;
  s.h_only = true;
  s.cols = a.f;
  o.codes = nullptr;
  o.codes_t = static_cast<uint8_t*>(a.h_codes_t);
  o.scales_t = a.h_scales_t;
  return vec ? launch_quant<SRC_SWIGLU_BWD, true>(s, a, o, true, st)
             : launch_quant<SRC_SWIGLU_BWD, false>(s, a, o, true, st);
}

cudaError_t launch_fp8_weights(const void* W, int G, int N, int K, void* codes, int64_t ld,
                               float* scales, void* codes_t, int64_t ld_t, float* scales_t,
                               int pow2, cudaStream_t st) {
  const int nb = (N + 127) / 128, kb = (K + 127) / 128;
  const dim3 grid(static_cast<unsigned>(static_cast<long long>(G) * nb * kb));
  auto go = [&](auto kern) {
    return launch_pdl(kern, grid, dim3(FQ_THREADS), 0, st, 1, static_cast<const __nv_bfloat16*>(W),
                      N, K, nb, kb, static_cast<uint8_t*>(codes), ld, scales,
                      static_cast<uint8_t*>(codes_t), ld_t, scales_t, pow2);
  };
  return on16(W) && K % 8 == 0 ? go(fp8_weights_kernel<true>) : go(fp8_weights_kernel<false>);
}

}  // namespace moe
