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
  __shared__ RowSums sh;
  row_sum_init(sh);
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
    const float2 c = row_sum2(c1, c2, sh, turn, w, nw);
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

// The same for rows of whole 16-byte vectors.  dy, v and add of the rows that follow come into
// shared memory by bulk copies while one is worked on; the statistics and a chunk's scale are loaded
// a row ahead.  With nw > 1 thread 0 copies for the CTA: when all have passed the barrier in a row's
// sums, all are done with the row before, whose slot is filled again.  With nw = 1 lane 0 copies for
// its warp.  gamma lies in shared memory too (but for the widest rows, which leave it no room): from
// L1, which the slots leave little of, it came from L2 for every row, and 16384 x 4096 took 107 us
// instead of 90.  With up to two chunks to a warp a row's G and xhat stay in registers between the two
// passes over it, with four they are computed again, from the slot.  S: the type of v or its codes,
// X: of add and dx, Y: of dy.
constexpr int MAX_SLOTS = 4;
constexpr long long BULK_BUDGET = 4000000000LL;   // clock cycles (about 2 s)

template <int N, int S, int X, int Y>
__global__ void __launch_bounds__(N == 1 ? 256 : 32 * MAX_WARPS, N == 1 ? 3 : 1)
norm_bwd_ring_kernel(const __grid_constant__ NormArgs a, int nw, int slots) {
  __shared__ RowSums sh;
  __shared__ __align__(8) uint64_t full[MAX_WARPS][MAX_SLOTS];
  __shared__ int gave_up;
  extern __shared__ __align__(16) uint8_t ring[];
  constexpr bool KEEP = N < 4, GAMMA = N < 4, CODES = S == ROW_INT8 || S == ROW_E4M3;
  constexpr int XS = X == ROW_BF16 ? 2 : 4, YS = Y == ROW_BF16 ? 2 : 4;
  constexpr int SS = CODES ? 1 : S == ROW_BF16 ? 2 : 4;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int w = nw == 1 ? 0 : warp, own = nw == 1 ? warp : 0;
  const bool copies = nw == 1 ? lane == 0 : threadIdx.x == 0;
  if (copies)
    for (int s = 0; s < slots; ++s) mbar_init(smem_u32(&full[own][s]), 1);
  if (threadIdx.x == 0) gave_up = 0;
  fence_mbar_init();
  row_sum_init(sh);
  griddep_wait();   // see common.cuh: dependent launches
  // (32 bits hold every row and the few steps past the last one)
  const uint32_t rows = static_cast<uint32_t>(a.rows), step = gridDim.x * (nw == 1 ? warps : 1);
  const uint32_t first = nw == 1 ? blockIdx.x * warps + warp : blockIdx.x;
  const float over = 1.0f / static_cast<float>(a.C);
  const bool layer = a.kind == MOE_NORM_LAYER, add = a.add != nullptr;
  // a slot: dy, v, add, each a whole row and up to 16 bytes
  const int y_bytes = a.C * YS, x_bytes = (a.C * SS + 15) / 16 * 16, a_bytes = add ? a.C * XS : 0;
  const int slot_bytes = y_bytes + x_bytes + a_bytes;
  uint8_t* const gam = ring + warp * N * 1024;   // each thread's gamma in fp32, then the slots
  uint8_t* const mine = ring + (GAMMA ? warps * N * 1024 : 0) + own * slots * slot_bytes;
  auto at = [](const void* p, uint32_t row, int64_t ld) {
    return static_cast<const uint8_t*>(p) + static_cast<int64_t>(row) * ld;
  };
  uint32_t odd = 0, started = 0;   // of the copying thread: slots filled an odd number of times, ever
  auto fetch = [&](uint32_t row, int slot) {
    if (*static_cast<volatile int*>(&gave_up)) return;
    odd ^= 1u << slot;
    started |= 1u << slot;
    const uint32_t bar = smem_u32(&full[own][slot]), to = smem_u32(mine + slot * slot_bytes);
    mbar_arrive_expect_tx(bar, slot_bytes);
    bulk_load(to, at(a.y, row, a.ld_y * YS), y_bytes, bar);
    bulk_load(to + y_bytes, at(a.x, row, a.ldx * SS), x_bytes, bar);
    if (add) bulk_load(to + y_bytes + x_bytes, at(a.add, row, a.ld_add * XS), a_bytes, bar);
  };
  if (copies)
    for (int s = 0; s < (slots > 1 ? slots - 1 : 1); ++s)
      if (first + s * step < rows) fetch(first + s * step, s);
  float2 dg[N][4], db[N][4];
  int col[N];
  float sc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    col[i] = (i * nw + w) * CHUNK + 8 * lane;
    sc[i] = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) dg[i][j] = db[i][j] = both(0.0f);
  }
  float mean = 0.0f, rstd = 0.0f;
  auto small = [&](uint32_t row) {
    if (layer) mean = a.mean[row];
    rstd = a.rstd[row];
    if (CODES) {
      const float* sr = a.x_scales + static_cast<int64_t>(row) * a.blocks;
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (col[i] < a.C) sc[i] = sr[col[i] >> 7];
    }
  };
  // G and xhat of a chunk in a slot; past the row's end zeros
  auto values = [&](const uint8_t* t, int i, float2 st, float scale, float2* g, float2* xh, bool sums) {
    if (col[i] >= a.C) {
#pragma unroll
      for (int j = 0; j < 4; ++j) g[j] = xh[j] = both(0.0f);
      return;
    }
    float2 p[4];
    smem_row_values<Y>(g, t, col[i]);
    smem_row_values<S>(xh, t + y_bytes, col[i]);
    if (GAMMA) slot_values(p, gam + i * 1024, ROW_FP32, lane);
    else if (a.gamma) vector_values(p, a.gamma, a.p_type, col[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (CODES) xh[j] = __fmul2_rn(xh[j], both(scale));
      xh[j] = __fmul2_rn(__fadd2_rn(xh[j], both(-st.x)), both(st.y));
      if (sums) {
        dg[i][j] = __ffma2_rn(g[j], xh[j], dg[i][j]);
        db[i][j] = __fadd2_rn(db[i][j], g[j]);
      }
      if (GAMMA || a.gamma) g[j] = __fmul2_rn(g[j], p[j]);
    }
  };
  if (GAMMA)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float2 p[4] = {both(1.0f), both(1.0f), both(1.0f), both(1.0f)};
      if (a.gamma && col[i] < a.C) vector_values(p, a.gamma, a.p_type, col[i]);
      *reinterpret_cast<float4*>(gam + i * 1024 + 16 * lane) = make_float4(p[0].x, p[0].y, p[1].x, p[1].y);
      *reinterpret_cast<float4*>(gam + i * 1024 + 512 + 16 * lane) = make_float4(p[2].x, p[2].y, p[3].x, p[3].y);
    }
  if (first < rows) small(first);
  int slot = 0, turn = 0;
  uint32_t phase = 0;
  for (uint32_t row = first; row < rows; row += step) {
    const float2 st = make_float2(mean, rstd);
    float s0[N];
#pragma unroll
    for (int i = 0; i < N; ++i) s0[i] = sc[i];
    if (row + step < rows) small(row + step);
    // (one that gives up goes on, so that the barriers below stay whole: the error word says so)
    mbar_wait_bounded(smem_u32(&full[own][slot]), phase, &gave_up, a.err, BULK_BUDGET);
    const uint8_t* from = mine + slot * slot_bytes;
    float2 g[KEEP ? N : 1][4], xh[KEEP ? N : 1][4], c1 = both(0.0f), c2 = both(0.0f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int k = KEEP ? i : 0;
      values(from, i, st, s0[i], g[k], xh[k], true);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        c1 = __fadd2_rn(c1, g[k][j]);
        c2 = __ffma2_rn(g[k][j], xh[k][j], c2);
      }
    }
    const float2 c = row_sum2(c1.x + c1.y, c2.x + c2.y, sh, turn, w, nw);
    turn ^= 1;
    if (nw == 1) __syncwarp();
    if (copies) {
      // the slot of the row before is free; with one slot it is this row's, filled below
      const uint32_t next = row + (slots - 1) * step;
      if (slots > 1 && next < rows) fetch(next, slot == 0 ? slots - 1 : slot - 1);
    }
    const float m1 = layer ? -c.x * over : 0.0f, m2 = -c.y * over;
    uint8_t* dr = const_cast<uint8_t*>(at(a.out, row, a.ld_out * XS));
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int k = KEEP ? i : 0;
      if (!KEEP) values(from, i, st, s0[i], g[k], xh[k], false);
      if (col[i] >= a.C) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        g[k][j] = __fmul2_rn(__ffma2_rn(xh[k][j], both(m2), __fadd2_rn(g[k][j], both(m1))), both(st.y));
      if (add) {
        float2 p[4];
        smem_row_values<X>(p, from + y_bytes + x_bytes, col[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) g[k][j] = __fadd2_rn(g[k][j], p[j]);
      }
      store_pairs(dr, X, col[i], g[k]);
    }
    if (slots == 1) {
      if (nw == 1) __syncwarp();
      else __syncthreads();
      if (copies && row + step < rows) fetch(row + step, 0);
    }
    if (++slot == slots) {
      slot = 0;
      phase ^= 1;
    }
  }
  if (copies && *static_cast<volatile int*>(&gave_up)) {
    // a copy may still be under way: this CTA's shared memory is not left to it
    const long long t0 = clock64();
    for (int s = 0; s < slots; ++s)
      if (started >> s & 1)
        while (!mbar_try_wait(smem_u32(&full[own][s]), (odd >> s & 1) ^ 1) && clock64() - t0 < BULK_BUDGET / 4) {
        }
  }
  griddep_launch();
  if (!a.part) return;
  const int64_t wide = norm_part_floats(a.C) / 2;
  float* out = a.part + 2 * wide * blockIdx.x;
  if (nw == 1) {
    // the warps' sums one after another, so that their order is fixed (every copy has been waited
    // for: none was started for rows past the last one)
    float2* cols = reinterpret_cast<float2*>(ring);
    __syncthreads();
    for (int k = 0; k < warps; ++k) {
      if (warp == k) {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float2* p = cols + (i * 4 + j) * 64 + lane;
            if (k > 0) {
              dg[i][j] = __fadd2_rn(dg[i][j], p[0]);
              db[i][j] = __fadd2_rn(db[i][j], p[32]);
            }
            p[0] = dg[i][j];
            p[32] = db[i][j];
          }
      }
      __syncthreads();
    }
    if (warp + 1 != warps) return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (col[i] >= a.C) continue;
    store_pairs(out, ROW_FP32, col[i], dg[i]);
    store_pairs(out + wide, ROW_FP32, col[i], db[i]);
  }
}

// Rows of more columns than stay in registers: two passes over the row, and the sums over the
// CTA's rows in its part of the workspace.
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

template <int N, int S, int X, int Y>
cudaError_t launch_ring(const NormArgs& a, int nw, cudaStream_t st, int* parts) {
  constexpr auto kern = norm_bwd_ring_kernel<N, S, X, Y>;
  const int warps = nw == 1 ? 8 : nw;
  const int row = a.C * row_size(Y) + (a.C * row_size(S) + 15) / 16 * 16 + (a.add ? a.C * row_size(X) : 0);
  const int slot = nw == 1 ? warps * row : row, least = nw == 1 ? 2 * N * CHUNK * 4 : 0;
  const int gam = N < 4 ? warps * N * 1024 : 0;
  // CTAs to an SM by registers, then as many slots as their shared memory allows
  int per = ctas_by_registers<kern>(32 * warps);
  if (per > NORM_PARTS / 152) per = NORM_PARTS / 152;
  while (per > 1 && per * (2 * slot + gam) > ROW_SMEM) --per;
  int slots = MAX_SLOTS;
  while (slots > 1 && per * (slots * slot + gam) > ROW_SMEM) --slots;
  const int smem = (slots * slot > least ? slots * slot : least) + gam;
  if (smem > 47 * 1024) {   // (the kernel has a little of its own)
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  const int64_t ctas = nw == 1 ? (a.rows + warps - 1) / warps : a.rows;
  int64_t most = static_cast<int64_t>(row_sms()) * per;
  if (most > NORM_PARTS) most = NORM_PARTS;
  *parts = static_cast<int>(ctas < most ? ctas : most);
  return launch_pdl(kern, dim3(*parts), dim3(32 * warps), smem, st, 1, a, nw, slots);
}
template <int S, int X, int Y>
cudaError_t launch_rows(const NormArgs& a, int chunks, cudaStream_t st, int* parts) {
  if (chunks == 1) return launch_ring<1, S, X, Y>(a, 1, st, parts);
  if (chunks <= 2 * MAX_WARPS) return launch_ring<2, S, X, Y>(a, (chunks + 1) / 2, st, parts);
  return launch_ring<4, S, X, Y>(a, (chunks + 3) / 4, st, parts);
}
// the types of a stream in bf16, or in fp32 with gradients of either type
template <int S, int X>
cudaError_t launch_stream(const NormArgs& a, int chunks, cudaStream_t st, int* parts) {
  if constexpr (X == ROW_FP32)
    if (a.y_type == ROW_FP32) return launch_rows<S, X, ROW_FP32>(a, chunks, st, parts);
  return launch_rows<S, X, ROW_BF16>(a, chunks, st, parts);
}
template <int X>
cudaError_t launch_source(const NormArgs& a, int chunks, cudaStream_t st, int* parts) {
  if (a.src_type == ROW_INT8) return launch_stream<ROW_INT8, X>(a, chunks, st, parts);
  if (a.src_type == ROW_E4M3) return launch_stream<ROW_E4M3, X>(a, chunks, st, parts);
  return launch_stream<X, X>(a, chunks, st, parts);
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
    if (v == 8 && !wide && (a.x_type == ROW_FP32 || a.y_type == ROW_BF16)) {
      e = a.x_type == ROW_BF16 ? launch_source<ROW_BF16>(a, chunks, st, &parts)
                               : launch_source<ROW_FP32>(a, chunks, st, &parts);
    } else {
    const int n = chunks == 1 ? 1 : chunks <= 2 * MAX_WARPS ? 2 : 4;
    const int nw = chunks <= 2 ? 1 : (chunks + n - 1) / n;
    const int warps = wide ? MAX_WARPS : nw == 1 ? 4 : nw;
    const int64_t ctas = nw == 1 ? (a.rows + 3) / 4 : a.rows;
    int64_t cap = static_cast<int64_t>(row_sms()) * (warps > 8 ? 1 : 16 / warps);
    if (cap > NORM_PARTS) cap = NORM_PARTS;
    parts = static_cast<int>(ctas < cap ? ctas : cap);
    const dim3 grid(parts), block(32 * warps);
    const size_t smem = nw == 1 ? static_cast<size_t>(2) * n * CHUNK * 4 : 0;
#define MOE_NORM(V, N) launch_pdl(norm_bwd_kernel<V, N>, grid, block, smem, st, 1, a, nw)
#define MOE_NORM_N(V)                                                                \
  (wide ? launch_pdl(norm_bwd_wide_kernel<V>, grid, block, 0, st, 1, a)              \
        : n == 1 ? MOE_NORM(V, 1) : n == 2 ? MOE_NORM(V, 2) : MOE_NORM(V, 4))
    e = v == 8 ? launch_pdl(norm_bwd_wide_kernel<8>, grid, dim3(512), 0, st, 1, a)
        : v == 2 ? MOE_NORM_N(2) : MOE_NORM_N(1);
#undef MOE_NORM_N
#undef MOE_NORM
    }
    if (e != cudaSuccess) return e;
  }
  if (!sums) return e;
  return launch_pdl(norm_sum_kernel, dim3((a.C + 31) / 32, 2), dim3(32, SUM_ROWS), 0, st, 1, a.part,
                    parts, norm_part_floats(a.C) / 2, a.C, a.dgamma, a.dbeta, a.g_type);
}

}  // namespace moe
