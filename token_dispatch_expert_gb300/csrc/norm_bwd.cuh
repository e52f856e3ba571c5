// norm_bwd.cuh -- the norms' gradient for rows that stay in registers (norm_bwd.cu has the formulas, the
// wider rows and the sums over the rows).  A header, so that the types are compiled side by side.
#pragma once

#include "rows8.cuh"

namespace moe {
namespace {

// nw warps share a row, N chunks to a warp; a CTA holds several such groups where nw is small.  dy, v
// and add of the rows that follow come into shared memory by bulk copies while one is worked on; the
// statistics and a chunk's scale are loaded a row ahead.  The first thread of a group of nw warps copies
// for it: when all have passed the barrier in a row's sums, all are done with the row before, whose slot
// is filled again.  gamma lies in shared memory too (but for the widest rows, which leave it no room):
// from L1, which the slots leave little of, it came from L2 for every row, and 16384 x 4096 took 107 us
// instead of 90.  With up to two chunks to a warp a row's G and xhat stay in registers between the two
// passes over it, with four they are computed again, from the slot.  Even so four chunks, whose sums
// alone are 64 registers, spill: up to 132 bytes a thread from codes, 64 from fp32 rows and 328 element
// by element (40 M elements of 16384 columns from int8 codes 119 us, of 256 to 7168 columns 60-67).
// S: the type of v or its codes, X: of add and dx, Y: of dy.  V = 8: rows of whole 16-byte vectors;
// V = 1: rows at any element and of any width, whose copies bring the whole 16-byte pieces that a row
// touches, and which are read and written element by element from there.
constexpr int MAX_SLOTS = 4, MAX_GROUPS = 8;
constexpr long long BULK_BUDGET = 4000000000LL;   // clock cycles (about 2 s)

template <int N, int S, int X, int Y, int V>
__global__ void __launch_bounds__(N == 1 ? 256 : 32 * MAX_WARPS, N == 1 ? 3 : 1)
norm_bwd_ring_kernel(const __grid_constant__ NormArgs a, int nw, int slots) {
  __shared__ RowSums sums[MAX_GROUPS];
  __shared__ __align__(8) uint64_t full[MAX_GROUPS][MAX_SLOTS];
  __shared__ int gave_up;
  extern __shared__ __align__(16) uint8_t ring[];
  constexpr bool KEEP = N < 4, CODES = S == ROW_INT8 || S == ROW_E4M3;
  constexpr int XS = X == ROW_BF16 ? 2 : 4, YS = Y == ROW_BF16 ? 2 : 4;
  constexpr int SS = CODES ? 1 : S == ROW_BF16 ? 2 : 4;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int own = warp / nw, w = warp - own * nw, groups = warps / nw;
  const bool copies = w == 0 && lane == 0, gamma_here = N < 4 || groups > 1;
  RowSums& sh = sums[own];
  if (copies)
    for (int s = 0; s < slots; ++s) mbar_init(smem_u32(&full[own][s]), 1);
  if (threadIdx.x == 0) gave_up = 0;
  fence_mbar_init();
  for (int i = threadIdx.x; i < static_cast<int>(sizeof(sums) / 4); i += blockDim.x)
    reinterpret_cast<float*>(sums)[i] = 0.0f;
  __syncthreads();
  griddep_wait();   // see common.cuh: dependent launches
  // (32 bits hold every row and the few steps past the last one)
  const uint32_t rows = static_cast<uint32_t>(a.rows), step = gridDim.x * groups;
  const uint32_t first = blockIdx.x * groups + own;
  const float over = 1.0f / static_cast<float>(a.C);
  const bool layer = a.kind == MOE_NORM_LAYER, add = a.add != nullptr;
  // a slot: dy, v, add, each as many whole pieces of 16 bytes as a row can touch
  const int pieces = V == 8 ? 15 : 31;
  const int y_bytes = (a.C * YS + pieces) / 16 * 16, x_bytes = (a.C * SS + (CODES ? 15 : pieces)) / 16 * 16;
  const int a_bytes = add ? (a.C * XS + pieces) / 16 * 16 : 0;
  const int slot_bytes = y_bytes + x_bytes + a_bytes;
  uint8_t* const gam = ring + w * N * 1024;   // the columns' gamma in fp32, then the slots
  uint8_t* const mine = ring + (gamma_here ? nw * N * 1024 : 0) + own * slots * slot_bytes;
  auto at = [](const void* p, uint32_t row, int64_t ld) {
    return static_cast<const uint8_t*>(p) + static_cast<int64_t>(row) * ld;
  };
  uint32_t odd = 0, started = 0;   // of the copying thread: slots filled an odd number of times, ever
  auto fetch = [&](uint32_t row, int slot) {
    if (*static_cast<volatile int*>(&gave_up)) return;
    odd ^= 1u << slot;
    started |= 1u << slot;
    uint8_t* to = mine + slot * slot_bytes;
    const uint32_t bar = smem_u32(&full[own][slot]);
    const uint8_t *yr = at(a.y, row, a.ld_y * YS), *xr = at(a.x, row, a.ldx * SS);
    const uint8_t* ar = at(a.add, row, a.ld_add * XS);
    if (V == 8) {
      mbar_arrive_expect_tx(bar, slot_bytes);
      bulk_load(smem_u32(to), yr, y_bytes, bar);
      bulk_load(smem_u32(to + y_bytes), xr, x_bytes, bar);
      if (add) bulk_load(smem_u32(to + y_bytes + x_bytes), ar, a_bytes, bar);
      return;
    }
    auto end = [&](const void* p, int64_t ld, int size) { return at(p, rows - 1, ld * size) + a.C * size; };
    Span sy = bulk_span(yr, a.C * YS, a.y, end(a.y, a.ld_y, YS)), sx, sa{0, 0};
    if (CODES) sx = {reinterpret_cast<uint64_t>(xr), reinterpret_cast<uint64_t>(xr) + x_bytes};
    else sx = bulk_span(xr, a.C * SS, a.x, end(a.x, a.ldx, SS));
    span_ends(to, yr, a.C * YS, sy);
    if (!CODES) span_ends(to + y_bytes, xr, a.C * SS, sx);
    if (add) {
      sa = bulk_span(ar, a.C * XS, a.add, end(a.add, a.ld_add, XS));
      span_ends(to + y_bytes + x_bytes, ar, a.C * XS, sa);
    }
    fence_proxy_async_smem();   // (a later row's bulk copy takes the same bytes of the slot)
    mbar_arrive_expect_tx(bar, static_cast<uint32_t>((sy.hi - sy.lo) + (sx.hi - sx.lo) + (sa.hi - sa.lo)));
    auto go = [&](uint8_t* t, const uint8_t* p, const Span& s) {
      if (s.hi > s.lo)
        bulk_load(smem_u32(t) + static_cast<uint32_t>(s.lo - (reinterpret_cast<uint64_t>(p) & ~15ull)),
                  reinterpret_cast<const void*>(s.lo), static_cast<uint32_t>(s.hi - s.lo), bar);
    };
    go(to, yr, sy);
    go(to + y_bytes, xr, sx);
    if (add) go(to + y_bytes + x_bytes, ar, sa);
  };
  if (copies)
    for (int s = 0; s < (slots > 1 ? slots - 1 : 1); ++s)
      if (first + s * step < rows) fetch(first + s * step, s);
  constexpr int NS = V == 8 ? 1 : 2;   // blocks of a chunk to a lane
  float2 dg[N][4], db[N][4];
  int chunk[N];
  float sc[N][NS];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    chunk[i] = (i * nw + w) * CHUNK;
#pragma unroll
    for (int h = 0; h < NS; ++h) sc[i][h] = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) dg[i][j] = db[i][j] = both(0.0f);
  }
  // whether a chunk has columns for this lane
  auto some = [&](int i) { return V == 8 ? chunk[i] + 8 * lane < a.C : chunk[i] + lane < a.C; };
  float mean = 0.0f, rstd = 0.0f;
  auto small = [&](uint32_t row) {
    if (layer) mean = a.mean[row];
    rstd = a.rstd[row];
    if (CODES) {
      const float* sr = a.x_scales + static_cast<int64_t>(row) * a.blocks;
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int h = 0; h < NS; ++h) {
          const int c = V == 8 ? chunk[i] + 8 * lane : chunk[i] + 128 * h;
          if (c < a.C) sc[i][h] = sr[c >> 7];
        }
    }
  };
  auto param_values = [&](float2* p, int i) {
    if (V == 8) {
      vector_values(p, a.gamma, a.p_type, chunk[i] + 8 * lane);
    } else {
      float f[8];
      load_values<1>(f, a.gamma, a.p_type, chunk[i], a.C, lane);
#pragma unroll
      for (int j = 0; j < 4; ++j) p[j] = make_float2(f[2 * j], f[2 * j + 1]);
    }
  };
  // the part of a row's first 16 bytes that is not the row's, by tensor
  auto skip = [](const void* p, uint32_t row, int64_t ld) {
    return V == 8 ? 0u : (static_cast<uint32_t>(reinterpret_cast<uint64_t>(p)) + row * static_cast<uint32_t>(ld)) & 15u;
  };
  // G and xhat of a chunk in a slot; past the row's end zeros
  auto values = [&](const uint8_t* yt, const uint8_t* xt, int i, float2 st, const float* scale, float2* g,
                    float2* xh, bool sums) {
    if (!some(i)) {
#pragma unroll
      for (int j = 0; j < 4; ++j) g[j] = xh[j] = both(0.0f);
      return;
    }
    float2 p[4];
    smem_row_values<Y, V>(g, yt, chunk[i], a.C, lane);
    smem_row_values<S, V>(xh, xt, chunk[i], a.C, lane);
    if (gamma_here) slot_values(p, gam + i * 1024, ROW_FP32, lane);
    else if (a.gamma) param_values(p, i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      xh[j] = CODES ? __ffma2_rn(xh[j], both(scale[NS == 1 ? 0 : j / 2]), both(-st.x))
                    : __fadd2_rn(xh[j], both(-st.x));
      xh[j] = __fmul2_rn(xh[j], both(st.y));
      if (sums) {
        dg[i][j] = __ffma2_rn(g[j], xh[j], dg[i][j]);
        db[i][j] = __fadd2_rn(db[i][j], g[j]);
      }
      if (gamma_here || a.gamma) g[j] = __fmul2_rn(g[j], p[j]);
    }
  };
  if (gamma_here)   // (each group writes the same; a thread reads what it wrote)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float2 p[4] = {both(1.0f), both(1.0f), both(1.0f), both(1.0f)};
      if (a.gamma && some(i)) param_values(p, i);
      *reinterpret_cast<float4*>(gam + i * 1024 + 16 * lane) = make_float4(p[0].x, p[0].y, p[1].x, p[1].y);
      *reinterpret_cast<float4*>(gam + i * 1024 + 512 + 16 * lane) = make_float4(p[2].x, p[2].y, p[3].x, p[3].y);
    }
  if (first < rows) small(first);
  auto put = [&](void* row, int type, int i, const float2* v) {
    if (V == 8) store_pairs(row, type, chunk[i] + 8 * lane, v);
    else store_values<1>(row, type, chunk[i], a.C, lane, reinterpret_cast<const float*>(v));
  };
  int slot = 0, turn = 0;
  uint32_t phase = 0;
  for (uint32_t row = first; row < rows; row += step) {
    const float2 st = make_float2(mean, rstd);
    float s0[N][NS];
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int h = 0; h < NS; ++h) s0[i][h] = sc[i][h];
    if (row + step < rows) small(row + step);
    // (one that gives up goes on, so that the barriers below stay whole: the error word says so)
    mbar_wait_bounded(smem_u32(&full[own][slot]), phase, &gave_up, a.err, BULK_BUDGET);
    const uint8_t* from = mine + slot * slot_bytes;
    const uint8_t* yt = from + skip(a.y, row, a.ld_y * YS);
    const uint8_t* xt = from + y_bytes + (CODES ? 0 : skip(a.x, row, a.ldx * SS));
    const uint8_t* at_add = from + y_bytes + x_bytes + skip(a.add, row, a.ld_add * XS);
    float2 g[KEEP ? N : 1][4], xh[KEEP ? N : 1][4], c1 = both(0.0f), c2 = both(0.0f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int k = KEEP ? i : 0;
      values(yt, xt, i, st, s0[i], g[k], xh[k], true);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        c1 = __fadd2_rn(c1, g[k][j]);
        c2 = __ffma2_rn(g[k][j], xh[k][j], c2);
      }
    }
    const float2 c = row_sum2(c1.x + c1.y, c2.x + c2.y, sh, turn, w, nw, groups == 1 ? 0 : 1 + own);
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
      if (!KEEP) values(yt, xt, i, st, s0[i], g[k], xh[k], false);
      if (!some(i)) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        g[k][j] = __fmul2_rn(__ffma2_rn(xh[k][j], both(m2), __fadd2_rn(g[k][j], both(m1))), both(st.y));
      if (add) {
        float2 p[4];
        smem_row_values<X, V>(p, at_add, chunk[i], a.C, lane);
#pragma unroll
        for (int j = 0; j < 4; ++j) g[k][j] = __fadd2_rn(g[k][j], p[j]);
      }
      put(dr, X, i, g[k]);
    }
    if (slots == 1) {
      // (only the widest rows, with one group to a CTA)
      __syncthreads();
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
  if (groups > 1) {
    // the groups' sums one after another, so that their order is fixed (every copy has been waited
    // for: none was started for rows past the last one)
    float2* cols = reinterpret_cast<float2*>(ring) + w * N * 256;
    __syncthreads();
    for (int k = 0; k < groups; ++k) {
      if (own == k) {
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
    if (own + 1 != groups) return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (!some(i)) continue;
    put(out, ROW_FP32, i, dg[i]);
    put(out + wide, ROW_FP32, i, db[i]);
  }
}

template <int N, int S, int X, int Y, int V>
cudaError_t launch_ring(const NormArgs& a, int nw, cudaStream_t st, int* parts) {
  constexpr auto kern = norm_bwd_ring_kernel<N, S, X, Y, V>;
  // rows of few chunks: groups of warps that fill a CTA of eight (fifteen for three to a row: an SM
  // holds sixteen warps)
  const int groups = nw > 4 ? 1 : nw == 3 ? 5 : 8 / nw, warps = groups * nw;
  auto bytes = [&](int size, int more) { return (a.C * size + more) / 16 * 16; };
  const int more = V == 8 ? 15 : 31;
  const int row = bytes(row_size(Y), more) + bytes(row_size(S), a.x_scales ? 15 : more) +
                  (a.add ? bytes(row_size(X), more) : 0);
  const int slot = groups * row, least = groups > 1 ? nw * N * 2048 : 0;
  const int gam = N < 4 || groups > 1 ? nw * N * 1024 : 0;
  // CTAs to an SM by registers, then as many slots as their shared memory allows
  int per = ctas_by_registers<kern>(32 * warps);
  if (per > NORM_PARTS / 152) per = NORM_PARTS / 152;
  while (per > 1 && per * (2 * slot + gam) > ROW_SMEM) --per;
  int slots = MAX_SLOTS;
  while (slots > 1 && per * (slots * slot + gam) > ROW_SMEM) --slots;
  const int smem = slots * slot + gam > least ? slots * slot + gam : least;
  const cudaError_t e = allow_smem<kern>(smem);
  if (e != cudaSuccess) return e;
  const int64_t ctas = (a.rows + groups - 1) / groups;
  int64_t most = static_cast<int64_t>(row_sms()) * per;
  if (most > NORM_PARTS) most = NORM_PARTS;
  *parts = static_cast<int>(ctas < most ? ctas : most);
  return launch_pdl(kern, dim3(*parts), dim3(32 * warps), smem, st, 1, a, nw, slots);
}
template <int S, int X, int Y, int V>
cudaError_t launch_rows(const NormArgs& a, int chunks, cudaStream_t st, int* parts) {
  if (chunks == 1) return launch_ring<1, S, X, Y, V>(a, 1, st, parts);
  if (chunks <= 2 * MAX_WARPS) return launch_ring<2, S, X, Y, V>(a, (chunks + 1) / 2, st, parts);
  return launch_ring<4, S, X, Y, V>(a, (chunks + 3) / 4, st, parts);
}
// the types of a stream in bf16, or in fp32 with gradients of either type
template <int S, int X, int V>
cudaError_t launch_stream(const NormArgs& a, int chunks, cudaStream_t st, int* parts) {
  if constexpr (X == ROW_FP32)
    if (a.y_type == ROW_FP32) return launch_rows<S, X, ROW_FP32, V>(a, chunks, st, parts);
  return launch_rows<S, X, ROW_BF16, V>(a, chunks, st, parts);
}
template <int X, int V>
cudaError_t launch_source(const NormArgs& a, int chunks, cudaStream_t st, int* parts) {
  if (a.src_type == ROW_INT8) return launch_stream<ROW_INT8, X, V>(a, chunks, st, parts);
  if (a.src_type == ROW_E4M3) return launch_stream<ROW_E4M3, X, V>(a, chunks, st, parts);
  return launch_stream<X, X, V>(a, chunks, st, parts);
}

}  // namespace
}  // namespace moe
