// norm.cu -- layer norm and root-mean-square norm of rows, their gradient, and the normalised
// rows again from a row's 8-bit checkpoint.
//
//   v = x, or x + residual rounded to the rows' type;  m = mean of v (0 for the RMS norm)
//   rstd = 1 / sqrt(mean of (v - m)^2 + eps);  xhat = (v - m) rstd;  y = xhat gamma + beta
//   G = dy gamma;  dv = rstd (G - mean G - xhat mean(G xhat)) + add   (no mean G for the RMS norm)
//   dgamma = sum over the rows of dy xhat,  dbeta = sum over the rows of dy
//
// The statistics take two passes over a row that stays in registers: the mean first, then the
// squares around it, with the mean of the differences as its correction (which also mends the
// rounding of the first sum), all in fp32.  By their bytes these kernels belong to memory: 4 bytes
// an element forward for bf16 rows (9 with a residual and a checkpoint), 6 backward (8 with the
// stream's gradient).  What is reached, where a copy reaches 6.79 TB/s:
//   16,384 x 4096 bf16 with sum, statistics and int8 codes   5.6 TB/s, 108 us: two barriers a row, and
//                                                gamma and beta from L1 for every row
//   40 M elements of 4096 or 7168 columns, alone 3.2, 2.8 TB/s, 49, 56 us: the same, and sixteen warps
//                                                to an SM (110 registers); a barrier less, by merging the
//                                                warps' own means and squares, is open
//   28,308 x 1413 with sum and codes             2.3 TB/s, 156 us: instructions, an element at a time
//   from codes, 4096 x 7168                      4.9 TB/s, 18 us: 3 of it the launch's ramp
//   from codes, 40 M elements of 1001 to 7169    1.7-2.0 TB/s, 61-70 us: loads of one or two bytes, not
//                                                fetched ahead
// (the gradient: norm_bwd.cu)
#include <type_traits>

#include "rows8.cuh"

namespace moe {
namespace {

// v of one chunk: x, or the sum with the residual rounded to the rows' type
template <int V>
__device__ __forceinline__ void stream_values(float* f, const NormArgs& a, const void* xr,
                                              const void* rr, int chunk, int lane) {
  load_values<V>(f, xr, a.x_type, chunk, a.C, lane);
  if (!rr) return;
  float g[8];
  load_values<V>(g, rr, a.x_type, chunk, a.C, lane);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    f[j] += g[j];
    if (a.x_type == ROW_BF16) f[j] = __bfloat162float(__float2bfloat16_rn(f[j]));
  }
}

// xhat gamma + beta of a chunk whose xhat is in f
template <int V>
__device__ __forceinline__ void affine_store(float* f, const NormArgs& a, void* yr, int chunk,
                                             int lane) {
  float p[8];
  if (a.gamma) {
    load_values<V>(p, a.gamma, a.p_type, chunk, a.C, lane);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] *= p[j];
  }
  if (a.beta) {
    load_values<V>(p, a.beta, a.p_type, chunk, a.C, lane);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] += p[j];
  }
  store_values<V>(yr, a.y_type, chunk, a.C, lane, f);
}

// Rows that stay in registers: nw warps share a row, N chunks to a warp; with nw = 1 the CTA's warps have
// rows of their own.  The rows that follow come through shared memory while one is worked on; slots:
// 2, or 1 for the widest rows, which are not fetched ahead.  V = 8: rows of whole 16-byte vectors, a
// thread copies what it reads; V = 1: rows at any element and of any width, a warp copies the pieces
// that its columns touch and reads them element by element, 32 columns apart.
template <int N, int X, bool ADD, int V>
__global__ void __launch_bounds__(32 * MAX_WARPS)
norm_ring_kernel(const __grid_constant__ NormArgs a, int nw, int slots) {
  griddep_wait();
  __shared__ RowSums sh;
  extern __shared__ __align__(16) uint8_t ring[];
  row_sum_init(sh);
  constexpr int XS = X == ROW_BF16 ? 2 : 4, BYTES = CHUNK * XS + (V == 1 ? 16 : 0), PARTS = ADD ? 2 : 1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int w = nw == 1 ? 0 : warp;
  const bool layer = a.kind == MOE_NORM_LAYER;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (nw == 1 ? warps : 1);
  const int64_t first = nw == 1 ? static_cast<int64_t>(blockIdx.x) * warps + warp : blockIdx.x;
  // V = 1: first the columns' gamma and beta in fp32, as each thread reads them
  uint8_t* const par = ring + w * N * 2048;
  uint8_t* const mine = ring + (V == 1 ? nw * N * 2048 : 0) + warp * (N * PARTS * BYTES);
  const int slot_bytes = warps * (N * PARTS * BYTES);
  int chunk[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    chunk[i] = (i * nw + w) * CHUNK;
    if (V == 8 && chunk[i] + 8 * lane >= a.C)
      for (int s = 0; s < slots; ++s)
#pragma unroll
        for (int t = 0; t < PARTS; ++t) clear_chunk(mine + s * slot_bytes + (i * PARTS + t) * BYTES, X, lane);
  }
  const uint8_t* xr = static_cast<const uint8_t*>(row_at(a.x, first, a.ldx, XS));
  const uint8_t* rr = ADD ? static_cast<const uint8_t*>(row_at(a.add, first, a.ld_add, XS)) : nullptr;
  const int64_t x_step = step * a.ldx * XS, r_step = step * a.ld_add * XS;
  const uint8_t* const x_end = static_cast<const uint8_t*>(row_at(a.x, a.rows - 1, a.ldx, XS)) + a.C * XS;
  const uint8_t* const r_end =
      ADD ? static_cast<const uint8_t*>(row_at(a.add, a.rows - 1, a.ld_add, XS)) + a.C * XS : nullptr;
  // columns of a chunk; where they begin in the first 16 bytes of their pieces
  auto width = [&](int i) { return a.C - chunk[i] < CHUNK ? a.C - chunk[i] : CHUNK; };
  auto skip = [&](const void* p, int64_t row, int64_t ld) {
    return (static_cast<uint32_t>(reinterpret_cast<uint64_t>(p)) +
            static_cast<uint32_t>(row) * static_cast<uint32_t>(ld * XS)) & 15u;
  };
  int64_t next = first;
  auto fetch = [&](int slot) {
    if (next < a.rows) {
      uint8_t* to = mine + slot * slot_bytes;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (chunk[i] >= a.C) break;
        if (V == 1) {
          const int at = chunk[i] * XS, n = width(i) * XS;
          copy_pieces<XS / 2>(to + i * PARTS * BYTES, xr + at, n, a.x, x_end, lane);
          if (ADD) copy_pieces<XS / 2>(to + (i * PARTS + 1) * BYTES, rr + at, n, a.add, r_end, lane);
          continue;
        }
        copy_chunk(to + i * PARTS * BYTES, xr, X, chunk[i], a.C, lane);
        if (ADD) copy_chunk(to + (i * PARTS + 1) * BYTES, rr, X, chunk[i], a.C, lane);
      }
      xr += x_step;
      if (ADD) rr += r_step;
      next += step;
    }
    copy_commit();
  };
  auto some = [&](int i) { return V == 8 ? chunk[i] + 8 * lane < a.C : chunk[i] + lane < a.C; };
  auto put = [&](void* row, int type, int i, const float2* v) {
    if (V == 1) store_values<1>(row, type, chunk[i], a.C, lane, reinterpret_cast<const float*>(v));
    else if (some(i)) store_pairs(row, type, chunk[i] + 8 * lane, v);
  };
  auto get = [&](float2* v, const void* p, int i, int which) {
    if (V == 1) slot_values(v, par + (which * N + i) * 1024, ROW_FP32, lane);
    else vector_values(v, p, a.p_type, chunk[i] + 8 * lane);
  };
  if (V == 1)
#pragma unroll 1
    for (int t = 0; t < 2; ++t) {
      const void* p = t ? a.beta : a.gamma;
      if (!p) continue;
#pragma unroll 1
      for (int i = 0; i < N; ++i) {   // (with nw = 1 every warp writes the same; a thread reads its own)
        float v[8];
        load_values<1>(v, p, a.p_type, (i * nw + w) * CHUNK, a.C, lane);
        uint8_t* to = par + (t * N + i) * 1024 + 16 * lane;
        *reinterpret_cast<float4*>(to) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(to + 512) = make_float4(v[4], v[5], v[6], v[7]);
      }
    }
  for (int s = 0; s + 1 < slots; ++s) fetch(s);
  int slot = 0, ahead = slots - 1;
  const float over = 1.0f / static_cast<float>(a.C);
  for (int64_t row = first; row < a.rows; row += step) {
    if (V == 1) __syncwarp();   // all are done with the slot that is filled now
    fetch(ahead);
    if (++ahead == slots) ahead = 0;
    copy_wait(slots - 1);
    if (V == 1) __syncwarp();   // ... and see what the others copied
    const uint8_t* from = mine + slot * slot_bytes;
    if (++slot == slots) slot = 0;
    float2 f[N][4];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      // (a chunk begins 512 or 1024 bytes after the one before: the same place in its first piece)
      if (V == 1)
        smem_row_values<X, 1>(f[i], from + i * PARTS * BYTES + skip(a.x, row, a.ldx), 0, width(i), lane);
      else
        slot_values(f[i], from + i * PARTS * BYTES, X, lane);
      if (ADD) {
        float2 r[4];
        if (V == 1)
          smem_row_values<X, 1>(r, from + (i * PARTS + 1) * BYTES + skip(a.add, row, a.ld_add), 0, width(i), lane);
        else
          slot_values(r, from + (i * PARTS + 1) * BYTES, X, lane);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f[i][j] = __fadd2_rn(f[i][j], r[j]);
          if (X == ROW_BF16) {
            const uint32_t u = pack_bf16x2(f[i][j].x, f[i][j].y);
            f[i][j] = make_float2(bf16_lo(u), bf16_hi(u));
          }
        }
      }
    }
    if (ADD && a.out) {
      void* tr = row_at(a.out, row, a.ld_out, XS);
#pragma unroll
      for (int i = 0; i < N; ++i) put(tr, X, i, f[i]);
    }
    float mean = 0.0f;
    if (layer) {
      float2 s = both(0.0f);
#pragma unroll
      for (int i = 0; i < N; ++i)
        s = __fadd2_rn(s, __fadd2_rn(__fadd2_rn(f[i][0], f[i][1]), __fadd2_rn(f[i][2], f[i][3])));
      // (a quotient, not a product: a constant row's mean is exact wherever its sum is)
      mean = row_sum1(s.x + s.y, sh, 0, w, nw) / static_cast<float>(a.C);
    }
    // (columns past the row's end must not count as differences from the mean)
    float2 s = both(0.0f), q = both(0.0f);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (V == 1 ? chunk[i] + lane < a.C : chunk[i] + 8 * lane < a.C) {
        const bool all = V == 8 || chunk[i] + CHUNK <= a.C;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float2 d = __fadd2_rn(f[i][j], both(-mean));
          if (!all) {
            if (chunk[i] + 64 * j + lane >= a.C) d.x = 0.0f;
            if (chunk[i] + 64 * j + 32 + lane >= a.C) d.y = 0.0f;
          }
          s = __fadd2_rn(s, d);
          q = __ffma2_rn(d, d, q);
        }
      }
    const float2 sq = row_sum2(s.x + s.y, q.x + q.y, sh, 1, w, nw);
    const float shift = layer ? sq.x * over : 0.0f;
    const float var = fmaxf(sq.y * over - shift * shift, 0.0f);
    const float rstd = rsqrtf((sq.y != sq.y ? sq.y : var) + a.eps);
    if (lane == 0 && w == 0) {
      if (a.mean) a.mean[row] = mean + shift;
      if (a.rstd) a.rstd[row] = rstd;
    }
    if (a.codes)
      save_row_chunks<V, N>(row_at(a.codes, row, a.ld_codes, 1), a.scales + row * a.blocks, a.format,
                            chunk, a.C, lane, reinterpret_cast<const float(*)[8]>(f));
    void* yr = row_at(a.y, row, a.ld_y, row_size(a.y_type));
    const float2 low = both(-shift * rstd);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (!some(i)) continue;
      float2 p[4], b[4];
      // xhat = (v - mean) rstd - shift rstd: the shift is the mean's rounding, far below a step of it
#pragma unroll
      for (int j = 0; j < 4; ++j)
        f[i][j] = __ffma2_rn(__fadd2_rn(f[i][j], both(-mean)), both(rstd), low);
      if (a.gamma && a.beta) {
        get(p, a.gamma, i, 0);
        get(b, a.beta, i, 1);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[i][j] = __ffma2_rn(f[i][j], p[j], b[j]);
      } else if (a.gamma) {
        get(p, a.gamma, i, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[i][j] = __fmul2_rn(f[i][j], p[j]);
      } else if (a.beta) {
        get(b, a.beta, i, 1);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[i][j] = __fadd2_rn(f[i][j], b[j]);
      }
      put(yr, a.y_type, i, f[i]);
    }
    // with several warps to a row: the first sum's parts of the next row are written only after all
    // have read the second's of this one at their next barrier, and the second's after the first's;
    // the RMS norm has the second alone
    if (nw > 1 && !layer) __syncthreads();
  }
  griddep_launch();
}

// Rows of more columns than stay in registers: three passes, the second and third from L2.
template <int V>
__global__ void __launch_bounds__(32 * MAX_WARPS)
norm_wide_kernel(const __grid_constant__ NormArgs a) {
  griddep_wait();
  __shared__ RowSums sh;
  row_sum_init(sh);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int xs = row_size(a.x_type);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const void* xr = row_at(a.x, row, a.ldx, xs);
    const void* rr = a.add ? row_at(a.add, row, a.ld_add, xs) : nullptr;
    float f[1][8];
    float mean = 0.0f, s = 0.0f, q = 0.0f;
    if (a.kind == MOE_NORM_LAYER) {
      for (int c = warp * CHUNK; c < a.C; c += nw * CHUNK) {
        stream_values<V>(f[0], a, xr, rr, c, lane);
        float t = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) t += f[0][j];
        s += t;
      }
      mean = row_sum1(s, sh, 0, warp, nw) / static_cast<float>(a.C);
      s = 0.0f;
    }
    for (int c = warp * CHUNK; c < a.C; c += nw * CHUNK) {
      stream_values<V>(f[0], a, xr, rr, c, lane);
      float t = 0.0f, u = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = elem_col<V>(c, lane, j) < a.C ? f[0][j] - mean : 0.0f;
        t += d;
        u = fmaf(d, d, u);
      }
      s += t;
      q += u;
    }
    const float2 sq = row_sum2(s, q, sh, 1, warp, nw);
    const float shift = a.kind == MOE_NORM_LAYER ? sq.x / static_cast<float>(a.C) : 0.0f;
    const float var = fmaxf(sq.y / static_cast<float>(a.C) - shift * shift, 0.0f);
    const float rstd = rsqrtf((sq.y != sq.y ? sq.y : var) + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean + shift;
      if (a.rstd) a.rstd[row] = rstd;
    }
    void* tr = a.out ? row_at(a.out, row, a.ld_out, xs) : nullptr;
    void* yr = row_at(a.y, row, a.ld_y, row_size(a.y_type));
    // (a thread writes only elements that it alone reads: the outputs may be the inputs' rows)
    for (int c = warp * CHUNK; c < a.C; c += nw * CHUNK) {
      stream_values<V>(f[0], a, xr, rr, c, lane);
      if (tr) store_values<V>(tr, a.x_type, c, a.C, lane, f[0]);
      if (a.codes)
        save_row_chunks<V, 1>(row_at(a.codes, row, a.ld_codes, 1), a.scales + row * a.blocks, a.format,
                          &c, a.C, lane, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[0][j] = ((f[0][j] - mean) - shift) * rstd;
      affine_store<V>(f[0], a, yr, c, lane);
    }
    __syncthreads();
  }
  griddep_launch();
}

// Normalised rows from a checkpoint and the statistics, N rows at a time; the columns' gamma and
// beta stay in registers.
template <int V, int N, int TYPE>
__global__ void __launch_bounds__(WALK_THREADS, V == 8 ? 3 : 1)
ckpt_norm_kernel(const __grid_constant__ NormArgs a, int per, int groups) {
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const Walk w = walk_start(per, groups);
  if (!w.any) return;
  const bool layer = a.kind == MOE_NORM_LAYER;
  const int ys = row_size(a.y_type);
  float g[8], b[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    g[j] = 1.0f;
    b[j] = 0.0f;
  }
  if (a.gamma) load_values<V>(g, a.gamma, a.p_type, w.chunk, a.C, lane);
  if (a.beta) load_values<V>(b, a.beta, a.p_type, w.chunk, a.C, lane);
  const uint8_t* codes = static_cast<const uint8_t*>(a.x) + w.row * a.ldx;
  const float* scales = a.x_scales + w.row * a.blocks;
  uint8_t* y = static_cast<uint8_t*>(a.y) + w.row * a.ld_y * ys;
  const int64_t c_step = w.groups * a.ldx, s_step = w.groups * a.blocks, y_step = w.groups * a.ld_y * ys;
  for (int64_t row = w.row; row < a.rows; row += N * w.groups) {
    Raw8 raw[N];
    float sc[N][8 / V], mean[N], rstd[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t r = row + i * w.groups;
      mean[i] = 0.0f;
      if (r < a.rows) {
        load_raw<V>(raw[i], codes, TYPE, w.chunk, a.C, lane);
        load_chunk_scales<V>(sc[i], scales, w.chunk, a.C, lane);
        if (layer) mean[i] = a.mean[r];
        rstd[i] = a.rstd[r];
      }
      codes += c_step;
      scales += s_step;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (row + i * w.groups < a.rows) {
        float f[8];
        unpack_raw<V>(raw[i], TYPE, f);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          float2 v = __ffma2_rn(make_float2(f[j], f[j + 1]), make_float2(sc[i][j / V], sc[i][(j + 1) / V]),
                                both(-mean[i]));
          v = __ffma2_rn(__fmul2_rn(v, both(rstd[i])), make_float2(g[j], g[j + 1]),
                         make_float2(b[j], b[j + 1]));
          f[j] = v.x;
          f[j + 1] = v.y;
        }
        store_values<V>(y, a.y_type, w.chunk, a.C, lane, f);
      }
      y += y_step;
    }
  }
  griddep_launch();
}

}  // namespace

// The widest vectors that every row's address, distance and width allow.
int norm_vector(const NormArgs& a) {
  const int xs = row_size(a.x_type), ys = row_size(a.y_type);
  for (int v : {8, 2})
    if (a.C % v == 0 && rows_fit(a.x, a.ldx, row_size(a.src_type), v) &&
        rows_fit(a.add, a.ld_add, xs, v) && rows_fit(a.out, a.ld_out, xs, v) &&
        rows_fit(a.y, a.ld_y, ys, v) && rows_fit(a.codes, a.ld_codes, 1, v))
      return v;
  return 1;
}

namespace {
template <int N, int X, bool ADD, int V>
cudaError_t launch_norm_ring(const NormArgs& a, int nw, cudaStream_t st) {
  constexpr auto kern = norm_ring_kernel<N, X, ADD, V>;
  const int warps = nw == 1 ? 4 : nw;
  const int slot = warps * N * (CHUNK * row_size(X) + (V == 1 ? 16 : 0)) * (ADD ? 2 : 1);
  // CTAs to an SM by threads (registers), then as many slots as their shared memory allows
  const int par = V == 1 ? nw * N * 2048 : 0;
  int per = ctas_by_registers<kern>(32 * warps);
  while (per > 1 && per * (2 * slot + par) > ROW_SMEM) --per;
  // (more than two took L1 from the parameters and gained nothing, for short rows either)
  const int slots = per * (2 * slot + par) <= ROW_SMEM ? 2 : 1;
  const int64_t ctas = nw == 1 ? (a.rows + warps - 1) / warps : a.rows;
  const int64_t most = static_cast<int64_t>(row_sms()) * per;
  const int smem = slots * slot + par;
  const cudaError_t e = allow_smem<kern>(smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(static_cast<unsigned>(ctas < most ? ctas : most)), dim3(32 * warps), smem,
                    st, 1, a, nw, slots);
}
// Chunks to a warp: four to all of a row of up to four, since then no barrier is needed (1024 columns
// with sum and checkpoint 65 us, with two to a warp 70); two up to eight chunks (2048 columns 71 us, with
// four 99) and where four leave an eighth of them empty; else four (4096 columns 69 us, with two 74).
// Element by element four from three chunks on (1413 columns without a sum 127 us, with two 215; since the
// parameters lie in shared memory there, 71).  Two chunks to a warp with a sum in bf16 spill two registers.
template <int X, bool ADD, int V>
cudaError_t launch_norm_rows(const NormArgs& a, int chunks, cudaStream_t st) {
  if (chunks == 1) return launch_norm_ring<1, X, ADD, V>(a, 1, st);
  const int fours = (chunks + 3) / 4, twos = (chunks + 1) / 2;
  const bool two = chunks == 2 || (V == 8 && chunks > 4 && twos <= MAX_WARPS &&
                                   (chunks <= 8 || 8 * (4 * fours - chunks) > chunks));
  return two ? launch_norm_ring<2, X, ADD, V>(a, twos, st) : launch_norm_ring<4, X, ADD, V>(a, fours, st);
}
}  // namespace

cudaError_t launch_norm(const NormArgs& a, cudaStream_t st) {
  const int chunks = (a.C + CHUNK - 1) / CHUNK;
  const int v = norm_vector(a);
  const int64_t most = static_cast<int64_t>(1) << 30;
  // (element by element the parameters take shared memory too: the widest fp32 rows with a residual
  // leave them no room)
  const int row = (chunks + 3) / 4 * 4 * ((CHUNK * row_size(a.x_type) + 16) * (a.add ? 2 : 1) + 2048);
  if (chunks > 4 * MAX_WARPS || (v != 8 && row > ROW_SMEM)) {
    const dim3 grid(static_cast<unsigned>(a.rows < most ? a.rows : most));
    if (v == 8) return launch_pdl(norm_wide_kernel<8>, grid, dim3(512), 0, st, 1, a);
    if (v == 2) return launch_pdl(norm_wide_kernel<2>, grid, dim3(512), 0, st, 1, a);
    return launch_pdl(norm_wide_kernel<1>, grid, dim3(512), 0, st, 1, a);
  }
  auto go = [&](auto vector) {
    constexpr int V = decltype(vector)::value;
    if (a.x_type == ROW_BF16)
      return a.add ? launch_norm_rows<ROW_BF16, true, V>(a, chunks, st)
                   : launch_norm_rows<ROW_BF16, false, V>(a, chunks, st);
    return a.add ? launch_norm_rows<ROW_FP32, true, V>(a, chunks, st)
                 : launch_norm_rows<ROW_FP32, false, V>(a, chunks, st);
  };
  return v == 8 ? go(std::integral_constant<int, 8>()) : go(std::integral_constant<int, 1>());
}

cudaError_t launch_ckpt_norm(const NormArgs& a, cudaStream_t st) {
  const int v = norm_vector(a);
  const WalkGrid g = walk_grid(a.rows, a.C, 64);
  auto go = [&](auto kern) {
    return launch_pdl(kern, g.grid, dim3(WALK_THREADS), 0, st, 1, a, g.per, g.groups);
  };
  if (a.src_type == ROW_INT8)
    return v == 8 ? go(ckpt_norm_kernel<8, 4, ROW_INT8>) : v == 2 ? go(ckpt_norm_kernel<2, 2, ROW_INT8>)
                                                                  : go(ckpt_norm_kernel<1, 2, ROW_INT8>);
  return v == 8 ? go(ckpt_norm_kernel<8, 4, ROW_E4M3>) : v == 2 ? go(ckpt_norm_kernel<2, 2, ROW_E4M3>)
                                                                : go(ckpt_norm_kernel<1, 2, ROW_E4M3>);
}

}  // namespace moe
