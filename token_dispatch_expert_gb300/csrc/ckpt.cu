// ckpt.cu -- activations held in 8 bits from the forward to the backward pass: saving rows,
// restoring them, the SwiGLU's gradient and the combine's gradient from them.
//
// A checkpoint is one code a value and one fp32 scale for each block of 128 along the row
// (rows8.cuh).  Everything here is memory's by its bytes: 3 a value to save bf16 rows or to restore
// them, 10 a column of the SwiGLU's gradient, 3 a value of the combine's.  What is reached, and what
// is left, where a copy reaches 6.79 TB/s:
//   save 65,536 x 1536 bf16 to int8              6.2 TB/s, 49 us
//   [a | b] and h, 44,236 rows of 2816           6.3 TB/s, 79 us
//   SwiGLU's gradient, 65,536 x 768, with h      6.5 TB/s, 78 us
//   the same, 15,563 x 1409 of E4M3 codes        4.1 TB/s, 53 us: instructions, an element at a time
//   restore 65,536 x 1536 from int8 to bf16      5.9 TB/s, 52 us
//   [a | b] and h of f = 1001 or 1409, 40 M codes   3.9 TB/s, 41 us: instructions, an element at a time
//   combine's gradient, 4096 tokens of 7168, 8 slots   6.4 TB/s, 120 us (six slots spill a register)
//   save 39,960 x 1001                           3.3 TB/s, 37 us: latency, loads of two bytes
// Rows fetched ahead through shared memory took the first three from 58, 88 and 94 us: with loads to
// registers a warp has nothing under way while it computes, and more registers for more rows leave
// fewer warps.
#include <type_traits>

#include "rows8.cuh"

namespace moe {
namespace {

constexpr int SLOTS = 3;

__device__ __forceinline__ int64_t live_rows(const CkptArgs& a) {
  if (!a.live) return a.rows;
  const int64_t n = *a.live;
  if (n < 0 || n > a.rows) {
    if (blockIdx.x == 0 && threadIdx.x == 0) flag_error(a.err, MOE_DEVERR_BAD_OFFSETS);
    return n < 0 ? 0 : a.rows;
  }
  return n;
}

// N rows at a time: with N = 4 one division and one set of shuffles serve four blocks.
template <int V, int N, int X, int FORMAT>
__global__ void __launch_bounds__(WALK_THREADS)
save_kernel(const __grid_constant__ CkptArgs a, int per, int groups) {
  griddep_wait();   // see common.cuh: dependent launches
  const int lane = threadIdx.x & 31;
  const Walk w = walk_start(per, groups);
  const int64_t live = w.any ? live_rows(a) : 0;
  constexpr int XS = X == ROW_BF16 ? 2 : 4;
  const uint8_t* x = static_cast<const uint8_t*>(a.x) + w.row * a.ldx * XS;
  uint8_t* codes = static_cast<uint8_t*>(a.codes) + w.row * a.ld;
  float* scales = a.scales + w.row * a.blocks;
  const int64_t x_step = w.groups * a.ldx * XS, c_step = w.groups * a.ld, s_step = w.groups * a.blocks;
  for (int64_t row = w.row; row < live; row += N * w.groups) {
    Raw8 raw[N];
    void* to[N];
    float* ts[N];
    int chunk[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      chunk[i] = row + i * w.groups < live ? w.chunk : a.C;   // (a chunk at C has no columns)
      to[i] = codes;
      ts[i] = scales;
      load_raw<V>(raw[i], x, X, chunk[i], a.C, lane);
      x += x_step;
      codes += c_step;
      scales += s_step;
    }
    float f[N][8];
#pragma unroll
    for (int i = 0; i < N; ++i) unpack_raw<V>(raw[i], X, f[i]);
    save_chunks<V, N>(to, ts, FORMAT, chunk, a.C, lane, f);
  }
  griddep_launch();
}

template <int V, int N, int X, int FORMAT>
__global__ void __launch_bounds__(WALK_THREADS)
load_kernel(const __grid_constant__ CkptArgs a, int per, int groups) {
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const Walk w = walk_start(per, groups);
  const int64_t live = w.any ? live_rows(a) : 0;
  constexpr int XS = X == ROW_BF16 ? 2 : 4, TYPE = FORMAT == MOE_CKPT_INT8 ? ROW_INT8 : ROW_E4M3;
  uint8_t* x = static_cast<uint8_t*>(a.out) + w.row * a.ldx * XS;
  const uint8_t* codes = static_cast<const uint8_t*>(a.codes_in) + w.row * a.ld;
  const float* scales = a.scales_in + w.row * a.blocks;
  const int64_t x_step = w.groups * a.ldx * XS, c_step = w.groups * a.ld, s_step = w.groups * a.blocks;
  for (int64_t row = w.row; row < live; row += N * w.groups) {
    Raw8 raw[N];
    float sc[N][8 / V];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (row + i * w.groups < live) {
        load_raw<V>(raw[i], codes, TYPE, w.chunk, a.C, lane);
        load_chunk_scales<V>(sc[i], scales, w.chunk, a.C, lane);
      }
      codes += c_step;
      scales += s_step;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (row + i * w.groups < live) {
        float f[8];
        unpack_raw<V>(raw[i], TYPE, f);
        scale_values<V>(f, sc[i]);
        store_values<V>(x, X, w.chunk, a.C, lane, f);
      }
      x += x_step;
    }
  }
  griddep_launch();
}

// [a | b] and h, or with BACK [da | db] and h from dh.  With s = sigma(a): h = a s b, da = dh b s (1 + a
// (1 - s)), db = dh a s, from the 32-bit restored values, each rounded once.  In place: a and b become
// what is stored for them.
template <bool BACK>
__device__ __forceinline__ void swiglu_pairs(float2* a, float2* b, const float2* d, float2* h) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 s = make_float2(sigmoid_fast(a[j].x), sigmoid_fast(a[j].y));
    const float2 as = __fmul2_rn(a[j], s);
    h[j] = __fmul2_rn(as, b[j]);
    if (BACK) {
      const float2 one = __ffma2_rn(s, both(-1.0f), both(1.0f));   // 1 - s
      a[j] = __fmul2_rn(__fmul2_rn(d[j], b[j]), __ffma2_rn(as, one, s));
      b[j] = __fmul2_rn(d[j], as);
    }
  }
}

// ------------------------------------------------------------------ rows of whole vectors
// The three above for rows of whole 16-byte vectors: the rows that follow come through shared memory
// (rows8.cuh) in SLOTS slots.
template <int N, int X, int FORMAT>
__global__ void __launch_bounds__(WALK_THREADS, 2)
save_ring_kernel(const __grid_constant__ CkptArgs a, int per, int groups) {
  griddep_wait();
  constexpr int XS = X == ROW_BF16 ? 2 : 4, BYTES = CHUNK * XS;
  __shared__ __align__(16) uint8_t ring[WALK_WARPS][SLOTS][N][BYTES];
  const int lane = threadIdx.x & 31;
  const Walk w = walk_start(per, groups);
  if (!w.any) return;
  const int64_t live = live_rows(a);
  uint8_t(*mine)[N][BYTES] = ring[threadIdx.x >> 5];
  const bool past = w.chunk + 8 * lane >= a.C;
  if (past)
    for (int s = 0; s < SLOTS; ++s)
#pragma unroll
      for (int i = 0; i < N; ++i) clear_chunk(mine[s][i], X, lane);
  const uint8_t* x = static_cast<const uint8_t*>(a.x) + w.row * a.ldx * XS;
  const int64_t x_step = w.groups * a.ldx * XS;
  int64_t next = w.row;
  auto fetch = [&](int slot) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (next < live) copy_chunk(mine[slot][i], x, X, w.chunk, a.C, lane);
      x += x_step;
      next += w.groups;
    }
    copy_commit();
  };
  for (int s = 0; s + 1 < SLOTS; ++s) fetch(s);
  uint8_t* codes = static_cast<uint8_t*>(a.codes) + w.row * a.ld;
  float* scales = a.scales + w.row * a.blocks;
  const int64_t c_step = w.groups * a.ld, s_step = w.groups * a.blocks;
  int slot = 0, ahead = SLOTS - 1;
  for (int64_t row = w.row; row < live; row += N * w.groups) {
    fetch(ahead);
    if (++ahead == SLOTS) ahead = 0;
    copy_wait(SLOTS - 1);
    void* to[N];
    float* ts[N];
    int chunk[N];
    float2 f[N][4];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      chunk[i] = row + i * w.groups < live ? w.chunk : a.C;   // (a chunk at C has no columns)
      to[i] = codes;
      ts[i] = scales;
      codes += c_step;
      scales += s_step;
      slot_values(f[i], mine[slot][i], X, lane);
    }
    if (++slot == SLOTS) slot = 0;
    save_chunks<8, N>(to, ts, FORMAT, chunk, a.C, lane, reinterpret_cast<const float(*)[8]>(f));
  }
  griddep_launch();
}

template <int X, int FORMAT>
__global__ void __launch_bounds__(WALK_THREADS, 4)
load_ring_kernel(const __grid_constant__ CkptArgs a, int per, int groups) {
  griddep_wait();
  constexpr int XS = X == ROW_BF16 ? 2 : 4, TYPE = FORMAT == MOE_CKPT_INT8 ? ROW_INT8 : ROW_E4M3;
  constexpr int N = 2;
  struct Slot { uint8_t codes[CHUNK]; float scale[32]; };
  __shared__ __align__(16) Slot ring[WALK_WARPS][SLOTS][N];
  const int lane = threadIdx.x & 31;
  const Walk w = walk_start(per, groups);
  if (!w.any) return;
  const int64_t live = live_rows(a);
  Slot(*mine)[N] = ring[threadIdx.x >> 5];
  const int col = w.chunk + 8 * lane;
  if (col >= a.C) return;   // (nothing below is for the whole warp)
  const uint8_t* codes = static_cast<const uint8_t*>(a.codes_in) + w.row * a.ld;
  const float* scales = a.scales_in + w.row * a.blocks + (col >> 7);
  const int64_t c_step = w.groups * a.ld, s_step = w.groups * a.blocks;
  int64_t next = w.row;
  auto fetch = [&](int slot) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (next < live) {
        copy_chunk(mine[slot][i].codes, codes, TYPE, w.chunk, a.C, lane);
        copy_async4(smem_u32(&mine[slot][i].scale[lane]), scales);
      }
      codes += c_step;
      scales += s_step;
      next += w.groups;
    }
    copy_commit();
  };
  for (int s = 0; s + 1 < SLOTS; ++s) fetch(s);
  uint8_t* x = static_cast<uint8_t*>(a.out) + w.row * a.ldx * XS;
  const int64_t x_step = w.groups * a.ldx * XS;
  int slot = 0, ahead = SLOTS - 1;
  for (int64_t row = w.row; row < live; row += N * w.groups) {
    fetch(ahead);
    if (++ahead == SLOTS) ahead = 0;
    copy_wait(SLOTS - 1);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (row + i * w.groups < live) {
        float2 f[4];
        slot_values(f, mine[slot][i].codes, TYPE, lane);
        const float2 sc = both(mine[slot][i].scale[lane]);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = __fmul2_rn(f[j], sc);
        store_pairs(x, X, col, f);
      }
      x += x_step;
    }
    if (++slot == SLOTS) slot = 0;
  }
  griddep_launch();
}

template <bool BACK, int TYPE>
__global__ void __launch_bounds__(WALK_THREADS, 4)
swiglu_ring_kernel(const __grid_constant__ CkptArgs p, int per, int groups) {
  griddep_wait();
  struct Slot { uint8_t dh[BACK ? 2 * CHUNK : 16]; uint8_t a[CHUNK], b[CHUNK]; float sa[32], sb[32]; };
  __shared__ __align__(16) Slot ring[WALK_WARPS][SLOTS];
  const int lane = threadIdx.x & 31;
  const int f = p.C / 2;
  const Walk w = walk_start(per, groups);
  if (!w.any) return;
  const int64_t live = live_rows(p);
  Slot* mine = ring[threadIdx.x >> 5];
  const int col = w.chunk + 8 * lane;
  if (col >= f) return;   // (nothing below is for the whole warp)
  const uint8_t* codes = static_cast<const uint8_t*>(p.codes_in) + w.row * p.ld;
  const float* scales = p.scales_in + w.row * p.blocks;
  const __nv_bfloat16* dh = static_cast<const __nv_bfloat16*>(p.dh) + w.row * f;
  const int64_t c_step = w.groups * p.ld, s_step = w.groups * p.blocks, h_step = w.groups * f;
  const int block_a = col >> 7, block_b = (f + col) >> 7;
  int64_t next = w.row;
  auto fetch = [&](int slot) {
    if (next < live) {
      Slot& t = mine[slot];
      copy_chunk(t.a, codes, TYPE, w.chunk, f, lane);
      copy_chunk(t.b, codes + f, TYPE, w.chunk, f, lane);
      if (BACK) copy_chunk(t.dh, dh, ROW_BF16, w.chunk, f, lane);
      copy_async4(smem_u32(&t.sa[lane]), scales + block_a);
      copy_async4(smem_u32(&t.sb[lane]), scales + block_b);
    }
    codes += c_step;
    scales += s_step;
    dh += h_step;
    next += w.groups;
    copy_commit();
  };
  for (int s = 0; s + 1 < SLOTS; ++s) fetch(s);
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + w.row * p.C;
  __nv_bfloat16* hr = static_cast<__nv_bfloat16*>(p.h) + w.row * f;
  int slot = 0, ahead = SLOTS - 1;
  for (int64_t row = w.row; row < live; row += w.groups) {
    fetch(ahead);
    if (++ahead == SLOTS) ahead = 0;
    copy_wait(SLOTS - 1);
    const Slot& t = mine[slot];
    if (++slot == SLOTS) slot = 0;
    float2 a[4], b[4], h[4], d[4];
    slot_values(a, t.a, TYPE, lane);
    slot_values(b, t.b, TYPE, lane);
    if (BACK) slot_values(d, t.dh, ROW_BF16, lane);
    const float2 sa = both(t.sa[lane]), sb = both(t.sb[lane]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      a[j] = __fmul2_rn(a[j], sa);
      b[j] = __fmul2_rn(b[j], sb);
    }
    swiglu_pairs<BACK>(a, b, d, h);
    if (BACK || p.out) {
      store_pairs(out, ROW_BF16, col, a);
      store_pairs(out + f, ROW_BF16, col, b);
    }
    if (p.h) store_pairs(hr, ROW_BF16, col, h);
    out += 2 * h_step;
    hr += h_step;
  }
  griddep_launch();
}

// The same for rows of any width: a warp copies the 16-byte pieces that its 256 columns touch (33 of
// dh, 16 of a's codes, 17 of b's) and the scales of their blocks (two and three), and reads them
// element by element, 32 columns apart.  Pieces of codes lie within a row's distance; one of dh that
// would pass the buffer's end is read by bytes.
template <bool BACK, int TYPE>
__global__ void __launch_bounds__(WALK_THREADS, 3)
swiglu_odd_kernel(const __grid_constant__ CkptArgs p, int per, int groups) {
  griddep_wait();
  struct Slot { uint8_t dh[BACK ? 33 * 16 : 16]; uint8_t a[16 * 16], b[17 * 16]; float sa[4], sb[4]; };
  __shared__ __align__(16) Slot ring[WALK_WARPS][SLOTS];
  const int lane = threadIdx.x & 31;
  const int f = p.C / 2;
  const Walk w = walk_start(per, groups);
  if (!w.any) return;
  const int64_t live = live_rows(p);
  Slot* mine = ring[threadIdx.x >> 5];
  const uint8_t* codes = static_cast<const uint8_t*>(p.codes_in) + w.row * p.ld;
  const float* scales = p.scales_in + w.row * p.blocks;
  const int64_t c_step = w.groups * p.ld, s_step = w.groups * p.blocks, h_step = w.groups * f;
  const int first_b = f + w.chunk, b_low = first_b & ~15, b_skip = first_b & 15, b_block = first_b & 127;
  const int n = f - w.chunk < CHUNK ? f - w.chunk : CHUNK;    // columns of this chunk
  const uint64_t dh_end = reinterpret_cast<uint64_t>(p.dh) + static_cast<uint64_t>(p.rows) * f * 2;
  uint64_t dh = reinterpret_cast<uint64_t>(p.dh) + (static_cast<uint64_t>(w.row) * f + w.chunk) * 2;
  int64_t next = w.row;
  // the lane's own piece and, of three lanes, what is left over
  const int block = lane < 4 ? (w.chunk >> 7) + lane - 2 : (first_b >> 7) + lane - 4;
  auto piece_of_dh = [&](uint8_t* to, int i) {
    const uint64_t low = dh & ~15ull, at = low + 16 * i;
    if (at >= dh + 2 * n) return;
    if (at + 16 <= dh_end) {
      copy_async16(smem_u32(to + 16 * i), reinterpret_cast<const void*>(at));
    } else {
      for (uint64_t b = at; b < dh_end; ++b) to[b - low] = *reinterpret_cast<const uint8_t*>(b);
    }
  };
  auto fetch = [&](int slot) {
    if (next < live) {
      Slot& t = mine[slot];
      if (BACK) piece_of_dh(t.dh, lane);
      if (lane < 16) {
        if (16 * lane < n) copy_async16(smem_u32(t.a + 16 * lane), codes + w.chunk + 16 * lane);
      } else if (b_low + 16 * (lane - 16) < first_b + n) {
        copy_async16(smem_u32(t.b + 16 * (lane - 16)), codes + b_low + 16 * (lane - 16));
      }
      if (BACK && lane == 0) piece_of_dh(t.dh, 32);
      if (lane == 1 && b_low + 256 < first_b + n) copy_async16(smem_u32(t.b + 256), codes + b_low + 256);
      if (lane >= 2 && lane < 7 && block < p.blocks)
        copy_async4(smem_u32(lane < 4 ? &t.sa[lane - 2] : &t.sb[lane - 4]), scales + block);
    }
    codes += c_step;
    scales += s_step;
    dh += 2 * h_step;
    next += w.groups;
    copy_commit();
  };
  for (int s = 0; s + 1 < SLOTS; ++s) fetch(s);
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + w.row * p.C;
  __nv_bfloat16* hr = static_cast<__nv_bfloat16*>(p.h) + w.row * f;
  // where this row's dh begins in its first piece: 2 * f bytes further with every row
  uint32_t skip = (static_cast<uint32_t>(reinterpret_cast<uint64_t>(p.dh)) +
                   (static_cast<uint32_t>(w.row) * static_cast<uint32_t>(f) + w.chunk) * 2u) & 15u;
  const uint32_t skip_step = static_cast<uint32_t>(h_step) * 2u;
  int slot = 0, ahead = SLOTS - 1;
  for (int64_t row = w.row; row < live; row += w.groups) {
    __syncwarp();   // all are done with the slot that is filled now
    fetch(ahead);
    if (++ahead == SLOTS) ahead = 0;
    copy_wait(SLOTS - 1);
    __syncwarp();   // ... and see what the others copied
    const Slot& t = mine[slot];
    if (++slot == SLOTS) slot = 0;
    float2 a[4], b[4], h[4], d[4];
    smem_row_values<TYPE, 1>(a, t.a, 0, n, lane);
    smem_row_values<TYPE, 1>(b, t.b + b_skip, 0, n, lane);
    if (BACK) smem_row_values<ROW_BF16, 1>(d, t.dh + skip, 0, n, lane);
    skip = (skip + skip_step) & 15u;
    const float2 lo = both(t.sa[0]), hi = both(t.sa[1]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      a[j] = __fmul2_rn(a[j], j < 2 ? lo : hi);
      b[j] = __fmul2_rn(b[j], make_float2(t.sb[(b_block + 64 * j + lane) >> 7],
                                          t.sb[(b_block + 64 * j + 32 + lane) >> 7]));
    }
    swiglu_pairs<BACK>(a, b, d, h);
    if (BACK || p.out) {
      store_values<1>(out + w.chunk, ROW_BF16, 0, n, lane, reinterpret_cast<const float*>(a));
      store_values<1>(out + f + w.chunk, ROW_BF16, 0, n, lane, reinterpret_cast<const float*>(b));
    }
    if (p.h) store_values<1>(hr + w.chunk, ROW_BF16, 0, n, lane, reinterpret_cast<const float*>(h));
    out += 2 * h_step;
    hr += h_step;
  }
  griddep_launch();
}

// One CTA per token, whose warps share its columns: dyp[p_j] = w_j dy[t], dw_j = <dy[t], codes *
// scales of row p_j>, 0 for a dropped slot.  dy and the slots' codes of the next chunks come through
// shared memory (rows8.cuh), their scales by one load of the warp a chunk ahead: lane 2 j + h holds
// the one of slot j's block h.  The codes of a lane's eight columns are summed before their scale
// multiplies them.  A warp to a token left the card's last round of tokens a third empty (4096 tokens
// of 7168 columns, 8 slots each: 137 us).
constexpr int COMBINE_WARPS = 8;
template <int KMAX, int TYPE>
__global__ void __launch_bounds__(32 * COMBINE_WARPS)
combine_bwd_kernel(const void* __restrict__ dy, const uint8_t* __restrict__ codes, int64_t ld,
                   const float* __restrict__ scales, int blocks, const float* __restrict__ topk_w,
                   const int32_t* __restrict__ dest_row, int64_t T, int k, int d, int64_t rows_cap,
                   __nv_bfloat16* __restrict__ dyp, float* __restrict__ dw, int* err) {
  griddep_wait();
  struct Slot { uint8_t dy[2 * CHUNK]; uint8_t codes[KMAX][CHUNK]; };
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float dots[COMBINE_WARPS][8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  Slot* mine = reinterpret_cast<Slot*>(smem) + warp * SLOTS;
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
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
    int p[KMAX];
    float wt[KMAX];
    float2 dot[KMAX];
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
      p[j] = __shfl_sync(FULL_MASK, my_p, j);
      wt[j] = __shfl_sync(FULL_MASK, my_w, j);
      dot[j] = both(0.0f);
    }
    // the slot and block whose scale this lane fetches
    const int of = __shfl_sync(FULL_MASK, my_p, lane >> 1);
    const bool mine_lives = lane < 2 * KMAX && of >= 0;
    const float* sr = scales + (mine_lives ? static_cast<int64_t>(of) * blocks + (lane & 1) : 0);
    const uint8_t* row = static_cast<const uint8_t*>(dy) + t * d * 2;
    auto scale_of = [&](int chunk) {
      return mine_lives && chunk + 128 * (lane & 1) < d ? sr[chunk >> 7] : 0.0f;
    };
    auto fetch = [&](int chunk, int slot) {
      if (chunk < d) {
        Slot& s = mine[slot];
        copy_chunk(s.dy, row, ROW_BF16, chunk, d, lane);
#pragma unroll
        for (int j = 0; j < KMAX; ++j)
          if (p[j] >= 0) copy_chunk(s.codes[j], codes + static_cast<int64_t>(p[j]) * ld, TYPE, chunk, d, lane);
      }
      copy_commit();
    };
    const int step = warps * CHUNK;
    for (int s = 0; s + 1 < SLOTS; ++s) fetch(warp * CHUNK + s * step, s);
    float sc_next = scale_of(warp * CHUNK);
    int slot = 0, ahead = SLOTS - 1;
    for (int chunk = warp * CHUNK; chunk < d; chunk += step) {
      fetch(chunk + (SLOTS - 1) * step, ahead);
      if (++ahead == SLOTS) ahead = 0;
      const float sc = sc_next;
      sc_next = chunk + step < d ? scale_of(chunk + step) : 0.0f;
      copy_wait(SLOTS - 1);
      const Slot& s = mine[slot];
      if (++slot == SLOTS) slot = 0;
      const int c = chunk + 8 * lane;
      const bool in = c < d;
      float2 g[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) g[q] = both(0.0f);
      if (in) slot_values(g, s.dy, ROW_BF16, lane);
#pragma unroll
      for (int j = 0; j < KMAX; ++j) {
        const float scale = __shfl_sync(FULL_MASK, sc, 2 * j + (lane >> 4));
        if (p[j] < 0 || !in) continue;
        float2 f[4], v = both(0.0f);
        slot_values(f, s.codes[j], TYPE, lane);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          v = __ffma2_rn(g[q], f[q], v);
          f[q] = __fmul2_rn(g[q], both(wt[j]));
        }
        dot[j] = __ffma2_rn(v, both(scale), dot[j]);
        store_pairs(dyp + static_cast<int64_t>(p[j]) * d, ROW_BF16, c, f);
      }
    }
    float all = 0.0f;
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
      const float v = warp_sum(dot[j].x + dot[j].y);
      if (j == lane) all = v;
    }
    if (warps > 1) {
      if (lane < 8) dots[warp][lane] = all;
      __syncthreads();
      if (warp == 0 && lane < k) {
        all = 0.0f;
        for (int i = 0; i < warps; ++i) all += dots[i][lane];
      }
    }
    if (warp == 0 && lane < k) dw[t * k + lane] = all;
    if (t + gridDim.x < T) __syncthreads();
  }
  griddep_launch();
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

template <typename K>
cudaError_t launch_walk(K kern, const CkptArgs& a, int C, cudaStream_t st, int warps = 64) {
  const WalkGrid g = walk_grid(a.rows, C, warps);
  return launch_pdl(kern, g.grid, dim3(WALK_THREADS), 0, st, 1, a, g.per, g.groups);
}

}  // namespace

cudaError_t launch_ckpt_save(const CkptArgs& a, cudaStream_t st) {
  const int xs = row_size(a.x_type);
  return by_types(a, [&](auto x, auto format) {
    constexpr int X = decltype(x)::value, F = decltype(format)::value;
    if (a.C % 8 == 0 && rows_fit(a.x, a.ldx, xs, 8)) return launch_walk(save_ring_kernel<X == ROW_BF16 ? 4 : 2, X, F>, a, a.C, st, 128);
    if (a.C % 2 == 0 && rows_fit(a.x, a.ldx, xs, 2)) return launch_walk(save_kernel<2, 2, X, F>, a, a.C, st);
    return launch_walk(save_kernel<1, 2, X, F>, a, a.C, st);
  });
}

cudaError_t launch_ckpt_load(const CkptArgs& a, cudaStream_t st) {
  const int xs = row_size(a.x_type);
  return by_types(a, [&](auto x, auto format) {
    constexpr int X = decltype(x)::value, F = decltype(format)::value;
    if (a.C % 8 == 0 && rows_fit(a.out, a.ldx, xs, 8)) return launch_walk(load_ring_kernel<X, F>, a, a.C, st, 256);
    if (a.C % 2 == 0 && rows_fit(a.out, a.ldx, xs, 2)) return launch_walk(load_kernel<2, 2, X, F>, a, a.C, st);
    return launch_walk(load_kernel<1, 2, X, F>, a, a.C, st);
  });
}

cudaError_t launch_ckpt_swiglu(const CkptArgs& a, cudaStream_t st) {
  const int f = a.C / 2;
  auto pick = [&](auto back, auto format) {
    constexpr bool B = decltype(back)::value;
    constexpr int T = decltype(format)::value == MOE_CKPT_INT8 ? ROW_INT8 : ROW_E4M3;
    // (dh, [a | b] and h are dense from 16-byte addresses: the width alone decides)
    if (f % 8 == 0) return launch_walk(swiglu_ring_kernel<B, T>, a, f, st, 256);
    return launch_walk(swiglu_odd_kernel<B, T>, a, f, st, 64);
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
  // warps to a token: a chunk each while there are few tokens, else about four
  const int chunks = (d + CHUNK - 1) / CHUNK;
  int warps = T < 4 * row_sms() ? chunks : (chunks + 3) / 4;
  if (warps > COMBINE_WARPS) warps = COMBINE_WARPS;
  const int64_t most = int64_t(1) << 30;
  const dim3 grid(static_cast<unsigned>(T < most ? T : most));
  auto go = [&](auto slots, auto type) {
    constexpr int KMAX = decltype(slots)::value;
    constexpr auto kern = combine_bwd_kernel<KMAX, decltype(type)::value>;
    const int smem = warps * SLOTS * (2 + KMAX) * CHUNK;
    const cudaError_t e = allow_smem<kern>(smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, grid, dim3(32 * warps), smem, st, 1, dy, static_cast<const uint8_t*>(codes), ld,
                      scales, (d + 127) / 128, topk_w, dest_row, T, k, d, rows_cap,
                      static_cast<__nv_bfloat16*>(dyp), dw, err);
  };
#define MOE_COMBINE(KM) \
  (format == MOE_CKPT_INT8                                                                       \
       ? go(std::integral_constant<int, KM>(), std::integral_constant<int, ROW_INT8>())          \
       : go(std::integral_constant<int, KM>(), std::integral_constant<int, ROW_E4M3>()))
  if (k <= 2) return MOE_COMBINE(2);
  if (k <= 4) return MOE_COMBINE(4);
  if (k <= 6) return MOE_COMBINE(6);
  return MOE_COMBINE(8);
#undef MOE_COMBINE
}

}  // namespace moe
