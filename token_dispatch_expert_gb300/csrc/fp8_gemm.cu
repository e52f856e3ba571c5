// fp8_gemm.cu -- products of E4M3 operands with one scale for each block of 128: a grouped
// product over the rows of each expert, and its weight gradient over each expert's tokens.
//
//   product       out[p][n]   = sum_kb sa[p][kb] sb[g][n/128][kb] sum_{k in kb} a[p][k] b[g][n][k]
//   weight grad   dW[g][m][n] = sum_kb sa[kb][m] sb[kb][n] sum_{t in kb} a[m][t] b[n][t]
//
// The inner sums are tensor-core products over one block (tcgen05.mma kind::f8f6f4, K 32 each),
// accumulated in fp32 in TMEM; the outer sum runs in fp32 registers of the epilogue warps,
// because a scale is any fp32 number and changes with every block.  So an accumulator leaves
// TMEM once per block, which is what bounds these kernels: 128 x 256 sums take 256 cycles of the
// SM's fp32 lanes (512 with per-column scales), next to 512 cycles of MMA, and every hand-over
// between the two costs a round trip of barriers.  Four accumulators of 128 columns rotate (two
// halves of a tile, two blocks), so that one's round trip lies behind the MMAs of the others;
// eight epilogue warps, four per half, own 128 sums a thread.  Another warp brings the scales into
// a ring in shared memory, up to eight blocks ahead.
//
// Measured: 2048 rows by 28672 x 4096 of two experts 177 us, 2.7 PFLOP/s at 1.9 GHz (840 cycles a
// block); without the additions it takes 153 us, without MMAs 162, without either 124, the rate
// of the operand loads (53 bytes an SM and cycle from L2).  8192 rows of eight experts 785 us, and
// 905 us (2.1 PFLOP/s) for as long as the power cap holds the clock down.  65,536 rows over 128
// experts by 1536 x 2048 222 us in a short run, 240 us (1.7 PFLOP/s) in a long one; weight gradients
// 2048 x 768 of 128 experts 194 us, 3.0 TB/s, where the additions are twice as many and the tiles
// short (135 us without them).
//
// Tiles are 256 x 256 on a CTA pair (cta_group::2, each CTA holding 128 rows of A and of B, which
// halves the operand bytes per multiply-add) or 128 x 256 on one CTA, where a pair's second half
// would mostly be padding.  A finished tile leaves through shared memory, one 32 x 128-byte box
// per warp, by TMA stores that overlap the next tile; boxes that a segment's end cuts, or a
// row's end off 16 bytes, and outputs whose rows TMA cannot address, are copied row by row from the
// same box.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cstddef>
#include <mutex>
#include <type_traits>

#include "fp8_tiles.cuh"

namespace moe {
namespace {

constexpr int FG_TILE_N = 256;
// Warps 0 - 3: producer, MMA issuer, scale loader, MMA issuer; warps 4 - 11: epilogue.  Launched
// with 168 registers a thread (64,512 in all); the first four warps hand most of theirs to the
// others: 128 * 56 + 256 * 224 = 64,512.
constexpr int FG_THREADS = 384;
constexpr int FG_EPI_WARP0 = 4;
constexpr int FG_EPI_WARPS = 8;
constexpr int FG_BUFS = 4;                // accumulators: (block & 1) * 2 + half
constexpr uint32_t FG_TMEM_COLS = 512;
constexpr int FG_BOX_BYTES = 32 * 128;    // a piece of a finished tile: 32 rows x 128 bytes
constexpr int FG_BOXES = 2;               // per epilogue warp

template <int PAIR>
struct FgGeo {
  static constexpr int TILE_M = 128 * PAIR;
  static constexpr int A_BYTES = 128 * FG_BK;
  static constexpr int B_ROWS = FG_TILE_N / PAIR;       // this CTA's rows of b
  static constexpr int B_BYTES = B_ROWS * FG_BK;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGES = PAIR == 2 ? 4 : 3;
};

// Scales of one block: a row's in row[], and in col[] the columns' (weight gradient) or the two
// 128-column blocks' (product).
struct alignas(16) FgScales {
  float row[128];
  float col[FG_TILE_N];
};
constexpr int FG_CHUNK = 4;    // blocks that are loaded, handed over and freed together

struct FgCtl {
  uint64_t full[5], empty[5], tfull[FG_BUFS], tempty[FG_BUFS], sfull[2], sempty[2], drain[2];
  uint32_t tmem_base;
  int abort, bad;
  int gstart[FG_MAX_G + 1];
  int tprefix[FG_MAX_G + 1];    // tiles before each group
  int kbpre[FG_MAX_G + 1];      // wgrad: token blocks before each group
  int order[FG_MAX_G];          // wgrad: the groups by their number of blocks, most first
  FgScales scales[2][FG_CHUNK];
};
static_assert(offsetof(FgCtl, scales) % 16 == 0, "read as float4");

template <int PAIR>
constexpr size_t fg_smem() {
  return FgGeo<PAIR>::STAGES * FgGeo<PAIR>::STAGE_BYTES + FG_EPI_WARPS * FG_BOXES * FG_BOX_BYTES +
         sizeof(FgCtl) + 1024;
}
static_assert(fg_smem<1>() <= 232448 && fg_smem<2>() <= 232448, "227 KB per CTA");

struct FgParams {
  int G, N, K;                  // K: of the product; wgrad: M
  int rows;
  int n_tiles, m_tiles;         // m_tiles: wgrad
  int kb;                       // product: blocks along K; wgrad: token block capacity
  int nb;                       // product: 128-row blocks of b per group
  const int32_t* offsets;
  const float* sa;
  const float* sb;
  void* out;
  long long ldo;
  int tma_out;                  // the output map is usable
  int tma_last;                 // product: the last column at which a box may begin to be stored by it
  int* err;
};

__device__ __forceinline__ void st_shared_v4(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}

// The first `nr` rows of a warp's box (32 rows x 128 bytes, 16-byte pieces XOR-swizzled by row) to
// rows of `out` starting at element `off`, `nc` columns of them: 4 bytes per lane and row.
template <bool F32>
__device__ __forceinline__ void copy_box(const uint8_t* box, void* out, long long off,
                                         long long ldo, int nr, int nc, int lane) {
  const uint8_t* src = box + (lane & 3) * 4;
  const int piece = lane >> 2;
  constexpr int SIZE = F32 ? 4 : 2;
  uint8_t* dst = static_cast<uint8_t*>(out) + off * SIZE + 4 * lane;
  const long long step = ldo * SIZE;
  const bool one = F32 ? lane < nc : 2 * lane < nc;      // of this lane's columns, any in the row
  const bool two = F32 || 2 * lane + 1 < nc;             // bf16: both
  // 4-byte stores: always possible in fp32, in bf16 where every row starts on 4 bytes
  const bool wide =
      F32 || ((reinterpret_cast<uintptr_t>(dst) | static_cast<uintptr_t>(step)) & 3u) == 0;
#pragma unroll 1
  for (int i0 = 0; i0 < nr; i0 += 8) {   // eight rows' reads before their stores
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w[i] = *reinterpret_cast<const uint32_t*>(src + (i0 + i) * 128 + ((piece ^ i) << 4));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (one && i0 + i < nr) {
        if (wide && two) {
          *reinterpret_cast<uint32_t*>(dst) = w[i];
        } else {
          *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(w[i]);
          if (two) *reinterpret_cast<uint16_t*>(dst + 2) = static_cast<uint16_t>(w[i] >> 16);
        }
      }
      dst += step;
    }
  }
}

// tmC: the output as [groups][rows][columns] (product: one group), box 128 bytes x 32 x 1.
template <bool WG, bool F32, int PAIR>
__global__ void __launch_bounds__(FG_THREADS, 1)
fp8_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                const __grid_constant__ CUtensorMap tmC, const FgParams p) {
  griddep_wait();   // see common.cuh: dependent launches
  using GE = FgGeo<PAIR>;
  constexpr int STAGES = GE::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* boxes = smem + STAGES * GE::STAGE_BYTES;
  FgCtl* ctl = reinterpret_cast<FgCtl*>(boxes + FG_EPI_WARPS * FG_BOXES * FG_BOX_BYTES);
  // as uniform values, here and below, the product's epilogue needs no spills (wide product 824 ->
  // 786 us); the weight gradient's is 1% slower with them
  const int warp = WG ? threadIdx.x >> 5 : fg_uniform(threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const uint32_t smem_base = smem_u32(smem);
  volatile int* abort_flag = &ctl->abort;
  const int rank = PAIR == 2 ? static_cast<int>(cluster_ctarank()) : 0;
  const int unit = blockIdx.x / PAIR, num_units = gridDim.x / PAIR;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(smem_u32(&ctl->full[s]), 1);
      mbar_init(smem_u32(&ctl->empty[s]), 2);   // both halves' MMAs
    }
    for (int b = 0; b < FG_BUFS; ++b) {
      mbar_init(smem_u32(&ctl->tfull[b]), 1);
      mbar_init(smem_u32(&ctl->tempty[b]), FG_EPI_WARPS / 2 * PAIR);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&ctl->sfull[b]), 32);
      mbar_init(smem_u32(&ctl->sempty[b]), FG_EPI_WARPS);
      mbar_init(smem_u32(&ctl->drain[b]), 1);
    }
    fence_mbar_init();
    ctl->abort = 0;
    ctl->bad = 0;
  }
  if (threadIdx.x == 32) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmC);
  }
  for (int g = threadIdx.x; g <= p.G; g += FG_THREADS)
    ctl->gstart[g] = p.offsets ? p.offsets[g] : (g ? p.rows : 0);
  __syncthreads();
  if (warp == 0) {
    const int per = (p.G + 31) / 32;
    auto tiles_of = [&](int a, int b) {
      return WG ? p.m_tiles * p.n_tiles : b > a ? ceil_div(b - a, GE::TILE_M) * p.n_tiles : 0;
    };
    auto blocks_of = [&](int a, int b) { return b > a ? ceil_div(b - a, 128) : 0; };
    int local = 0, local_kb = 0, bad = 0;
    for (int i = 0; i < per; ++i) {
      const int g = lane * per + i;
      if (g < p.G) {
        const int a = ctl->gstart[g], b = ctl->gstart[g + 1];
        if (b < a || a < 0 || b > p.rows) bad = 1;
        else {
          local += tiles_of(a, b);
          local_kb += blocks_of(a, b);
        }
      }
    }
    const int incl = warp_incl_scan(local), incl_kb = warp_incl_scan(local_kb);
    int run = incl - local, run_kb = incl_kb - local_kb;
    if (ctl->gstart[0] != 0) bad = 1;
    bad = __any_sync(FULL_MASK, bad);
    if (!bad) {
      for (int i = 0; i < per; ++i) {
        const int g = lane * per + i;
        if (g < p.G) {
          const int a = ctl->gstart[g], b = ctl->gstart[g + 1];
          ctl->tprefix[g] = run;
          ctl->kbpre[g] = run_kb;
          run += tiles_of(a, b);
          run_kb += blocks_of(a, b);
        }
      }
    }
    if (lane == 31) {
      ctl->tprefix[p.G] = incl;
      ctl->kbpre[p.G] = incl_kb;
    }
    if (lane == 0 && bad) {
      ctl->bad = 1;
      if (blockIdx.x == 0) flag_error(p.err, MOE_DEVERR_BAD_OFFSETS);
    }
  }
  if (warp == 1) {
    if (PAIR == 2) {
      tmem_alloc_pair(smem_u32(&ctl->tmem_base), FG_TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(&ctl->tmem_base), FG_TMEM_COLS);
      tmem_relinquish();
    }
  }
  if (WG) {
    for (int g = threadIdx.x; g < p.G; g += FG_THREADS) {
      auto blocks_of = [&](int i) { return ceil_div(ctl->gstart[i + 1] - ctl->gstart[i], 128); };
      const int n = blocks_of(g);
      int before = 0;
      for (int i = 0; i < p.G; ++i) {
        const int m = blocks_of(i);
        before += m > n || (m == n && i < g);
      }
      ctl->order[before] = g;
    }
  }
  tc_fence_before();
  if (PAIR == 2) cluster_sync_all();
  else __syncthreads();
  tc_fence_after();
  const int total = fg_uniform(ctl->bad ? 0 : ctl->tprefix[p.G]);
  const uint32_t tmem_base =
      WG ? ctl->tmem_base : static_cast<uint32_t>(fg_uniform(static_cast<int>(ctl->tmem_base)));

  // tile -> group, row tile, column tile; row tiles run fastest, so the CTAs at work share the
  // group's weight rows in L2.  Every role walks its tiles in ascending order, so the group is
  // found by going on from the last one; with fewer than 2^16 column tiles the fp32 quotient is
  // off by at most one, which the remainder corrects.  The weight gradient's groups have equally
  // many tiles and unequal ones: its order is the longest first.
  int pos = 0;
  auto map_tile = [&](int tile, int& g, int& mt, int& nt) {
    while (ctl->tprefix[pos + 1] <= tile) ++pos;
    g = WG ? ctl->order[pos] : pos;
    const int local = tile - ctl->tprefix[pos];
    const int mtg =
        WG ? p.m_tiles : ceil_div(ctl->gstart[g + 1] - ctl->gstart[g], GE::TILE_M);
    nt = static_cast<int>(__fdividef(static_cast<float>(local), static_cast<float>(mtg)));
    mt = local - nt * mtg;
    if (mt < 0) {
      --nt;
      mt += mtg;
    } else if (mt >= mtg) {
      ++nt;
      mt -= mtg;
    }
  };
  // tiles are dealt out in rounds, the weight gradient's in turns from the first unit to the last
  // and back, so that nobody gets the longest of every round
  const int first_step = WG ? 2 * (num_units - unit) - 1 : num_units;
  auto next_step = [&](int step) { return WG ? 2 * num_units - step : step; };
  auto blocks = [&](int g) { return WG ? ctl->kbpre[g + 1] - ctl->kbpre[g] : p.kb; };

  if (warp < FG_EPI_WARP0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;" ::: "memory");
    if (warp == 0) {
      // -------------------------------------------------------------- producer
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int tile = unit, step = first_step; tile < total && ok;
           tile += step, step = next_step(step)) {
        int g, mt, nt;
        map_tile(tile, g, mt, nt);
        const int nkb = fg_uniform(blocks(g));
        int x = fg_uniform(WG ? ctl->kbpre[g] * FG_BK : 0);
        const int arow =
            fg_uniform((WG ? 0 : ctl->gstart[g]) + mt * GE::TILE_M + 128 * rank);
        // this CTA's rows of b: one CTA all 256; of a pair, 64 of each 128-column half
        const int brow = fg_uniform((WG ? 0 : g * p.N) + nt * FG_TILE_N + 64 * rank);
        for (int kb = 0; kb < nkb; ++kb, x += FG_BK) {
          if (!fg_wait(smem_u32(&ctl->empty[s]), ph ^ 1u, abort_flag, p.err)) {
            ok = false;
            break;
          }
          if (fg_elect()) {
            const uint32_t sa = smem_base + s * GE::STAGE_BYTES;
            const uint32_t full = smem_u32(&ctl->full[s]);
            // the leader's single arrive announces both CTAs' bytes
            if (rank == 0) mbar_arrive_expect_tx(full, PAIR * GE::STAGE_BYTES);
            if (PAIR == 2) {
              const uint32_t lead = mapa_shared(full, 0);
              tma_load_2d_pair(sa, &tmA, lead, x, arow);
              tma_load_2d_pair(sa + GE::A_BYTES, &tmB, lead, x, brow);
              tma_load_2d_pair(sa + GE::A_BYTES + 64 * FG_BK, &tmB, lead, x, brow + 128);
            } else {
              tma_load_2d(sa, &tmA, full, x, arow);
              tma_load_2d(sa + GE::A_BYTES, &tmB, full, x, brow);
            }
          }
          __syncwarp();
          if (++s == STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      griddep_launch();
      const int s_end = s;
      const uint32_t ph_end = ph;
      for (int i = 0; i < STAGES && ok; ++i) {   // every copy of this CTA has been consumed
        ok = fg_wait(smem_u32(&ctl->empty[s]), ph ^ 1u, abort_flag, p.err);
        if (++s == STAGES) {
          s = 0;
          ph ^= 1u;
        }
      }
      // (the leader's barriers count both CTAs' bytes, and neither leaves before the other)
      if (!ok && rank == 0) fg_drain_copies<STAGES>(ctl->full, s_end, ph_end);
    } else if (warp & 1) {
      // -------------------------------------------------------------- MMA issuers (the leader's)
      // warp 1 the tile's left half, warp 3 the right one, so that neither waits for the other's
      // accumulator
      if (rank == 0) {
        const uint32_t h = static_cast<uint32_t>(warp >> 1);
        int s = 0;
        uint32_t ph = 0;
        uint32_t it = 0;   // blocks issued
        bool ok = true;
        const uint32_t tmem = static_cast<uint32_t>(fg_uniform(static_cast<int>(tmem_base)));
        const uint64_t da0 = make_smem_desc(smem_base, 16, 1024);
        const uint64_t db0 =
            make_smem_desc(smem_base + GE::A_BYTES + h * (GE::B_BYTES / 2), 16, 1024);
        for (int tile = unit, step = first_step; tile < total && ok;
           tile += step, step = next_step(step)) {
          int nkb = p.kb;
          if (WG) {
            int g, mt, nt;
            map_tile(tile, g, mt, nt);
            nkb = fg_uniform(blocks(g));
          }
          for (int kb = 0; kb < nkb; ++kb, ++it) {
            const uint32_t buf = (it & 1u) * 2u + h;
            if (!fg_wait(smem_u32(&ctl->full[s]), ph, abort_flag, p.err) ||
                !fg_wait(smem_u32(&ctl->tempty[buf]), ((it >> 1) & 1u) ^ 1u, abort_flag, p.err)) {
              ok = false;
              break;
            }
            tc_fence_after();
            if (fg_elect()) {
              const uint64_t da = da0 + static_cast<uint32_t>(s * (GE::STAGE_BYTES >> 4));
              const uint64_t db = db0 + static_cast<uint32_t>(s * (GE::STAGE_BYTES >> 4));
#pragma unroll
              for (uint32_t kk = 0; kk < FG_BK / 32; ++kk) {   // 32 bytes on, in 16-byte units
                if (PAIR == 2)
                  fg_mma_pair(tmem + buf * 128, da + 2 * kk, db + 2 * kk, fg_idesc(256, 128),
                              kk != 0);
                else
                  fg_mma(tmem + buf * 128, da + 2 * kk, db + 2 * kk, fg_idesc(128, 128), kk != 0);
              }
              if (PAIR == 2) {
                tc_commit_pair_mc(smem_u32(&ctl->tfull[buf]), 0x3);
                tc_commit_pair_mc(smem_u32(&ctl->empty[s]), 0x3);
              } else {
                tc_commit(smem_u32(&ctl->tfull[buf]));
                tc_commit(smem_u32(&ctl->empty[s]));
              }
            }
            __syncwarp();
            if (++s == STAGES) {
              s = 0;
              ph ^= 1u;
            }
          }
        }
        if (!ok && lane == 0) {   // gave up: wait (bounded) for the MMAs in flight
          const uint32_t drain = smem_u32(&ctl->drain[h]);
          if (PAIR == 2) tc_commit_pair(drain);
          else tc_commit(drain);
          const long long t0 = clock64();
          while (!mbar_try_wait(drain, 0) && clock64() - t0 < FG_WAIT_BUDGET / 4) {
          }
        }
        __syncwarp();
      }
    } else {
      // -------------------------------------------------------------- scale loader (warp 2)
      uint32_t ci = 0;   // chunks loaded
      bool ok = true;
      for (int tile = unit, step = first_step; tile < total && ok;
           tile += step, step = next_step(step)) {
        int g, mt, nt;
        map_tile(tile, g, mt, nt);
        const int nkb = blocks(g);
        const int m0 = mt * GE::TILE_M + 128 * rank;
        const int rows_g = WG ? p.K : ctl->gstart[g + 1] - ctl->gstart[g];
        for (int k0 = 0; k0 < nkb; k0 += FG_CHUNK, ++ci) {
          const uint32_t buf = ci & 1u;
          if (!fg_wait(smem_u32(&ctl->sempty[buf]), ((ci >> 1) & 1u) ^ 1u, abort_flag, p.err)) {
            ok = false;
            break;
          }
          const int n = min(FG_CHUNK, nkb - k0);
          FgScales* dst = ctl->scales[buf];
          // rows and columns past the end get 0; their sums are not stored
          if (WG) {
            for (int j = 0; j < n; ++j) {
              const long long blk = ctl->kbpre[g] + k0 + j;
              const float* a = p.sa + blk * p.K + m0;
              const float* b = p.sb + blk * p.N + nt * FG_TILE_N;
#pragma unroll
              for (int r = lane; r < 128; r += 32)
                cp_async4(&dst[j].row[r], a + r, m0 + r < rows_g);
#pragma unroll
              for (int c = lane; c < FG_TILE_N; c += 32)
                cp_async4(&dst[j].col[c], b + c, nt * FG_TILE_N + c < p.N);
            }
          } else {
            const int j = lane & (FG_CHUNK - 1);
            const float* a = p.sa + static_cast<long long>(ctl->gstart[g] + m0) * p.kb + k0 + j;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int r = (lane >> 2) + 8 * i;
              cp_async4(&dst[j].row[r], a + static_cast<long long>(r) * p.kb,
                        j < n && m0 + r < rows_g);
            }
            if (lane < 2 * FG_CHUNK) {
              const int blk = min(2 * nt + (lane >> 2), p.nb - 1);
              cp_async4(&dst[j].col[lane >> 2],
                        p.sb + (static_cast<long long>(g) * p.nb + blk) * p.kb + k0 + j, j < n);
            }
          }
          cp_async_arrive(smem_u32(&ctl->sfull[buf]));
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;" ::: "memory");
    // ---------------------------------------------------------------- epilogue (8 warps)
    const int q = warp & 3;                          // the lane quarter this warp may read
    const int hh = (warp - FG_EPI_WARP0) >> 2;       // which 128 of the 256 columns
    uint8_t* my_boxes = boxes + (warp - FG_EPI_WARP0) * FG_BOXES * FG_BOX_BYTES;
    // this half's two accumulators: TMEM address, barriers (the leader counts both CTAs' warps)
    const uint32_t taddr0 = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + 128 * hh;
    const uint32_t tfull0 = smem_u32(&ctl->tfull[hh]);
    const uint32_t tempty0 =
        PAIR == 2 ? mapa_shared(smem_u32(&ctl->tempty[hh]), 0) : smem_u32(&ctl->tempty[hh]);
    uint32_t it = 0;   // blocks added
    uint32_t ci = 0;   // scale chunks used up
    bool ok = true;
    for (int tile = unit, step = first_step; tile < total && ok;
           tile += step, step = next_step(step)) {
      int g, mt, nt;
      map_tile(tile, g, mt, nt);
      const int nkb = blocks(g);
      float2 acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = make_float2(0.0f, 0.0f);
      for (int left = nkb; left > 0 && ok; left -= FG_CHUNK, ++ci) {
        if (!fg_wait(smem_u32(&ctl->sfull[ci & 1u]), (ci >> 1) & 1u, abort_flag, p.err)) {
          ok = false;
          break;
        }
        const FgScales* sc = ctl->scales[ci & 1u];
        const int n = min(left, FG_CHUNK);
        for (int j = 0; j < n; ++j, ++sc, ++it) {
          const uint32_t par = it & 1u;
          float s = sc->row[32 * q + lane];
          if (!WG) s *= sc->col[hh];
          if (!fg_wait(tfull0 + par * 16, (it >> 1) & 1u, abort_flag, p.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          // 64 columns at a time; 32 where the column scales take registers too
          constexpr int W = WG ? 32 : 64;
#pragma unroll
          for (int c = 0; c < 128 / W; ++c) {
            uint32_t d[W];
            if constexpr (WG) tmem_ld32(taddr0 + par * 256 + W * c, d);
            else tmem_ld64(taddr0 + par * 256 + W * c, d);
            tmem_ld_wait();
            if (c == 128 / W - 1) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) {   // the accumulator is free
                if (PAIR == 2) mbar_arrive_remote(tempty0 + par * 16);
                else mbar_arrive(tempty0 + par * 16);
              }
            }
            const float2 s2 = make_float2(s, s);
            auto sums = [&](int i) {
              return make_float2(__uint_as_float(d[2 * i]), __uint_as_float(d[2 * i + 1]));
            };
            if constexpr (WG) {
              const float4* cs = reinterpret_cast<const float4*>(sc->col + 128 * hh + W * c);
#pragma unroll
              for (int i = 0; i < W / 4; ++i) {
                const float4 f = cs[i];
                float2* a = acc + W / 2 * c + 2 * i;
                a[0] = __ffma2_rn(sums(2 * i), __fmul2_rn(make_float2(f.x, f.y), s2), a[0]);
                a[1] = __ffma2_rn(sums(2 * i + 1), __fmul2_rn(make_float2(f.z, f.w), s2), a[1]);
              }
            } else {
#pragma unroll
              for (int i = 0; i < W / 2; ++i)
                acc[W / 2 * c + i] = __ffma2_rn(sums(i), s2, acc[W / 2 * c + i]);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl->sempty[ci & 1u]));   // the scales are used up
      }
      const int lrow0 = mt * GE::TILE_M + 128 * rank + 32 * q;   // this warp's first row
      const int rows_g = WG ? p.K : ctl->gstart[g + 1] - ctl->gstart[g];
      const int nr = min(max(rows_g - lrow0, 0), 32);            // rows of it in the output
      const int n0 = nt * FG_TILE_N + 128 * hh;
      if (!ok || nr == 0 || n0 >= p.N) continue;
      // through the box, 128 bytes of a row at a time
      constexpr int BOX_COLS = F32 ? 32 : 64;
#pragma unroll
      for (int part = 0; part < 128 / BOX_COLS; ++part) {
        const int n = n0 + BOX_COLS * part;
        // a TMA store clips a row's end at 16 bytes only: where N lies off them, the last box
        // would write up to 14 bytes of a wider output's next columns (tma_last)
        const bool by_tma = WG ? p.tma_out : nr == 32 && n <= p.tma_last;
        uint8_t* box = my_boxes + part % FG_BOXES * FG_BOX_BYTES;
        const uint32_t box_row = smem_u32(box) + lane * 128;
        if (lane == 0) bulk_wait_group_read<FG_BOXES - 1>();   // the store before last has read it
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint4 v;
          if (F32) {
            const float2* x = acc + BOX_COLS / 2 * part + 2 * j;
            v = make_uint4(__float_as_uint(x[0].x), __float_as_uint(x[0].y),
                           __float_as_uint(x[1].x), __float_as_uint(x[1].y));
          } else {
            const float2* x = acc + BOX_COLS / 2 * part + 4 * j;
            v = make_uint4(pack_bf16x2(x[0].x, x[0].y), pack_bf16x2(x[1].x, x[1].y),
                           pack_bf16x2(x[2].x, x[2].y), pack_bf16x2(x[3].x, x[3].y));
          }
          st_shared_v4(box_row + ((j ^ (lane & 7)) << 4), v);
        }
        if (by_tma) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {   // a group even where there is nothing to store: one per box
            if (n < p.N)
              tma_store_3d(&tmC, smem_u32(box), n, WG ? lrow0 : ctl->gstart[g] + lrow0,
                           WG ? g : 0);
            bulk_commit_group();
          }
        } else {
          __syncwarp();
          const long long row =
              WG ? static_cast<long long>(g) * p.K + lrow0 : ctl->gstart[g] + lrow0;
          if (n < p.N) copy_box<F32>(box, p.out, row * p.ldo + n, p.ldo, nr, p.N - n, lane);
          if (lane == 0) bulk_commit_group();   // empty: one group per box, as above
          __syncwarp();
        }
      }
    }
    if (lane == 0) bulk_wait_group_all();   // stores done before exit
    __syncwarp();
  }
  tc_fence_before();
  if (PAIR == 2) cluster_sync_all();
  else __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    if (PAIR == 2) tmem_dealloc_pair(tmem_base, FG_TMEM_COLS);
    else tmem_dealloc(tmem_base, FG_TMEM_COLS);
  }
}

// ------------------------------------------------------------------ host side
PFN_cuTensorMapEncodeTiled_v12000 fg_encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                         cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// The output [groups][rows][cols] with rows `ld` elements apart, 128-byte swizzle, box 128 bytes
// x 32 rows x 1 group: a store never crosses into the next group's rows.  False where TMA
// cannot address it (a base or a row off 16 bytes).
bool fg_out_map(CUtensorMap* m, const void* base, bool fp32, uint64_t cols, uint64_t ld,
                uint64_t rows, uint64_t groups) {
  auto enc = fg_encode_fn();
  const uint64_t size = fp32 ? 4 : 2;
  if (!enc || (reinterpret_cast<uintptr_t>(base) & 15u) || ld * size % 16) return false;
  cuuint64_t dims[3] = {cols, rows, groups};
  cuuint64_t strides[2] = {ld * size, ld * rows * size};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / size), 32, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
             const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool WG, bool F32, int PAIR>
cudaError_t fg_launch(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tc,
                      const FgParams& p, cudaStream_t st) {
  auto kern = fp8_gemm_kernel<WG, F32, PAIR>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(fg_smem<PAIR>()));
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return launch_pdl(kern, dim3(static_cast<unsigned>(sms / PAIR * PAIR)), dim3(FG_THREADS),
                    fg_smem<PAIR>(), st, PAIR, ta, tb, tc, p);
}

}  // namespace

bool fp8_codes_map(CUtensorMap* m, const void* base, uint64_t cols, uint64_t ld, uint64_t rows,
                   uint32_t box_rows) {
  auto enc = fg_encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {ld};
  cuuint32_t box[2] = {FG_BK, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

cudaError_t launch_fp8_gemm(const Fp8GemmArgs& a, cudaStream_t st) {
  if (fp8_few_rows(a)) return launch_fp8_few(a, st);
  FgParams p{};
  p.G = a.G;
  p.N = a.N;
  p.K = a.K;
  p.rows = static_cast<int>(a.rows);
  p.n_tiles = (a.N + FG_TILE_N - 1) / FG_TILE_N;
  p.nb = (a.N + 127) / 128;
  p.offsets = a.offsets;
  p.sa = a.a_scales;
  p.sb = a.b_scales;
  p.out = a.out;
  p.ldo = a.ldo;
  p.err = a.err;
  // pairs: weight gradients of more than 128 rows (5% faster than one CTA at 2048 x 768 of 128
  // experts), products with 768 rows or more to the average segment.  Below, a pair's
  // padding of the last tile outweighs its cheaper operands where segments are uneven (249 us
  // against 231 for one CTA at 512 rows on average of 1536 x 2048, but 185 against 204 at 1024
  // rows of 28672 x 4096)
  const bool pair = a.wgrad ? a.K > 128 : a.rows >= 768 * static_cast<int64_t>(a.G);
  const uint32_t b_rows = pair ? 64 : 256;   // a box of b
  CUtensorMap ta, tb, tc;
  bool ok;
  if (a.wgrad) {
    const int tile_m = pair ? 256 : 128;
    p.m_tiles = (a.K + tile_m - 1) / tile_m;
    p.kb = static_cast<int>(fp8_token_blocks(a.rows, a.G));
    const uint64_t len = 128ull * static_cast<uint64_t>(p.kb);
    ok = fp8_codes_map(&ta, a.a, len, len, static_cast<uint64_t>(a.K), 128) &&
         fp8_codes_map(&tb, a.b, len, len, static_cast<uint64_t>(a.N), b_rows);
    p.tma_out = fg_out_map(&tc, a.out, a.out_fp32, static_cast<uint64_t>(a.N),
                           static_cast<uint64_t>(a.N), static_cast<uint64_t>(a.K),
                           static_cast<uint64_t>(a.G));
  } else {
    p.kb = (a.K + 127) / 128;
    ok = fp8_codes_map(&ta, a.a, static_cast<uint64_t>(a.K), static_cast<uint64_t>(a.lda),
                static_cast<uint64_t>(a.rows), 128) &&
         fp8_codes_map(&tb, a.b, static_cast<uint64_t>(a.K), static_cast<uint64_t>(a.ldb),
                static_cast<uint64_t>(a.G) * static_cast<uint64_t>(a.N), b_rows);
    p.tma_out = fg_out_map(&tc, a.out, a.out_fp32, static_cast<uint64_t>(a.N),
                           static_cast<uint64_t>(a.ldo), static_cast<uint64_t>(a.rows), 1);
  }
  if (!ok) return cudaErrorInvalidValue;
  const int edge = a.out_fp32 ? 4 : 8, box_cols = a.out_fp32 ? 32 : 64;
  p.tma_last = !p.tma_out ? -1 : a.N % edge == 0 ? a.N : a.N - box_cols;
  if (!p.tma_out) tc = ta;   // a valid map that no store uses
  auto go = [&](auto wg, auto f32) {
    return pair ? fg_launch<decltype(wg)::value, decltype(f32)::value, 2>(ta, tb, tc, p, st)
                : fg_launch<decltype(wg)::value, decltype(f32)::value, 1>(ta, tb, tc, p, st);
  };
  if (a.wgrad) return a.out_fp32 ? go(std::true_type{}, std::true_type{})
                                 : go(std::true_type{}, std::false_type{});
  return a.out_fp32 ? go(std::false_type{}, std::true_type{})
                    : go(std::false_type{}, std::false_type{});
}

}  // namespace moe
