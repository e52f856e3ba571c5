// fp8_few.cu -- the grouped product of fp8_gemm.cu for few rows: decoding, where every weight is
// read for a handful of tokens.
//
// The operands change places: D[n][t] = sum_kb sb[kb] sa[t][kb] sum_k b[n][k] a[t][k], the tensor
// core's 128 rows are weight rows and its 16 columns the tokens, so that a tile's rows are all
// work and its accumulators small: eight of them rotate in TMEM, and one epilogue warp per lane
// quarter adds them up, scaled, one thread per weight row.
//
// Bound by the weights' bytes, and in small calls by the chain of one tile's blocks.  A stage is
// 128 weight rows x 128 bytes (16 KB) and the tokens' 2 KB; ten of them, 160 KB of weights a CTA
// on its way, read eight experts of 4096 x 7168 for one token in 47 us, 5.0 TB/s with the launch
// (fp8_gemm's three 48 KB stages: 57 us, 4.1 TB/s).
//
// Where one tile's blocks are many and the tiles few, clusters of 2, 4 or 8 CTAs share a tile's
// blocks: each sums its part of them, sends each CTA of the cluster the columns that it owns
// through distributed shared memory, and every owner adds the parts in rank order and stores its
// columns (one row by 256 x 16384: 41.6 us alone, 27.4, 19.1 and 17.2 us by 2, 4 and 8).
#include <cuda.h>

#include <cstddef>

#include "fp8_tiles.cuh"

namespace moe {
namespace {

// Warps 0 - 3: producer, MMA issuer, scale loader, none; warps 4 - 7: epilogue.
constexpr int FW_THREADS = 256;
constexpr int FW_BUFS = 8;      // accumulators
constexpr int FW_CHUNK = 4;     // blocks whose scales are loaded and freed together
constexpr int FW_CHUNKS = 4;

constexpr int NT = 16;          // tokens of a tile
constexpr int FW_W_BYTES = 128 * FG_BK;
constexpr int FW_STAGE_BYTES = FW_W_BYTES + NT * FG_BK;   // a multiple of 1 KB
constexpr int FW_STAGES = 10;
constexpr int FW_PART_BYTES = NT * 128 * 4;
constexpr uint32_t FW_TMEM_COLS = FW_BUFS * NT;

struct FwCtl {
  uint64_t full[FW_STAGES], empty[FW_STAGES], tfull[FW_BUFS], tempty[FW_BUFS], sfull[FW_CHUNKS],
      sempty[FW_CHUNKS], pfull, pempty, drain;
  uint32_t tmem_base;
  int abort, bad;
  int gstart[FG_MAX_G + 1];
  int tprefix[FG_MAX_G + 1];    // tiles before each group
  alignas(16) float sa[FW_CHUNKS][FW_CHUNK][NT];
  float sb[FW_CHUNKS][FW_CHUNK];
};

constexpr size_t FW_SMEM = FW_STAGES * FW_STAGE_BYTES + FW_PART_BYTES + sizeof(FwCtl) + 1024;
static_assert(FW_SMEM <= 232448, "227 KB per CTA");

struct FwParams {
  int G, N, rows, kb, nb;
  int w_tiles;            // 128-row tiles of a group's weights
  int split;              // CTAs of a cluster
  const int32_t* offsets;
  const float* sa;
  const float* sb;
  void* out;
  long long ldo;
  int* err;
};

// 32 lanes x 16 consecutive fp32 columns
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// a store to, and an arrival (releasing to the cluster the stores ordered before it) in, another
// CTA's shared memory
__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr)
               : "memory");
}
__device__ __forceinline__ bool try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// mbar_wait_bounded over the cluster's arrivals
__device__ __forceinline__ bool fw_wait_cluster(uint32_t bar, uint32_t parity,
                                                volatile int* abort, int* err) {
  bool ok = try_wait_cluster(bar, parity);
  const long long t0 = clock64();
  while (!ok && !*abort) {
    ok = try_wait_cluster(bar, parity);
    if (!ok && clock64() - t0 > FG_WAIT_BUDGET) {
      flag_error(err, MOE_DEVERR_TIMEOUT);
      *abort = 1;
    }
  }
  return __all_sync(FULL_MASK, ok);
}

template <bool F32>
__device__ __forceinline__ void store1(void* out, long long at, float v) {
  if (F32) static_cast<float*>(out)[at] = v;
  else static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(v);
}

// tmW: the weights' codes [G N][K], box 128 x 128; tmT: the rows' codes, box 128 x NT.
template <bool F32>
__global__ void __launch_bounds__(FW_THREADS, 1)
fp8_few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmT,
               const FwParams p) {
  griddep_wait();   // see common.cuh: dependent launches
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  // parts of this CTA's columns, by the rank that summed them: [split][NT / split][128]
  float* part = reinterpret_cast<float*>(smem + FW_STAGES * FW_STAGE_BYTES);
  FwCtl* ctl = reinterpret_cast<FwCtl*>(smem + FW_STAGES * FW_STAGE_BYTES + FW_PART_BYTES);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t smem_base = smem_u32(smem);
  volatile int* abort_flag = &ctl->abort;
  const int split = p.split;
  const int rank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int unit = blockIdx.x / split, num_units = gridDim.x / split;

  if (threadIdx.x == 0) {
    for (int s = 0; s < FW_STAGES; ++s) {
      mbar_init(smem_u32(&ctl->full[s]), 1);
      mbar_init(smem_u32(&ctl->empty[s]), 1);
    }
    for (int b = 0; b < FW_BUFS; ++b) {
      mbar_init(smem_u32(&ctl->tfull[b]), 1);
      mbar_init(smem_u32(&ctl->tempty[b]), 4);
    }
    for (int b = 0; b < FW_CHUNKS; ++b) {
      mbar_init(smem_u32(&ctl->sfull[b]), 32);
      mbar_init(smem_u32(&ctl->sempty[b]), 4);
    }
    mbar_init(smem_u32(&ctl->pfull), 4 * split);
    mbar_init(smem_u32(&ctl->pempty), 4 * split);
    mbar_init(smem_u32(&ctl->drain), 1);
    fence_mbar_init();
    ctl->abort = 0;
    ctl->bad = 0;
  }
  if (threadIdx.x == 32) {
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmT);
  }
  for (int g = threadIdx.x; g <= p.G; g += FW_THREADS)
    ctl->gstart[g] = p.offsets ? p.offsets[g] : (g ? p.rows : 0);
  __syncthreads();
  if (warp == 0) {
    const int per = (p.G + 31) / 32;
    auto tiles_of = [&](int a, int b) { return b > a ? ceil_div(b - a, NT) * p.w_tiles : 0; };
    int local = 0, bad = 0;
    for (int i = 0; i < per; ++i) {
      const int g = lane * per + i;
      if (g < p.G) {
        const int a = ctl->gstart[g], b = ctl->gstart[g + 1];
        if (b < a || a < 0 || b > p.rows) bad = 1;
        else local += tiles_of(a, b);
      }
    }
    const int incl = warp_incl_scan(local);
    int run = incl - local;
    if (ctl->gstart[0] != 0) bad = 1;
    bad = __any_sync(FULL_MASK, bad);
    if (!bad) {
      for (int i = 0; i < per; ++i) {
        const int g = lane * per + i;
        if (g < p.G) {
          ctl->tprefix[g] = run;
          run += tiles_of(ctl->gstart[g], ctl->gstart[g + 1]);
        }
      }
    }
    if (lane == 31) ctl->tprefix[p.G] = incl;
    if (lane == 0 && bad) {
      ctl->bad = 1;
      if (blockIdx.x == 0) flag_error(p.err, MOE_DEVERR_BAD_OFFSETS);
    }
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&ctl->tmem_base), FW_TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  if (split > 1) cluster_sync_all();
  else __syncthreads();
  tc_fence_after();
  const int total = fg_uniform(ctl->bad ? 0 : ctl->tprefix[p.G]);
  const uint32_t tmem_base = ctl->tmem_base;
  // this CTA's blocks of every tile
  const int kb_lo = static_cast<int>(static_cast<long long>(p.kb) * rank / split);
  const int nkb = static_cast<int>(static_cast<long long>(p.kb) * (rank + 1) / split) - kb_lo;

  // tile -> group, first row, weight tile; the weight tiles run fastest, token tiles of a group
  // (more than NT rows) follow one another and find its weights in L2
  auto map_tile = [&](int tile, int& g, int& row0, int& wt) {
    while (ctl->tprefix[g + 1] <= tile) ++g;
    const int local = tile - ctl->tprefix[g];
    const int tt = local / p.w_tiles;
    wt = local - tt * p.w_tiles;
    row0 = ctl->gstart[g] + tt * NT;
  };

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    int s = 0, g = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int tile = unit; tile < total && ok; tile += num_units) {
      int row0, wt;
      map_tile(tile, g, row0, wt);
      const int wrow = fg_uniform(g * p.N + wt * 128);
      const int trow = fg_uniform(row0);
      for (int kb = 0; kb < nkb; ++kb) {
        if (!fg_wait(smem_u32(&ctl->empty[s]), ph ^ 1u, abort_flag, p.err)) {
          ok = false;
          break;
        }
        if (fg_elect()) {
          const uint32_t sw = smem_base + s * FW_STAGE_BYTES;
          const uint32_t full = smem_u32(&ctl->full[s]);
          mbar_arrive_expect_tx(full, FW_STAGE_BYTES);
          tma_load_2d(sw, &tmW, full, (kb_lo + kb) * FG_BK, wrow);
          tma_load_2d(sw + FW_W_BYTES, &tmT, full, (kb_lo + kb) * FG_BK, trow);
        }
        __syncwarp();
        if (++s == FW_STAGES) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    griddep_launch();
    const int s_end = s;
    const uint32_t ph_end = ph;
    for (int i = 0; i < FW_STAGES && ok; ++i) {   // every copy of this CTA has been consumed
      ok = fg_wait(smem_u32(&ctl->empty[s]), ph ^ 1u, abort_flag, p.err);
      if (++s == FW_STAGES) {
        s = 0;
        ph ^= 1u;
      }
    }
    if (!ok) fg_drain_copies<FW_STAGES>(ctl->full, s_end, ph_end);
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    int s = 0;
    uint32_t ph = 0;
    uint32_t it = 0;   // blocks issued
    bool ok = true;
    const uint32_t tmem = static_cast<uint32_t>(fg_uniform(static_cast<int>(tmem_base)));
    const uint64_t da0 = make_smem_desc(smem_base, 16, 1024);
    const uint64_t db0 = make_smem_desc(smem_base + FW_W_BYTES, 16, 1024);
    for (int tile = unit; tile < total && ok; tile += num_units) {
      for (int kb = 0; kb < nkb; ++kb, ++it) {
        const uint32_t buf = it % FW_BUFS;
        if (!fg_wait(smem_u32(&ctl->tempty[buf]), ((it / FW_BUFS) & 1u) ^ 1u, abort_flag, p.err) ||
            !fg_wait(smem_u32(&ctl->full[s]), ph, abort_flag, p.err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (fg_elect()) {
          const uint64_t da = da0 + static_cast<uint32_t>(s * (FW_STAGE_BYTES >> 4));
          const uint64_t db = db0 + static_cast<uint32_t>(s * (FW_STAGE_BYTES >> 4));
#pragma unroll
          for (uint32_t kk = 0; kk < FG_BK / 32; ++kk)   // 32 bytes on, in 16-byte units
            fg_mma(tmem + buf * NT, da + 2 * kk, db + 2 * kk, fg_idesc(128, NT), kk != 0);
          tc_commit(smem_u32(&ctl->tfull[buf]));
          tc_commit(smem_u32(&ctl->empty[s]));
        }
        __syncwarp();
        if (++s == FW_STAGES) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    if (!ok && lane == 0) {   // gave up: wait (bounded) for the MMAs in flight
      tc_commit(smem_u32(&ctl->drain));
      const long long t0 = clock64();
      while (!mbar_try_wait(smem_u32(&ctl->drain), 0) && clock64() - t0 < FG_WAIT_BUDGET / 4) {
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    // ---------------------------------------------------------------- scale loader
    uint32_t ci = 0;   // chunks loaded
    int g = 0;
    bool ok = true;
    for (int tile = unit; tile < total && ok; tile += num_units) {
      int row0, wt;
      map_tile(tile, g, row0, wt);
      const int nt = min(ctl->gstart[g + 1] - row0, NT);
      const float* sb = p.sb + (static_cast<long long>(g) * p.nb + wt) * p.kb + kb_lo;
      const float* sa = p.sa + static_cast<long long>(row0) * p.kb + kb_lo;
      for (int k0 = 0; k0 < nkb; k0 += FW_CHUNK, ++ci) {
        const uint32_t c = ci % FW_CHUNKS;
        if (!fg_wait(smem_u32(&ctl->sempty[c]), ((ci / FW_CHUNKS) & 1u) ^ 1u, abort_flag, p.err)) {
          ok = false;
          break;
        }
        const int j = lane & (FW_CHUNK - 1);
        const bool in = k0 + j < nkb;
#pragma unroll
        for (int t = lane >> 2; t < NT; t += 8)   // rows past the segment's get 0
          cp_async4(&ctl->sa[c][j][t], sa + static_cast<long long>(t) * p.kb + k0 + j,
                    in && t < nt);
        if (lane < FW_CHUNK) cp_async4(&ctl->sb[c][j], sb + k0 + j, in);
        cp_async_arrive(smem_u32(&ctl->sfull[c]));
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- epilogue (4 warps)
    const int q = warp & 3;
    const int row = 32 * q + lane;           // of the tile's 128 weight rows
    const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    const int own = NT / split;              // columns that a CTA of the cluster owns
    uint32_t it = 0, ci = 0, round = 0;
    int g = 0;
    bool ok = true;
    for (int tile = unit; tile < total && ok; tile += num_units, ++round) {
      int row0, wt;
      map_tile(tile, g, row0, wt);
      const int nt = min(ctl->gstart[g + 1] - row0, NT);
      const int n = wt * 128 + row;
      float2 acc[NT / 2];
#pragma unroll
      for (int i = 0; i < NT / 2; ++i) acc[i] = make_float2(0.0f, 0.0f);
      for (int left = nkb; left > 0 && ok; left -= FW_CHUNK, ++ci) {
        const uint32_t c = ci % FW_CHUNKS;
        if (!fg_wait(smem_u32(&ctl->sfull[c]), (ci / FW_CHUNKS) & 1u, abort_flag, p.err)) {
          ok = false;
          break;
        }
        const int m = min(left, FW_CHUNK);
        for (int j = 0; j < m; ++j, ++it) {
          const uint32_t buf = it % FW_BUFS;
          if (!fg_wait(smem_u32(&ctl->tfull[buf]), (it / FW_BUFS) & 1u, abort_flag, p.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          uint32_t d[NT];
          tmem_ld16(taddr + buf * NT, d);
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&ctl->tempty[buf]));
          const float sb = ctl->sb[c][j];
          const float2 sb2 = make_float2(sb, sb);
          const float4* sa = reinterpret_cast<const float4*>(ctl->sa[c][j]);
#pragma unroll
          for (int i = 0; i < NT / 4; ++i) {
            const float4 f = sa[i];
            const float2 lo = make_float2(__uint_as_float(d[4 * i]), __uint_as_float(d[4 * i + 1]));
            const float2 hi =
                make_float2(__uint_as_float(d[4 * i + 2]), __uint_as_float(d[4 * i + 3]));
            acc[2 * i] = __ffma2_rn(lo, __fmul2_rn(make_float2(f.x, f.y), sb2), acc[2 * i]);
            acc[2 * i + 1] =
                __ffma2_rn(hi, __fmul2_rn(make_float2(f.z, f.w), sb2), acc[2 * i + 1]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl->sempty[c]));   // the scales are used up
      }
      if (!ok) break;
      if (split == 1) {
        if (n < p.N) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
            if (t < nt)
              store1<F32>(p.out, static_cast<long long>(row0 + t) * p.ldo + n,
                          (t & 1) ? acc[t / 2].y : acc[t / 2].x);
        }
        continue;
      }
      // every owner has added up the last tile's parts
      if (!fw_wait_cluster(smem_u32(&ctl->pempty), (round & 1u) ^ 1u, abort_flag, p.err)) break;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int owner = t / own;
        st_cluster(mapa_shared(smem_u32(part + (rank * own + (t - owner * own)) * 128 + row),
                               static_cast<uint32_t>(owner)),
                   (t & 1) ? acc[t / 2].y : acc[t / 2].x);
      }
      __syncwarp();
      if (lane < split)
        arrive_cluster(mapa_shared(smem_u32(&ctl->pfull), static_cast<uint32_t>(lane)));
      if (!fw_wait_cluster(smem_u32(&ctl->pfull), round & 1u, abort_flag, p.err)) break;
      for (int i = 0; i < own; ++i) {
        float v = 0.0f;
        for (int r = 0; r < split; ++r) v += part[(r * own + i) * 128 + row];
        const int t = rank * own + i;
        if (t < nt && n < p.N)
          store1<F32>(p.out, static_cast<long long>(row0 + t) * p.ldo + n, v);
      }
      __syncwarp();
      if (lane < split)
        arrive_cluster(mapa_shared(smem_u32(&ctl->pempty), static_cast<uint32_t>(lane)));
    }
  }
  tc_fence_before();
  if (split > 1) cluster_sync_all();   // nobody leaves while the others may write to it
  else __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, FW_TMEM_COLS);
}

template <bool F32>
cudaError_t fw_launch(const CUtensorMap& tw, const CUtensorMap& tt, const FwParams& p, int units,
                      cudaStream_t st) {
  auto kern = fp8_few_kernel<F32>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(FW_SMEM));
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(static_cast<unsigned>(units * p.split)), dim3(FW_THREADS), FW_SMEM,
                    st, static_cast<unsigned>(p.split), tw, tt, p);
}

}  // namespace

// Up to 16 rows in all; up to 64, or 2 to the average segment, if there are no more than 8 to it.
// One row to each of eight experts of 4096 x 7168 takes 47 us here and 57 us in fp8_gemm's kernel;
// 4 rows to each of 128 experts of 1536 x 2048 85 us here and 91 us there, to each of 256 of 512 x
// 1024 40 and 46 us, 8 rows to each of 8 of 2048 x 4096 23 and 31 us.  With 16 rows to each the two
// are even, and with 64, four tiles, 181 us here and 95 us there.  The host does not see the
// segments: where one of 128 has half of 1024 rows, 76 us here and 73 us there, and all 2048 rows
// in one of 256 of 4096 x 7168 389 and 61 us, hence the lower bound for many rows.
bool fp8_few_rows(const Fp8GemmArgs& a) {
  const int64_t G = a.G;
  return !a.wgrad &&
         (a.rows <= 16 || (a.rows <= 8 * G && a.rows <= (2 * G > 64 ? 2 * G : 64)));
}

cudaError_t launch_fp8_few(const Fp8GemmArgs& a, cudaStream_t st) {
  FwParams p{};
  p.G = a.G;
  p.N = a.N;
  p.rows = static_cast<int>(a.rows);
  p.kb = (a.K + 127) / 128;
  p.nb = (a.N + 127) / 128;
  p.w_tiles = p.nb;
  p.offsets = a.offsets;
  p.sa = a.a_scales;
  p.sb = a.b_scales;
  p.out = a.out;
  p.ldo = a.ldo;
  p.err = a.err;
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  // Clusters while all the tiles (one token tile to every segment that can have rows) still run at
  // once and 12 blocks are left to a CTA: one row by 4096 x 7168 takes 25.2 us alone, 21.1 by 2,
  // 19.1 by 4 and, in two rounds, 29.3 us by 8; with 8 blocks, 4096 x 1024, 13 us alone, 15 by 2.
  const int64_t tiles = (a.rows < a.G ? a.rows : a.G) * p.w_tiles;
  p.split = 1;
  while (p.split < 8 && tiles * 2 * p.split <= sms && p.kb >= 24 * p.split) p.split *= 2;
  // no more units than there can be tiles: a segment has at most one that is not full
  const int64_t most = (a.rows < a.G ? a.rows : a.G) + a.rows / NT;
  const int64_t units = most * p.w_tiles;
  const int fit = sms / p.split;
  CUtensorMap tw, tt;
  if (!fp8_codes_map(&tw, a.b, static_cast<uint64_t>(a.K), static_cast<uint64_t>(a.ldb),
                     static_cast<uint64_t>(a.G) * static_cast<uint64_t>(a.N), 128) ||
      !fp8_codes_map(&tt, a.a, static_cast<uint64_t>(a.K), static_cast<uint64_t>(a.lda),
                     static_cast<uint64_t>(a.rows), NT))
    return cudaErrorInvalidValue;
  const int n = units < fit ? static_cast<int>(units) : fit;
  return a.out_fp32 ? fw_launch<true>(tw, tt, p, n, st) : fw_launch<false>(tw, tt, p, n, st);
}

}  // namespace moe
