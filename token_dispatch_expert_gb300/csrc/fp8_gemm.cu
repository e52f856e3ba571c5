// fp8_gemm.cu -- products of E4M3 operands with one scale for each block of 128: a grouped
// product over the rows of each expert, and its weight gradient over each expert's tokens.
//
//   product       out[p][n]   = sum_kb sa[p][kb] sb[g][n/128][kb] sum_{k in kb} a[p][k] b[g][n][k]
//   weight grad   dW[g][m][n] = sum_kb sa[kb][m] sb[kb][n] sum_{t in kb} a[m][t] b[n][t]
//
// The inner sums are tensor-core products over one block (tcgen05.mma kind::f8f6f4, four of
// K 32), accumulated in fp32 in TMEM; the outer sum runs in fp32 registers of the epilogue
// warps, because a scale is any fp32 number and changes with every block.  So the accumulator
// leaves TMEM once per block: two 256-column accumulators alternate, the MMA fills one while
// eight epilogue warps read the other and add it, scaled, to 128 sums per thread (packed
// fma.rn.f32x2).
//
// Per 128 x 256 tile and block the MMA takes 512 cycles (8192 multiply-adds per cycle and SM);
// the epilogue's 128 columns per warp are 64 packed multiply-adds (128 with per-column scales)
// and 4 TMEM loads, two warps per scheduler.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cstddef>
#include <mutex>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int FG_BK = 128;
constexpr int FG_TILE_M = 128;
constexpr int FG_TILE_N = 256;
// Warps 0 - 3: producer, MMA issuer, two idle; warps 4 - 11: epilogue.  Launched with 168
// registers a thread (64,512 in all); the first four warps hand theirs to the other eight,
// whose 128 sums and 32 loaded columns need more: 128 * 40 + 256 * 232 = 64,512.
constexpr int FG_THREADS = 384;
constexpr int FG_EPI_WARP0 = 4;
constexpr int FG_EPI_WARPS = 8;
constexpr int FG_MAX_G = 256;
constexpr int FG_STAGES = 4;
constexpr int FG_A_BYTES = FG_TILE_M * FG_BK;
constexpr int FG_B_BYTES = FG_TILE_N * FG_BK;
constexpr int FG_STAGE_BYTES = FG_A_BYTES + FG_B_BYTES;
constexpr uint32_t FG_TMEM_COLS = 512;
constexpr long long FG_WAIT_BUDGET = 4000000000LL;

struct FgCtl {
  uint64_t full[FG_STAGES], empty[FG_STAGES], tfull[2], tempty[2], drain;
  uint32_t tmem_base;
  int abort, bad;
  long long gstart[FG_MAX_G + 1];
  int tprefix[FG_MAX_G + 1];    // tiles before each group
  int kbpre[FG_MAX_G + 1];      // wgrad: token blocks before each group
  alignas(16) float bscale[FG_EPI_WARPS][2][128];   // read as float4
};
static_assert(offsetof(FgCtl, bscale) % 16 == 0, "read as float4");
constexpr size_t FG_SMEM = FG_STAGES * FG_STAGE_BYTES + sizeof(FgCtl) + 1024;

struct FgParams {
  int G, N, K;                  // K: of the product; wgrad: M
  long long rows;
  int n_tiles, m_tiles;         // m_tiles: wgrad
  int kb;                       // product: blocks along K; wgrad: token block capacity
  int nb;                       // product: 128-row blocks of b per group
  const int32_t* offsets;
  const float* sa;
  const float* sb;
  void* out;
  long long ldo;
  int* err;
};

__device__ __forceinline__ bool fg_wait(uint32_t bar, uint32_t parity, volatile int* abort,
                                        int* err) {
  return __all_sync(FULL_MASK, mbar_wait_bounded(bar, parity, abort, err, FG_WAIT_BUDGET));
}

// kind::f8f6f4 instruction descriptor: E4M3 x E4M3 -> fp32, both K-major
__host__ __device__ constexpr uint32_t fg_idesc(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ void fg_mma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

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

__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(lo), "r"(hi));
  return v;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ int ceil_div(long long a, int b) {
  return static_cast<int>((a + b - 1) / b);
}

// One row's 128 sums to its place; n0 is the first column, cols the row's width.
template <bool F32>
__device__ __forceinline__ void store_row(void* out, long long off, const uint64_t* acc, int n0,
                                          int cols) {
  if (n0 >= cols) return;
  if (F32) {
    float* dst = static_cast<float*>(out) + off + n0;
    if (n0 + 128 <= cols && (reinterpret_cast<uintptr_t>(dst) & 15u) == 0) {
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float2 a = unpack2(acc[2 * i]), b = unpack2(acc[2 * i + 1]);
        reinterpret_cast<float4*>(dst)[i] = make_float4(a.x, a.y, b.x, b.y);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 64; ++i) {
        const float2 a = unpack2(acc[i]);
        if (n0 + 2 * i < cols) dst[2 * i] = a.x;
        if (n0 + 2 * i + 1 < cols) dst[2 * i + 1] = a.y;
      }
    }
  } else {
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(out) + off + n0;
    if (n0 + 128 <= cols && (reinterpret_cast<uintptr_t>(dst) & 15u) == 0) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 a = unpack2(acc[4 * i + j]);
          w[j] = pack_bf16x2(a.x, a.y);
        }
        reinterpret_cast<uint4*>(dst)[i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 64; ++i) {
        const float2 a = unpack2(acc[i]);
        if (n0 + 2 * i < cols) dst[2 * i] = __float2bfloat16_rn(a.x);
        if (n0 + 2 * i + 1 < cols) dst[2 * i + 1] = __float2bfloat16_rn(a.y);
      }
    }
  }
}

template <bool WG, bool F32>
__global__ void __launch_bounds__(FG_THREADS, 1)
fp8_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                const FgParams p) {
  griddep_wait();   // see common.cuh: dependent launches
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  FgCtl* ctl = reinterpret_cast<FgCtl*>(smem + FG_STAGES * FG_STAGE_BYTES);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t smem_base = smem_u32(smem);
  volatile int* abort_flag = &ctl->abort;

  if (threadIdx.x == 0) {
    for (int s = 0; s < FG_STAGES; ++s) {
      mbar_init(smem_u32(&ctl->full[s]), 1);
      mbar_init(smem_u32(&ctl->empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&ctl->tfull[b]), 1);
      mbar_init(smem_u32(&ctl->tempty[b]), FG_EPI_WARPS);
    }
    mbar_init(smem_u32(&ctl->drain), 1);
    fence_mbar_init();
    ctl->abort = 0;
    ctl->bad = 0;
  }
  if (threadIdx.x == 32) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  for (int g = threadIdx.x; g <= p.G; g += FG_THREADS)
    ctl->gstart[g] = p.offsets ? p.offsets[g] : (g ? p.rows : 0LL);
  __syncthreads();
  if (warp == 0) {
    auto blocks_of = [&](long long a, long long b) { return b > a ? ceil_div(b - a, 128) : 0; };
    const int per = (p.G + 31) / 32;
    int local = 0, local_kb = 0, bad = 0;
    for (int i = 0; i < per; ++i) {
      const int g = lane * per + i;
      if (g < p.G) {
        const long long a = ctl->gstart[g], b = ctl->gstart[g + 1];
        if (b < a || a < 0 || b > p.rows) bad = 1;
        const int n = blocks_of(a, b);
        local += WG ? p.m_tiles * p.n_tiles : n * p.n_tiles;
        local_kb += n;
      }
    }
    const int incl = warp_incl_scan(local), incl_kb = warp_incl_scan(local_kb);
    int run = incl - local, run_kb = incl_kb - local_kb;
    for (int i = 0; i < per; ++i) {
      const int g = lane * per + i;
      if (g < p.G) {
        const int n = blocks_of(ctl->gstart[g], ctl->gstart[g + 1]);
        ctl->tprefix[g] = run;
        ctl->kbpre[g] = run_kb;
        run += WG ? p.m_tiles * p.n_tiles : n * p.n_tiles;
        run_kb += n;
      }
    }
    if (lane == 31) {
      ctl->tprefix[p.G] = incl;
      ctl->kbpre[p.G] = incl_kb;
    }
    if (ctl->gstart[0] != 0) bad = 1;
    bad = __any_sync(FULL_MASK, bad);
    if (lane == 0 && bad) {
      ctl->bad = 1;
      if (blockIdx.x == 0) flag_error(p.err, MOE_DEVERR_BAD_OFFSETS);
    }
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&ctl->tmem_base), FG_TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const int total = ctl->bad ? 0 : ctl->tprefix[p.G];
  const uint32_t tmem_base = ctl->tmem_base;

  // tile -> group, row tile, column tile; row tiles run fastest, so the CTAs at work share the
  // group's weight rows in L2
  auto map_tile = [&](int tile, int& g, int& mt, int& nt) {
    int lo = 0, hi = p.G;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (ctl->tprefix[mid] <= tile) lo = mid;
      else hi = mid;
    }
    g = lo;
    const int local = tile - ctl->tprefix[g];
    const int mtg = WG ? p.m_tiles : ceil_div(ctl->gstart[g + 1] - ctl->gstart[g], FG_TILE_M);
    nt = local / mtg;
    mt = local - nt * mtg;
  };
  auto blocks = [&](int g) { return WG ? ctl->kbpre[g + 1] - ctl->kbpre[g] : p.kb; };

  if (warp < FG_EPI_WARP0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;" ::: "memory");
    if (warp == 0) {
      // ---------------------------------------------------------------- producer
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
        int g, mt, nt;
        map_tile(tile, g, mt, nt);
        const int nkb = blocks(g);
        const int x0 = WG ? ctl->kbpre[g] * FG_BK : 0;
        const int arow = WG ? mt * FG_TILE_M : static_cast<int>(ctl->gstart[g]) + mt * FG_TILE_M;
        const int brow = WG ? nt * FG_TILE_N : g * p.N + nt * FG_TILE_N;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!fg_wait(smem_u32(&ctl->empty[s]), ph ^ 1u, abort_flag, p.err)) {
            ok = false;
            break;
          }
          if (lane == 0) {
            const uint32_t sa = smem_base + s * FG_STAGE_BYTES;
            const uint32_t full = smem_u32(&ctl->full[s]);
            mbar_arrive_expect_tx(full, FG_STAGE_BYTES);
            tma_load_2d(sa, &tmA, full, x0 + kb * FG_BK, arow);
            tma_load_2d(sa + FG_A_BYTES, &tmB, full, x0 + kb * FG_BK, brow);
          }
          __syncwarp();
          if (++s == FG_STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      griddep_launch();
      for (int i = 0; i < FG_STAGES && ok; ++i) {   // every copy of this CTA has been consumed
        if (!fg_wait(smem_u32(&ctl->empty[s]), ph ^ 1u, abort_flag, p.err)) break;
        if (++s == FG_STAGES) {
          s = 0;
          ph ^= 1u;
        }
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------------- MMA issuer
      int s = 0;
      uint32_t ph = 0;
      uint32_t it = 0;   // blocks issued: accumulator it & 1
      bool ok = true;
      for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
        int g, mt, nt;
        map_tile(tile, g, mt, nt);
        const int nkb = blocks(g);
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          const uint32_t buf = it & 1u, use = it >> 1;
          if (!fg_wait(smem_u32(&ctl->tempty[buf]), (use & 1u) ^ 1u, abort_flag, p.err) ||
              !fg_wait(smem_u32(&ctl->full[s]), ph, abort_flag, p.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (lane == 0) {
            const uint32_t sa = smem_base + s * FG_STAGE_BYTES;
            const uint32_t sb = sa + FG_A_BYTES;
#pragma unroll
            for (int kk = 0; kk < FG_BK / 32; ++kk)
              fg_mma(tmem_base + buf * FG_TILE_N, make_smem_desc(sa + kk * 32, 16, 1024),
                     make_smem_desc(sb + kk * 32, 16, 1024), fg_idesc(FG_TILE_M, FG_TILE_N),
                     kk != 0 ? 1u : 0u);
            tc_commit(smem_u32(&ctl->empty[s]));
            tc_commit(smem_u32(&ctl->tfull[buf]));
          }
          __syncwarp();
          if (++s == FG_STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      if (!ok && it > 0 && lane == 0) {   // gave up: wait (bounded) for the MMAs in flight
        tc_commit(smem_u32(&ctl->drain));
        const long long t0 = clock64();
        while (!mbar_try_wait(smem_u32(&ctl->drain), 0) && clock64() - t0 < FG_WAIT_BUDGET / 4) {
        }
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 232;" ::: "memory");
    // ---------------------------------------------------------------- epilogue (8 warps)
    const int q = warp & 3;               // the lane quarter this warp may read
    const int hh = (warp - FG_EPI_WARP0) >> 2;       // which 128 of the 256 columns
    const int r_in_tile = q * 32 + lane;
    float* bs = ctl->bscale[warp - FG_EPI_WARP0][0];
    uint32_t it = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
      int g, mt, nt;
      map_tile(tile, g, mt, nt);
      const int nkb = blocks(g);
      const int lrow = mt * FG_TILE_M + r_in_tile;
      const long long row = WG ? lrow : ctl->gstart[g] + lrow;
      const bool valid = WG ? lrow < p.K : row < ctl->gstart[g + 1];
      const int n0 = nt * FG_TILE_N + 128 * hh;
      // a row or a column block past the end takes the scales of the last one; its sums are
      // not stored
      const float* sa;
      const float* sb;
      if (WG) {
        sa = p.sa + static_cast<long long>(ctl->kbpre[g]) * p.K + (valid ? lrow : 0);
        sb = p.sb + static_cast<long long>(ctl->kbpre[g]) * p.N + n0;
      } else {
        sa = p.sa + (valid ? row : 0) * p.kb;
        const int blk = 2 * nt + hh < p.nb ? 2 * nt + hh : p.nb - 1;
        sb = p.sb + (static_cast<long long>(g) * p.nb + blk) * p.kb;
      }
      uint64_t acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = 0ull;
      for (int kb = 0; kb < nkb; ++kb, ++it) {
        const uint32_t buf = it & 1u, use = it >> 1;
        float s;
        if (WG) {
          s = valid ? __ldg(sa + static_cast<long long>(kb) * p.K) : 0.0f;
          float* mine = bs + buf * 128;   // alternates with the accumulator
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = lane + 32 * i;
            mine[c] = n0 + c < p.N ? __ldg(sb + static_cast<long long>(kb) * p.N + c) : 0.0f;
          }
          __syncwarp();
        } else {
          s = __ldg(sa + kb) * __ldg(sb + kb);
        }
        if (!fg_wait(smem_u32(&ctl->tfull[buf]), use & 1u, abort_flag, p.err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t taddr =
            tmem_base + (static_cast<uint32_t>(q * 32) << 16) + buf * FG_TILE_N + 128 * hh;
        const uint64_t s2 = pack2(s, s);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t d[16];
          tmem_ld16(taddr + 16 * c, d);
          tmem_ld_wait();
          if (c == 7) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ctl->tempty[buf]));
          }
          if (WG) {
            const float4* cs = reinterpret_cast<const float4*>(bs + buf * 128 + 16 * c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 f = cs[i];
              acc[8 * c + 2 * i] = fma2(pack2(d[4 * i], d[4 * i + 1]), mul2(pack2(f.x, f.y), s2),
                                        acc[8 * c + 2 * i]);
              acc[8 * c + 2 * i + 1] = fma2(pack2(d[4 * i + 2], d[4 * i + 3]),
                                            mul2(pack2(f.z, f.w), s2), acc[8 * c + 2 * i + 1]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              acc[8 * c + i] = fma2(pack2(d[2 * i], d[2 * i + 1]), s2, acc[8 * c + i]);
          }
        }
      }
      if (ok && valid)
        store_row<F32>(p.out, (WG ? static_cast<long long>(g) * p.K + lrow : row) * p.ldo, acc, n0,
                       p.N);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, FG_TMEM_COLS);
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

// codes [rows][ld] of which `cols` are read (zeros past them), boxes of 128 x box_rows
bool fg_map(CUtensorMap* m, const void* base, uint64_t cols, uint64_t ld, uint64_t rows,
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

template <bool WG, bool F32>
cudaError_t fg_launch(const CUtensorMap& ta, const CUtensorMap& tb, const FgParams& p,
                      cudaStream_t st) {
  auto kern = fp8_gemm_kernel<WG, F32>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(FG_SMEM));
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return launch_pdl(kern, dim3(static_cast<unsigned>(sms)), dim3(FG_THREADS), FG_SMEM, st, 1, ta,
                    tb, p);
}

}  // namespace

cudaError_t launch_fp8_gemm(const Fp8GemmArgs& a, cudaStream_t st) {
  FgParams p{};
  p.G = a.G;
  p.N = a.N;
  p.K = a.K;
  p.rows = a.rows;
  p.n_tiles = (a.N + FG_TILE_N - 1) / FG_TILE_N;
  p.nb = (a.N + 127) / 128;
  p.offsets = a.offsets;
  p.sa = a.a_scales;
  p.sb = a.b_scales;
  p.out = a.out;
  p.ldo = a.ldo;
  p.err = a.err;
  CUtensorMap ta, tb;
  bool ok;
  if (a.wgrad) {
    p.m_tiles = (a.K + FG_TILE_M - 1) / FG_TILE_M;
    p.kb = static_cast<int>(fp8_token_blocks(a.rows, a.G));
    const uint64_t len = 128ull * static_cast<uint64_t>(p.kb);
    ok = fg_map(&ta, a.a, len, len, static_cast<uint64_t>(a.K), FG_TILE_M) &&
         fg_map(&tb, a.b, len, len, static_cast<uint64_t>(a.N), FG_TILE_N);
  } else {
    p.kb = (a.K + 127) / 128;
    ok = fg_map(&ta, a.a, static_cast<uint64_t>(a.K), static_cast<uint64_t>(a.lda),
                static_cast<uint64_t>(a.rows), FG_TILE_M) &&
         fg_map(&tb, a.b, static_cast<uint64_t>(a.K), static_cast<uint64_t>(a.ldb),
                static_cast<uint64_t>(a.G) * static_cast<uint64_t>(a.N), FG_TILE_N);
  }
  if (!ok) return cudaErrorInvalidValue;
  if (a.wgrad)
    return a.out_fp32 ? fg_launch<true, true>(ta, tb, p, st) : fg_launch<true, false>(ta, tb, p, st);
  return a.out_fp32 ? fg_launch<false, true>(ta, tb, p, st) : fg_launch<false, false>(ta, tb, p, st);
}

}  // namespace moe
