// fp8_tiles.cuh -- what the block-scaled products (fp8_gemm.cu, fp8_few.cu) share: bounded waits of
// a warp, the E4M3 tensor-core instruction, TMEM loads, and asynchronous 4-byte copies.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace moe {

constexpr int FG_BK = 128;                // elements (bytes) of a block
constexpr int FG_MAX_G = 256;
constexpr long long FG_WAIT_BUDGET = 4000000000LL;

// A whole warp's wait.
__device__ __forceinline__ bool fg_wait(uint32_t bar, uint32_t parity, volatile int* abort,
                                        int* err) {
  if (__all_sync(FULL_MASK, mbar_try_wait(bar, parity))) return true;
  return __all_sync(FULL_MASK, mbar_wait_bounded(bar, parity, abort, err, FG_WAIT_BUDGET));
}
// After giving up: waits, again with a limit, until the copies issued into a ring of N stages have
// landed, so that none arrives in the shared memory of a CTA that has left.  `s`, `ph`: the stage that
// would have been filled next and its parity; the stages before it were filled last with that parity,
// the others with the opposite one (or never: such a wait returns at once).
template <int N>
__device__ __forceinline__ void fg_drain_copies(const uint64_t* full, int s, uint32_t ph) {
  const long long t0 = clock64();
#pragma unroll 1
  for (int j = 0; j < N; ++j)
    while (!mbar_try_wait(smem_u32(full + j), j < s ? ph : ph ^ 1u) &&
           clock64() - t0 < FG_WAIT_BUDGET / 4) {
    }
}
// One thread of the warp, in a form that leaves the code around it warp-uniform: the operands of
// tcgen05.mma and of the TMA copies are uniform registers, and in a branch on the lane's number
// each of them was moved there first, about 100 cycles per MMA.
__device__ __forceinline__ bool fg_elect() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}
// a value that is the same in every lane, as a uniform one
__device__ __forceinline__ int fg_uniform(int v) { return __reduce_max_sync(FULL_MASK, v); }

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
__device__ __forceinline__ void fg_mma_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 32 lanes x 64 consecutive fp32 columns
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
      "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
        "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
        "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
        "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]),
        "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]),
        "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]),
        "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]),
        "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// 4 bytes global -> shared, asynchronously; zero where !ok (nothing is read)
__device__ __forceinline__ void cp_async4(float* dst, const float* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(ok ? 4 : 0)
               : "memory");
}
// one arrival on `bar` when this thread's copies so far have landed
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(bar) : "memory");
}

}  // namespace moe
