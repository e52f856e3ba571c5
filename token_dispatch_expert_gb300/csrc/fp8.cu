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
// By their bytes these kernels belong to memory: a bf16 value is read once (2 bytes) and one byte
// or, with both orientations, two bytes are written.  What they reach, and what holds them up, at
// 6.7 TB/s for a copy:
//   weights 8 x 4096 x 7168 and transposes 6.5 TB/s, 145 us: memory
//   rows in order, 21,240 x 6656           6.6 TB/s, 64 us: memory
//   rows 32,768 x 7168 gathered from 4096  4.7 TB/s, 64 us: every row passes L2 eight times;
//                                          instructions
//   along the tokens alone, 16,382 x 2056  4.4 TB/s, 23 us: as the next
//   both ways, 16,382 x 2056               4.2 TB/s, 33 us: instructions, and barriers between the
//                                          two orientations
//   SwiGLU, rows 65,536 x 768              4.5 TB/s, 57 us: instructions, about 30 a column for an
//                                          exactly rounded h and its code
//   both ways, 16,383 x 1408               3.0 TB/s, 47 us: instructions
//   its backward, rows alone, 16,383 x 1408
//                                          2.8 TB/s, 66 us: instructions
//   its backward, both ways with h         2.5 TB/s, 102 us: instructions, about 100 a column for
//                                          three values and five codes
#include <cuda.h>
#include <cuda_fp8.h>

#include <type_traits>

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

// A block's factor (which = 0) or scale (1), from the bits of its largest magnitude.
__device__ __forceinline__ float block_quotient(uint32_t amax, int pow2, int which) {
  float a = __uint_as_float(amax << 16);
  if (a < AMAX_FLOOR) a = AMAX_FLOOR;
  if (pow2 && a < INFINITY) {
    // 448 = 1.75 * 2^8: the exponent of a less 8, and one more where a's fraction is above
    const uint32_t u = __float_as_uint(a);
    const uint32_t n = (u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1u : 0u);
    return __uint_as_float((which ? n : 254 - n) << 23);
  }
  return __fdiv_rn(which ? a : E4M3_TOP, which ? E4M3_TOP : a);
}

// two 16-bit maxima at once
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// the larger of m's values (magnitudes) and x's magnitudes, for a pair of bf16 values; a NaN wins, as
// the largest of 16-bit patterns (one instruction, where clearing the signs took another)
__device__ __forceinline__ uint32_t max_mag(uint32_t m, uint32_t x) {
  uint32_t d;
  asm("{\n\t.reg .b32 t;\n\t"
      "abs.bf16x2 t, %2;\n\t"
      "max.NaN.bf16x2 %0, %1, t;\n\t}"
      : "=r"(d)
      : "r"(m), "r"(x));
  return d;
}
__device__ __forceinline__ uint32_t max_mag8(const uint4& v) {
  return max_mag(max_mag(max_mag(max_mag(0u, v.x), v.y), v.z), v.w);
}
// four values (two packed words) times r
__device__ __forceinline__ uint32_t codes4(uint32_t a, uint32_t b, float r) {
  const float2 r2 = make_float2(r, r);
  const float2 x = __fmul2_rn(make_float2(bf16_lo(a), bf16_hi(a)), r2);
  const float2 y = __fmul2_rn(make_float2(bf16_lo(b), bf16_hi(b)), r2);
  return e4m3x2(x.x, x.y) | (e4m3x2(y.x, y.y) << 16);
}
__device__ __forceinline__ uint2 codes8(const uint4& v, float r) {
  return make_uint2(codes4(v.x, v.y, r), codes4(v.z, v.w, r));
}

// ------------------------------------------------------------------ SwiGLU values
// h = silu(a) b and its derivatives are rounded to bf16 once from their exact value, so that
// codes and scales do not depend on how a kernel groups the arithmetic.  A value is computed in
// fp32 with a known error bound; where the bound reaches a border between two bf16 numbers (one
// h in about 3000, one da in about 1000) it is computed again in pairs of fp32 numbers, and where
// even those do not settle it (practically never) or its magnitude is out of their range, in
// 64 bits.  64 bits in the first place would cost three times the kernel: the card has two
// 64-bit multiply-adds per SM and cycle.
// Unevaluated sums of two fp32 numbers (about 48 bits).
struct Pair {
  float h, l;
};
__device__ __forceinline__ Pair quick_sum(float a, float b) {   // |a| >= |b|
  const float s = a + b;
  return {s, b - (s - a)};
}
__device__ __forceinline__ Pair exact_sum(float a, float b) {
  const float s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
__device__ __forceinline__ Pair pair_mul(Pair x, Pair y) {
  const float p = x.h * y.h;
  return quick_sum(p, fmaf(x.h, y.h, -p) + fmaf(x.h, y.l, x.l * y.h));
}
// 2^(j/8), each as the nearest fp32 number and the nearest to what it leaves
__constant__ float kRootHi[8] = {1.0f, 0x1.172b84p+0f, 0x1.306fe0p+0f, 0x1.4bfdaep+0f,
                                 0x1.6a09e6p+0f, 0x1.8ace54p+0f, 0x1.ae89fap+0f, 0x1.d5818ep+0f};
__constant__ float kRootLo[8] = {0.0f, -0x1.c15742p-27f, 0x1.4636e2p-25f, -0x1.593abcp-25f,
                                 0x1.9fcef4p-26f, 0x1.15506ep-27f, -0x1.a94b14p-26f,
                                 -0x1.822dbcp-27f};
// t = e^-a and s = 1 / (1 + t) for |a| <= 80, off by less than 2^-31.5 of themselves: with
// -a = n ln2 / 8 + r, e^-a = 2^(n/8) e^r, |r| < 0.0434, and e^r = 1 + r + r^2/2 in pairs plus a
// tail r^3 (1/6 + ...) below 2^-16, for which fp32 is enough.
__device__ __forceinline__ void sigmoid_pair(float a, Pair& t, Pair& s) {
  const float x = -a;
  const float n = rintf(x * 0x1.715476p+3f);        // 8 / ln 2
  const float d = fmaf(-n, 0x1.62e0p-4f, x);        // ln 2 / 8 to 13 bits: exact
  const float rh = fmaf(-n, 0x1.0bfbe8p-18f, d);    // and 24 more
  const float rl = fmaf(-n, 0x1.0bfbe8p-18f, d - rh);
  const float r2 = rh * rh;
  const float tail =
      r2 * rh * fmaf(rh, fmaf(rh, fmaf(rh, 1.0f / 720, 1.0f / 120), 1.0f / 24), 1.0f / 6);
  const Pair s1 = quick_sum(1.0f, rh);
  const Pair s2 = quick_sum(s1.h, 0.5f * r2);
  const float low = (s1.l + s2.l) + (fmaf(0.5f, fmaf(rh, rh, -r2), fmaf(rh, rl, rl)) + tail);
  const int ni = static_cast<int>(n), j = ni & 7;
  const Pair e = pair_mul(quick_sum(s2.h, low), Pair{kRootHi[j], kRootLo[j]});
  const float scale = __uint_as_float(static_cast<uint32_t>(127 + (ni - j) / 8) << 23);
  t = {e.h * scale, e.l * scale};
  const Pair den0 = exact_sum(1.0f, t.h);
  const Pair den = quick_sum(den0.h, den0.l + t.l);
  const float q = 1.0f / den.h;
  s = quick_sum(q, q * (fmaf(-q, den.h, 1.0f) - q * den.l));
}

__device__ __noinline__ float silu_mul_64(float a, float b) {
  const double x = static_cast<double>(a);
  return __double2float_rn(x * (1.0 / (1.0 + exp(-x))) * static_cast<double>(b));
}
__device__ __noinline__ float dsilu_mul_64(float a, float b, float dh) {
  const double x = static_cast<double>(a);
  const double sg = 1.0 / (1.0 + exp(-x));
  return __double2float_rn(static_cast<double>(dh) * static_cast<double>(b) * sg *
                           (1.0 + x * (1.0 / (1.0 + exp(x)))));
}

__device__ __forceinline__ uint32_t bf16_bits(float v) {
  return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}
// v within e of the exact value: its fp32 neighbour(s) there, if both round to one bf16 number
__device__ __forceinline__ bool settled(Pair v, float e, float& out) {
  out = v.h + (v.l - e);
  return bf16_bits(out) == bf16_bits(v.h + (v.l + e));
}
// results far from fp32's smallest and largest numbers
__device__ __forceinline__ bool in_range(float v) {
  return fabsf(v) >= 0x1p-100f && fabsf(v) < 0x1p126f;
}
constexpr float GATE_MAX = 80.0f;   // above it, and for results out of range, 64 bits

__device__ __noinline__ float silu_mul_exact(float a, float b) {
  const float p = a * b;   // exact: two 8-bit significands
  if (p == 0.0f) return p;
  if (fabsf(a) <= GATE_MAX && in_range(p)) {
    Pair t, s;
    sigmoid_pair(a, t, s);
    const float v = p * s.h;
    float out;
    if (in_range(v) &&
        settled(quick_sum(v, fmaf(p, s.h, -v) + p * s.l), fabsf(v) * 0x1p-31f, out))
      return out;
  }
  return silu_mul_64(a, b);
}
__device__ __noinline__ float dsilu_mul_exact(float a, float b, float dh) {
  const float p = dh * b;
  if (fabsf(a) <= GATE_MAX && (p == 0.0f || in_range(p))) {
    if (p == 0.0f) return p;
    Pair t, s;
    sigmoid_pair(a, t, s);
    Pair u = pair_mul(t, s);                   // 1 - sigma
    u = {a * u.h, fmaf(a, u.h, -(a * u.h)) + a * u.l};
    Pair g = exact_sum(1.0f, u.h);
    g = quick_sum(g.h, g.l + u.l);
    const Pair m = pair_mul(s, g);
    const float v = p * m.h;
    float out;
    if (in_range(v) && settled(quick_sum(v, fmaf(p, m.h, -v) + p * m.l),
                               fabsf(p * s.h) * (fabsf(u.h) + fabsf(g.h)) * 0x1p-30f, out))
      return out;
  }
  return dsilu_mul_64(a, b, dh);
}

// The fp32 values, two at a time.  Whether any of them has to be computed again is asked once for
// all, in few instructions (these kernels are bound by the instructions they issue): values are
// settled if
//   their low 16 bits are more than 10 from 0x8000, that is, they lie more than 10 fp32 steps from
//   every border between bf16 numbers;
//   their magnitudes are between 2^-100 and the largest number (a 0 is computed again too, which
//   returns at once); and the gates are within +-80.
__device__ __forceinline__ float2 wide2(uint32_t w) { return make_float2(bf16_lo(w), bf16_hi(w)); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
constexpr uint32_t SETTLE_STEPS = 10;
// distance from the border plus SETTLE_STEPS, modulo 2^16, in the upper half
__device__ __forceinline__ uint32_t border_place(float v) {
  return __float_as_uint(v) * 0x10000u + ((0x8000u + SETTLE_STEPS) << 16);
}
constexpr uint32_t BORDER_END = (2 * SETTLE_STEPS + 1) << 16;
__device__ __forceinline__ bool unsettled(float v, float gate) {
  return border_place(v) < BORDER_END || !(fabsf(v) >= 0x1p-100f && fabsf(v) < INFINITY) ||
         !(fabsf(gate) <= GATE_MAX);
}
__device__ __forceinline__ float least(float a, float b) { return fminf(fabsf(a), fabsf(b)); }
__device__ __forceinline__ float most(float a, float b) { return fmaxf(fabsf(a), fabsf(b)); }

__device__ __forceinline__ float ex2(float x) {   // off by at most two ulp
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// 1 / d for d >= 1, off by at most one ulp (0 from 2^126 on)
__device__ __forceinline__ float fast_rcp(float d) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  return r;
}
// t = e^-a: 2^y with y = -a / ln 2 rounded, times 1 + c, c = -a - y ln 2 (ln 2 in two parts).  Off
// by ex2's two ulp (2^-22) and one rounding: 1.25 * 2^-22.
__device__ __forceinline__ float2 exp_neg2(float2 a) {
  const float2 na = __fmul2_rn(a, both(-1.0f));
  const float2 y = __fmul2_rn(na, both(0x1.715476p+0f));
  float2 c = __ffma2_rn(y, both(-0x1.62e430p-1f), na);
  c = __ffma2_rn(y, both(0x1.05c610p-29f), c);
  const float2 t = make_float2(ex2(y.x), ex2(y.y));
  return __ffma2_rn(t, c, t);
}

// silu(a) b = a b s, s = 1 / (1 + t): a b is exact; t 1.25 * 2^-22, the sum 2^-24, the reciprocal
// 2^-23, the product 2^-24: below 2.25 * 2^-22, 9 fp32 steps.
__device__ __forceinline__ uint32_t silu_mul2(uint32_t a, uint32_t b) {
  const float2 fa = wide2(a), fb = wide2(b);
  const float2 den = __fadd2_rn(exp_neg2(fa), both(1.0f));
  float2 h = __fmul2_rn(__fmul2_rn(fa, fb), make_float2(fast_rcp(den.x), fast_rcp(den.y)));
  const float far = most(h.x, h.y);
  if (min(border_place(h.x), border_place(h.y)) < BORDER_END || !(least(h.x, h.y) >= 0x1p-100f) ||
      !(far < INFINITY) || !(most(fa.x, fa.y) <= GATE_MAX)) {
    if (unsettled(h.x, fa.x)) h.x = silu_mul_exact(fa.x, fb.x);
    if (unsettled(h.y, fa.y)) h.y = silu_mul_exact(fa.y, fb.y);
  }
  return pack_bf16x2(h.x, h.y);
}
__device__ __forceinline__ uint4 silu_mul8(const uint4& a, const uint4& b) {
  return make_uint4(silu_mul2(a.x, b.x), silu_mul2(a.y, b.y), silu_mul2(a.z, b.z),
                    silu_mul2(a.w, b.w));
}

// All three of a pair of columns from one exponential: h = a b s, db = dh a s, da = dh b s g with
// u = a t s = a (1 - s), g = 1 + u.  h and db as above.  da: |dh b s| (|u| + |g|) 4 * 2^-22 (t
// 1.25 * 2^-22; s 2 * 2^-22; two roundings of u, one of g and two of the products 2^-24 each),
// which near the zero of silu' is many steps of da: both ends of that bound are rounded instead.
struct Swiglu2 {
  uint32_t da, db, h;
};
// One of a pair of da: its two ends' bf16 if they agree and can be trusted, else computed again.
__device__ __forceinline__ float dsilu_mul_settled(uint32_t lo, uint32_t hi, int shift, float w,
                                                   float a, float b, float dh) {
  if (((lo ^ hi) >> shift & 0xffffu) || !(w >= 0x1p-100f && w < INFINITY) ||
      !(fabsf(a) <= GATE_MAX))
    return dsilu_mul_exact(a, b, dh);
  return __uint_as_float((lo >> shift) << 16);
}
__device__ __forceinline__ Swiglu2 swiglu_bwd2(uint32_t a, uint32_t b, uint32_t dh) {
  const float2 fa = wide2(a), fb = wide2(b), fd = wide2(dh);
  const float2 t = exp_neg2(fa);
  const float2 den = __fadd2_rn(t, both(1.0f));
  const float2 s = make_float2(fast_rcp(den.x), fast_rcp(den.y));
  const float2 u = __fmul2_rn(__fmul2_rn(fa, t), s);
  const float2 g = __fadd2_rn(u, both(1.0f));
  float2 h = __fmul2_rn(__fmul2_rn(fa, fb), s);
  float2 db = __fmul2_rn(__fmul2_rn(fd, fa), s);
  const float2 qs = __fmul2_rn(__fmul2_rn(fd, fb), s);
  const float2 v = __fmul2_rn(qs, g);
  const float2 w = make_float2((fabsf(u.x) + fabsf(g.x)) * fabsf(qs.x),
                               (fabsf(u.y) + fabsf(g.y)) * fabsf(qs.y));
  const uint32_t lo = pack_bf16x2(fmaf(w.x, -0x1p-20f, v.x), fmaf(w.y, -0x1p-20f, v.y));
  const uint32_t hi = pack_bf16x2(fmaf(w.x, 0x1p-20f, v.x), fmaf(w.y, 0x1p-20f, v.y));
  const uint32_t near = min(min(border_place(h.x), border_place(h.y)),
                            min(border_place(db.x), border_place(db.y)));
  const float close = fminf(fminf(least(h.x, h.y), least(db.x, db.y)), fminf(w.x, w.y));
  const float far = fmaxf(fmaxf(most(h.x, h.y), most(db.x, db.y)), fmaxf(w.x, w.y));
  uint32_t da = lo;
  if (near < BORDER_END || lo != hi || !(close >= 0x1p-100f) || !(far < INFINITY) ||
      !(most(fa.x, fa.y) <= GATE_MAX)) {
    if (unsettled(h.x, fa.x)) h.x = silu_mul_exact(fa.x, fb.x);
    if (unsettled(h.y, fa.y)) h.y = silu_mul_exact(fa.y, fb.y);
    if (unsettled(db.x, fa.x)) db.x = silu_mul_exact(fa.x, fd.x);
    if (unsettled(db.y, fa.y)) db.y = silu_mul_exact(fa.y, fd.y);
    da = pack_bf16x2(dsilu_mul_settled(lo, hi, 0, w.x, fa.x, fb.x, fd.x),
                     dsilu_mul_settled(lo, hi, 16, w.y, fa.y, fb.y, fd.y));
  }
  return {da, pack_bf16x2(db.x, db.y), pack_bf16x2(h.x, h.y)};
}

// da alone (db alone is silu_mul2(a, dh))
__device__ __forceinline__ uint32_t dsilu_mul2(uint32_t a, uint32_t b, uint32_t dh) {
  const float2 fa = wide2(a), fb = wide2(b), fd = wide2(dh);
  const float2 t = exp_neg2(fa);
  const float2 den = __fadd2_rn(t, both(1.0f));
  const float2 s = make_float2(fast_rcp(den.x), fast_rcp(den.y));
  const float2 u = __fmul2_rn(__fmul2_rn(fa, t), s);
  const float2 g = __fadd2_rn(u, both(1.0f));
  const float2 qs = __fmul2_rn(__fmul2_rn(fd, fb), s);
  const float2 v = __fmul2_rn(qs, g);
  const float2 w = make_float2((fabsf(u.x) + fabsf(g.x)) * fabsf(qs.x),
                               (fabsf(u.y) + fabsf(g.y)) * fabsf(qs.y));
  const uint32_t lo = pack_bf16x2(fmaf(w.x, -0x1p-20f, v.x), fmaf(w.y, -0x1p-20f, v.y));
  const uint32_t hi = pack_bf16x2(fmaf(w.x, 0x1p-20f, v.x), fmaf(w.y, 0x1p-20f, v.y));
  if (lo == hi && fminf(w.x, w.y) >= 0x1p-100f && fmaxf(w.x, w.y) < INFINITY &&
      most(fa.x, fa.y) <= GATE_MAX)
    return lo;
  return pack_bf16x2(dsilu_mul_settled(lo, hi, 0, w.x, fa.x, fb.x, fd.x),
                     dsilu_mul_settled(lo, hi, 16, w.y, fa.y, fb.y, fd.y));
}
__device__ __forceinline__ uint4 dsilu_mul8(const uint4& a, const uint4& b, const uint4& dh) {
  return make_uint4(dsilu_mul2(a.x, b.x, dh.x), dsilu_mul2(a.y, b.y, dh.y),
                    dsilu_mul2(a.z, b.z, dh.z), dsilu_mul2(a.w, b.w, dh.w));
}

// ------------------------------------------------------------------ sources
// What a quantiser reads: eight consecutive values of a row, as packed bf16; columns at or past
// `cols` are 0.  W: what is loaded at once, 8 values (every row starts on 16 bytes and a chunk
// never crosses an end), 2 (on 4 bytes, an even width) or 1.
enum { SRC_ROWS, SRC_SWIGLU, SRC_SWIGLU_BWD };

struct Source {
  const __nv_bfloat16* x;    // rows: [src_rows][ld]; SwiGLU: ab [rows][2f]
  const __nv_bfloat16* dh;   // backward: [rows][f]
  long long ld;
  int f;
  int cols;                  // columns quantised: C, f, or 2f
};

__device__ __forceinline__ uint32_t load1(const __nv_bfloat16* p) {
  return static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(p)));
}
__device__ __forceinline__ uint32_t load2(const __nv_bfloat16* p) {
  return __ldg(reinterpret_cast<const uint32_t*>(p));
}
template <int W>
__device__ __forceinline__ uint4 load8(const __nv_bfloat16* p, int n) {
  if constexpr (W == 8) {
    return __ldg(reinterpret_cast<const uint4*>(p));
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (W == 2) {
        w[i] = 2 * i < n ? load2(p + 2 * i) : 0u;
      } else {
        const uint32_t lo = 2 * i < n ? load1(p + 2 * i) : 0u;
        const uint32_t hi = 2 * i + 1 < n ? load1(p + 2 * i + 1) : 0u;
        w[i] = lo | (hi << 16);
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <int SRC, int W>
__device__ __forceinline__ uint4 value8(const Source& s, long long row, int c) {
  const int n = s.cols - c;
  if (n <= 0) return make_uint4(0u, 0u, 0u, 0u);
  if constexpr (SRC == SRC_ROWS) {
    return load8<W>(s.x + row * s.ld + c, n);
  } else {
    const __nv_bfloat16* ab = s.x + row * 2 * s.f;
    if constexpr (SRC == SRC_SWIGLU)
      return silu_mul8(load8<W>(ab + c, n), load8<W>(ab + s.f + c, n));
    // a chunk of da, of db, or (where the halves meet inside it) of both; widths of whole blocks
    // have code of their own
    const __nv_bfloat16* dh = s.dh + row * s.f;
    if (c + 8 <= s.f)
      return dsilu_mul8(load8<W>(ab + c, 8), load8<W>(ab + s.f + c, 8), load8<W>(dh + c, 8));
    if (c >= s.f) return silu_mul8(load8<W>(ab + c - s.f, n), load8<W>(dh + c - s.f, n));
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c0 = c + 2 * i, c1 = c0 + 1;
      w[i] = 0u;
      if (c0 >= s.cols) continue;   // (cols = 2 f is even)
      const int k0 = c0 < s.f ? c0 : c0 - s.f, k1 = c1 < s.f ? c1 : c1 - s.f;
      const Swiglu2 x = swiglu_bwd2(load1(ab + k0) | (load1(ab + k1) << 16),
                                    load1(ab + s.f + k0) | (load1(ab + s.f + k1) << 16),
                                    load1(dh + k0) | (load1(dh + k1) << 16));
      w[i] = ((c0 < s.f ? x.da : x.db) & 0xffffu) | ((c1 < s.f ? x.da : x.db) & 0xffff0000u);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
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

// 16 bytes global -> shared, asynchronously, of which the first n are read and the rest zeros
__device__ __forceinline__ void cp_async_n(uint32_t dst, const void* src, int n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool ok) {
  cp_async_n(smem_u32(dst), src, ok ? 16 : 0);
}

// a box of 128 bytes x 128 rows, shared -> global (parts past the map's rows are not written)
__device__ __forceinline__ void tma_store_2d(const void* tmap, uint32_t src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(src), "r"(x), "r"(y)
               : "memory");
}

// Four blocks of a row (or of four rows), a chunk of eight values per lane in each, sixteen lanes
// to a block: their scales and factors, by one pass of shuffles (two blocks' maxima to a
// word) and one division, of whose lanes one divides for each block's factor and its neighbour
// for the scale.  `quot` gets this lane's quotient.
__device__ __forceinline__ void four_scales(const uint4* v, int pow2, int lane, float* r,
                                            float& quot) {
  uint32_t m[4];
#pragma unroll
  for (int b = 0; b < 4; ++b) m[b] = max_mag8(v[b]);
  const uint32_t x = max2(__byte_perm(m[0], m[1], 0x5410), __byte_perm(m[0], m[1], 0x7632));
  const uint32_t y = max2(__byte_perm(m[2], m[3], 0x5410), __byte_perm(m[2], m[3], 0x7632));
  // eight lanes go on with blocks 0 and 1, the other eight with 2 and 3
  const bool upper = lane & 8;
  uint32_t w = max2(upper ? y : x, __shfl_xor_sync(FULL_MASK, upper ? x : y, 8));
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) w = max2(w, __shfl_xor_sync(FULL_MASK, w, o));
  quot = block_quotient((lane & 2) ? w >> 16 : w & 0xffffu, pow2, lane & 1);
#pragma unroll
  for (int b = 0; b < 4; ++b)
    r[b] = __shfl_sync(FULL_MASK, quot, (lane & 16) | ((b & 2) << 2) | ((b & 1) << 1));
}
// the block whose scale this lane's quotient is, or -1
__device__ __forceinline__ int scale_of_lane(int lane) {
  return (lane & 5) == 1 ? ((lane >> 2) & 2) | ((lane >> 1) & 1) : -1;
}

// ------------------------------------------------------------------ along the rows
// One warp per row; a lane takes eight values (16 bytes), half a warp a block, four chunks'
// loads before any is used.  W = 128: the backward of a width of whole blocks, where a chunk's
// values of da and db come from one computation.
template <int SRC, int W>
__global__ void __launch_bounds__(FQ_THREADS, 4)
fp8_rows_kernel(const Source src, const int32_t* __restrict__ src_tok, long long src_rows,
                const int32_t* __restrict__ offsets, int G, long long rows, const QuantOut out,
                int* err) {
  griddep_wait();   // see common.cuh: dependent launches
  const int lane = threadIdx.x & 31;
  const long long gw = (static_cast<long long>(blockIdx.x) * FQ_THREADS + threadIdx.x) >> 5;
  const long long nw = (static_cast<long long>(gridDim.x) * FQ_THREADS) >> 5;
  const long long n_rows = live_rows(offsets, G, rows, err, gw == 0 && lane == 0);
  // the next row's source is looked up while this row is quantised
  long long t_next = gw;
  if (src_tok && gw < n_rows) t_next = __ldg(src_tok + gw);
  for (long long p = gw; p < n_rows; p += nw) {
    const long long t = t_next;
    t_next = p + nw;
    if (src_tok) {
      if (p + nw < n_rows) t_next = __ldg(src_tok + p + nw);
      if (t < 0 || t >= src_rows) {
        if (lane == 0) flag_error(err, MOE_DEVERR_BAD_INDEX);
        continue;
      }
    }
    constexpr bool BOTH = SRC == SRC_SWIGLU_BWD && W == 128;   // two chunks of da, two of db
    const int span = BOTH ? src.f : src.cols;
    for (int c0 = 0; c0 < span; c0 += BOTH ? 512 : 1024) {
      uint4 v[4];
      int col[4];
      if constexpr (BOTH) {
        uint4 a[2], b[2], d[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int c = c0 + 256 * i + 8 * lane;
          col[i] = c;
          col[2 + i] = src.f + c;
          a[i] = b[i] = d[i] = make_uint4(0u, 0u, 0u, 0u);
          if (c < src.f) {
            a[i] = load8<8>(src.x + t * 2 * src.f + c, 8);
            b[i] = load8<8>(src.x + t * 2 * src.f + src.f + c, 8);
            d[i] = load8<8>(src.dh + t * src.f + c, 8);
          } else {
            col[i] = col[2 + i] = 1 << 28;   // past every column
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t *pa = &a[i].x, *pb = &b[i].x, *pd = &d[i].x;
          uint32_t x[4], y[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const Swiglu2 w = swiglu_bwd2(pa[k], pb[k], pd[k]);
            x[k] = w.da;
            y[k] = w.db;
          }
          v[i] = make_uint4(x[0], x[1], x[2], x[3]);
          v[2 + i] = make_uint4(y[0], y[1], y[2], y[3]);
        }
      } else if constexpr (SRC == SRC_SWIGLU && W == 8) {   // all loads before the arithmetic
        uint4 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          col[i] = c0 + 256 * i + 8 * lane;
          a[i] = b[i] = make_uint4(0u, 0u, 0u, 0u);
          if (col[i] < src.cols) {
            a[i] = load8<8>(src.x + t * 2 * src.f + col[i], 8);
            b[i] = load8<8>(src.x + t * 2 * src.f + src.f + col[i], 8);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[i] = col[i] < src.cols ? silu_mul8(a[i], b[i]) : a[i];
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          col[i] = c0 + 256 * i + 8 * lane;
          v[i] = value8<SRC, W>(src, t, col[i]);
        }
      }
      float r[4], quot;
      four_scales(v, out.pow2, lane, r, quot);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (col[i] < src.cols)
          __stcs(reinterpret_cast<uint2*>(out.codes + p * out.ld + col[i]), codes8(v[i], r[i]));
      const int sb = scale_of_lane(lane);
      const int c =
          (sb == 1 ? col[1] : sb == 2 ? col[2] : sb == 3 ? col[3] : col[0]) - 8 * (lane & 15);
      if (sb >= 0 && c < src.cols) out.scales[p * out.kb + (c >> 7)] = quot;
    }
  }
  griddep_launch();
}

// Plain rows on 16 bytes: a lane's pieces come through a ring in shared memory that it alone writes
// (cp.async) and reads, so that two spans of 1024 columns are under way while one is worked on,
// with nothing to wait for but the lane's own copies.  (Loaded into registers, as above: 77 us
// instead of 63 for 32,768 gathered rows of 7168, 69 instead of 64 for 21,240 rows of 6656 in
// order.  The SwiGLU, with two inputs to a column and bound by its instructions, is 10% slower
// this way.)  A grid of four waves: the rows are spread evenly.
constexpr int FR_STAGES = 3;
constexpr int FR_CTAS = 4;   // per SM
constexpr int FR_SMEM = FR_STAGES * 4 * FQ_THREADS * 16;

__global__ void __launch_bounds__(FQ_THREADS, FR_CTAS)
fp8_rows_ring_kernel(const Source src, const int32_t* __restrict__ src_tok, long long src_rows,
                     const int32_t* __restrict__ offsets, int G, long long rows,
                     const QuantOut out, int* err) {
  griddep_wait();   // see common.cuh: dependent launches
  extern __shared__ uint4 dyn[];   // [FR_STAGES][4][FQ_THREADS]
  const uint4* mine = dyn + threadIdx.x;
  const uint32_t mine_addr = smem_u32(mine);
  const int lane = threadIdx.x & 31;
  const long long gw = (static_cast<long long>(blockIdx.x) * FQ_THREADS + threadIdx.x) >> 5;
  const long long nw = (static_cast<long long>(gridDim.x) * FQ_THREADS) >> 5;
  const long long n_rows = live_rows(offsets, G, rows, err, gw == 0 && lane == 0);
  // the next fetch: its row, source row and first column, and the source of the row after it
  long long fp = gw, ft = gw, ft_next = gw + nw;
  int fc = 0, f_stage = 0;
  if (src_tok) {
    if (gw < n_rows) ft = __ldg(src_tok + gw);
    if (gw + nw < n_rows) ft_next = __ldg(src_tok + gw + nw);
  }
  auto fetch = [&]() {
    if (fp < n_rows) {
      const bool ok = !src_tok || (ft >= 0 && ft < src_rows);
      const __nv_bfloat16* row = src.x + (ok ? ft : 0) * src.ld + fc + 8 * lane;
      const uint32_t dst = mine_addr + f_stage * (4 * FQ_THREADS * 16);
      if (fc + 1024 <= src.cols) {   // the whole span: constant distances
        const int n = ok ? 16 : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) cp_async_n(dst + i * (FQ_THREADS * 16), row + 256 * i, n);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool in = ok && fc + 256 * i + 8 * lane < src.cols;
          cp_async_n(dst + i * (FQ_THREADS * 16), in ? row + 256 * i : src.x, in ? 16 : 0);
        }
      }
      if (++f_stage == FR_STAGES) f_stage = 0;
      fc += 1024;
      if (fc >= src.cols) {
        fc = 0;
        fp += nw;
        ft = ft_next;
        ft_next = fp + nw;
        if (src_tok && ft_next < n_rows) ft_next = __ldg(src_tok + ft_next);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < FR_STAGES - 1; ++i) fetch();
  int stage = 0;
  for (long long p = gw; p < n_rows; p += nw) {
    bool live = true;   // its source is a row (the ring holds zeros if not)
    if (src_tok) {
      const long long t = __ldg(src_tok + p);
      live = t >= 0 && t < src_rows;
      if (!live && lane == 0) flag_error(err, MOE_DEVERR_BAD_INDEX);
    }
    for (int c0 = 0; c0 < src.cols; c0 += 1024) {
      asm volatile("cp.async.wait_group %0;" ::"n"(FR_STAGES - 2) : "memory");
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = mine[(stage * 4 + i) * FQ_THREADS];
      if (++stage == FR_STAGES) stage = 0;
      float r[4], quot;
      four_scales(v, out.pow2, lane, r, quot);
      fetch();   // to where the span before this one was
      if (!live) continue;
      const int c = c0 + 8 * lane;
      uint8_t* to = out.codes + p * out.ld + c;
      if (c0 + 1024 <= src.cols) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          __stcs(reinterpret_cast<uint2*>(to + 256 * i), codes8(v[i], r[i]));
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c + 256 * i < src.cols)
            __stcs(reinterpret_cast<uint2*>(to + 256 * i), codes8(v[i], r[i]));
      }
      const int sb = scale_of_lane(lane);
      const int cs = c0 + 256 * sb + 8 * (lane & 16);   // its block's first column
      if (sb >= 0 && cs < src.cols) out.scales[p * out.kb + (cs >> 7)] = quot;
    }
  }
  griddep_launch();
}

// The SwiGLU of widths of 8 whose chunks of 256 columns do not come in fours: a warp takes four
// chunks at a time, one after another over the rows' ends, so that no place of four_scales() stays
// empty (65,536 rows of 768 columns 56.4 us, in spans of 1024 columns 61.8; 32,768 rows of 1408 57.4
// and 60.7).  Where they do, fp8_rows_kernel's spans are the same chunks with less arithmetic
// (65,536 rows of 2048 133.4 us, here 140.4; 16,384 rows of 2048 37.9 and 39.0; 4096 rows of 1024
// 7.5 and 8.6; 40,000 rows of 1000 46.3 and 47.4).
__global__ void __launch_bounds__(FQ_THREADS, 4)
fp8_swiglu_rows_kernel(const Source src, const int32_t* __restrict__ offsets, int G,
                       long long rows, const QuantOut out, int* err) {
  griddep_wait();   // see common.cuh: dependent launches
  const int lane = threadIdx.x & 31;
  const long long gw = (static_cast<long long>(blockIdx.x) * FQ_THREADS + threadIdx.x) >> 5;
  const long long nw = (static_cast<long long>(gridDim.x) * FQ_THREADS) >> 5;
  const uint32_t n_rows =
      static_cast<uint32_t>(live_rows(offsets, G, rows, err, gw == 0 && lane == 0));
  const int nch = (src.f + 255) / 256;
  uint32_t row = static_cast<uint32_t>(4 * gw / nch);
  int ch = static_cast<int>(4 * gw - static_cast<long long>(row) * nch);
  // from the end of a warp's four chunks to its next ones
  const uint32_t skip_rows = static_cast<uint32_t>(4 * (nw - 1) / nch);
  const int skip = static_cast<int>(4 * (nw - 1) - static_cast<long long>(skip_rows) * nch);
  while (row < n_rows) {
    uint4 a[4], b[4];
    uint32_t at[4];
    int col[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      at[i] = row;
      // past the last row: past every width by more than a block, so that no code and no scale of
      // it is stored
      col[i] = row < n_rows ? 256 * ch + 8 * lane : 1 << 28;
      a[i] = b[i] = make_uint4(0u, 0u, 0u, 0u);
      if (col[i] < src.f) {
        const __nv_bfloat16* x = src.x + static_cast<long long>(row) * (2 * src.f) + col[i];
        a[i] = __ldcs(reinterpret_cast<const uint4*>(x));
        b[i] = __ldcs(reinterpret_cast<const uint4*>(x + src.f));
      }
      if (++ch == nch) {
        ch = 0;
        ++row;
      }
    }
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = col[i] < src.f ? silu_mul8(a[i], b[i]) : a[i];
    float r[4], quot;
    four_scales(v, out.pow2, lane, r, quot);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (col[i] < src.f)
        __stcs(reinterpret_cast<uint2*>(out.codes + static_cast<long long>(at[i]) * out.ld +
                                        col[i]),
               codes8(v[i], r[i]));
    const int sb = scale_of_lane(lane);
    const uint32_t p = sb == 1 ? at[1] : sb == 2 ? at[2] : sb == 3 ? at[3] : at[0];
    const int c =
        (sb == 1 ? col[1] : sb == 2 ? col[2] : sb == 3 ? col[3] : col[0]) - 8 * (lane & 15);
    if (sb >= 0 && c < src.f) out.scales[static_cast<long long>(p) * out.kb + (c >> 7)] = quot;
    row += skip_rows;
    ch += skip;
    if (ch >= nch) {
      ch -= nch;
      ++row;
    }
  }
  griddep_launch();
}

// ------------------------------------------------------------------ along the tokens (and rows)
// Tiles of 128 columns and one 128-row block of a segment (blocks are counted from the segment's
// first row), column tiles fastest.
struct Blocks {
  int first[FQ_MAX_G + 1];   // first block of every segment
  int start[FQ_MAX_G + 1];   // first row
  int sum[8];
  int bad;
};
struct TileAt {
  int kb, c0, nr, r0;        // block, first column, rows in it, the first of them
};
__device__ __forceinline__ long long segment_start(const int32_t* offsets, int g, long long rows) {
  return offsets ? static_cast<long long>(__ldg(offsets + g)) : (g ? rows : 0LL);
}
// All threads of the CTA (at least 256); false for bad offsets.
__device__ __forceinline__ bool count_blocks(Blocks& s, const int32_t* offsets, int G,
                                             long long rows, int* err) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) s.bad = 0;
  __syncthreads();
  int nb = 0;   // G <= 256: one segment per thread of the first eight warps
  if (tid < G) {
    const long long a = segment_start(offsets, tid, rows);
    const long long b = segment_start(offsets, tid + 1, rows);
    if (a < 0 || b < a || b > rows || (tid == 0 && a != 0)) s.bad = 1;
    else nb = static_cast<int>((b - a + 127) / 128);
    s.start[tid] = static_cast<int>(a);
    if (tid == G - 1) s.start[G] = static_cast<int>(b);
  }
  const int incl = warp_incl_scan(nb);
  if (lane == 31 && warp < 8) s.sum[warp] = incl;
  __syncthreads();
  if (tid < G) {
    int before = 0;
    for (int w = 0; w < warp; ++w) before += s.sum[w];
    s.first[tid] = before + incl - nb;
    if (tid == G - 1) s.first[G] = before + incl;
  }
  __syncthreads();
  if (s.bad && blockIdx.x == 0 && tid == 0) flag_error(err, MOE_DEVERR_BAD_OFFSETS);
  return s.bad == 0;
}
// A CTA's tiles, `step` apart, from number `item`: the column tile, block and segment go on from the
// last tile's (a division and a search for each took a fifth of the instructions of the quantiser
// without SwiGLU).
struct Walk {
  int cx, kb, g;             // column tile, block, segment
  int dc, dk, gx;
  __device__ __forceinline__ Walk(long long item, int step, int gx_) : g(0), gx(gx_) {
    kb = static_cast<int>(item / gx);
    cx = static_cast<int>(item - static_cast<long long>(kb) * gx);
    dk = step / gx;
    dc = step - dk * gx;
  }
  __device__ __forceinline__ void next() {
    kb += dk;
    cx += dc;
    if (cx >= gx) {
      cx -= gx;
      ++kb;
    }
  }
  // (kb below the number of blocks)
  __device__ __forceinline__ TileAt at(const Blocks& s) {
    while (s.first[g + 1] <= kb) ++g;
    TileAt t;
    t.kb = kb;
    t.c0 = cx * 128;
    t.r0 = s.start[g] + 128 * (kb - s.first[g]);
    t.nr = min(s.start[g + 1] - t.r0, 128);
    return t;
  }
};

constexpr int FT_TILE = 128 * 16;   // 16-byte pieces

constexpr int FT_THREADS = 512;

// A tile's columns (c0 ..) along the tokens into block kb, by FT_THREADS threads of which this is
// number `th`: two columns and 16 rows (one 16-byte piece of codes) each.  Joined by a barrier of the
// whole CTA.  The codes go to their places, or to `box`: 128 columns of 128 bytes, 16-byte pieces
// XOR-swizzled by the column, for a TMA store (a column's 128 codes are one line in memory, and 16
// bytes of 32 lines at a time halved the stores' rate).
struct Columns {
  static constexpr int Q = FT_THREADS / 64;
  static_assert(128 / Q == 16, "a thread's codes are one 16-byte piece");
  uint32_t w[128 / Q];
  uint32_t m;
  __device__ __forceinline__ void read(const uint4* tile, int th, uint32_t (*s_max)[64]) {
    const int cp = th & 63, q = th >> 6;
    const uint32_t* words = reinterpret_cast<const uint32_t*>(tile);
    m = 0u;
#pragma unroll
    for (int i = 0; i < 128 / Q; ++i) {
      w[i] = words[(128 / Q * q + i) * 64 + cp];
      m = max_mag(m, w[i]);
    }
    s_max[q][cp] = m;
  }
  // columns from c0 of a part of `width` columns that begins at `first` of all `cols`
  __device__ __forceinline__ void write(int th, uint32_t (*s_max)[64], int c0, int first,
                                        int width, int cols, int kb, const QuantOut& o,
                                        uint8_t* box) {
    const int cp = th & 63, q = th >> 6;
#pragma unroll
    for (int i = 0; i < Q; ++i) m = max2(m, s_max[i][cp]);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (c0 + 2 * cp + j >= width) continue;
      const int c = first + c0 + 2 * cp + j;
      const uint32_t amax = j ? m >> 16 : m & 0xffffu;
      const float r = block_quotient(amax, o.pow2, 0);
      uint32_t code[32 / Q];
#pragma unroll
      for (int i = 0; i < 32 / Q; ++i) {
        auto at = [&](int k) { return j ? bf16_hi(w[4 * i + k]) : bf16_lo(w[4 * i + k]); };
        const float2 x = __fmul2_rn(make_float2(at(0), at(1)), both(r));
        const float2 y = __fmul2_rn(make_float2(at(2), at(3)), both(r));
        code[i] = e4m3x2(x.x, x.y) | (e4m3x2(y.x, y.y) << 16);
      }
      constexpr int N = 128 / Q;   // codes
      const int at = N * q, cc = 2 * cp + j;
      uint8_t* dst = box ? box + cc * 128 + ((at & 112) ^ ((cc & 7) << 4)) + (at & 15)
                         : o.codes_t + (static_cast<long long>(c) * o.kb_cap + kb) * 128 + at;
      *reinterpret_cast<uint4*>(dst) = make_uint4(code[0], code[1], code[2], code[3]);
      if (q == 0)
        o.scales_t[static_cast<long long>(kb) * cols + c] = block_quotient(amax, o.pow2, 1);
    }
  }
};

// Four blocks along the row: row and column of each from at(i) (a half-warp each).
template <typename At>
__device__ __forceinline__ void tile_rows(const uint4* v, const TileAt& t, int cols,
                                          const QuantOut& out, At at) {
  const int lane = threadIdx.x & 31;
  float f[4], quot;
  four_scales(v, out.pow2, lane, f, quot);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int2 rc = at(i);
    if (rc.x < t.nr && rc.y < cols)
      *reinterpret_cast<uint2*>(out.codes + (t.r0 + rc.x) * out.ld + rc.y) = codes8(v[i], f[i]);
  }
  const int sb = scale_of_lane(lane);
  if (sb >= 0) {
    const int2 rc = at(sb);
    const int c = rc.y - 8 * (lane & 15);
    if (rc.x < t.nr && c < cols)
      out.scales[static_cast<long long>(t.r0 + rc.x) * out.kb + (c >> 7)] = quot;
  }
}

// Rows read by one or two elements: any width and alignment.
template <int SRC, int W>
__global__ void __launch_bounds__(FT_THREADS, 2)
fp8_tokens_any_kernel(const Source src, const int32_t* __restrict__ src_tok, long long src_rows,
                      const int32_t* __restrict__ offsets, int G, long long rows,
                      const QuantOut out, int* err) {
  griddep_wait();   // see common.cuh: dependent launches
  __shared__ uint4 tile[FT_TILE];
  __shared__ uint32_t s_max[8][64];
  __shared__ Blocks blocks;
  if (!count_blocks(blocks, offsets, G, rows, err)) return;
  const int tid = threadIdx.x;
  const int gx = (src.cols + 127) / 128;
  const long long total = static_cast<long long>(blocks.first[G]) * gx;
  Walk walk(blockIdx.x, gridDim.x, gx);
  for (long long item = blockIdx.x; item < total; item += gridDim.x, walk.next()) {
    const TileAt t = walk.at(blocks);
    const int r = tid >> 4, c = t.c0 + 8 * (tid & 15);
    uint4 v[4];
    uint32_t bad = 0u;   // bit u: the row's source is none (read as row 0, and no row codes)
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      v[u] = make_uint4(0u, 0u, 0u, 0u);
      if (r + 32 * u < t.nr) {
        int row = t.r0 + r + 32 * u;
        if (src_tok) {
          row = __ldg(src_tok + row);
          if (row < 0 || row >= src_rows) {
            flag_error(err, MOE_DEVERR_BAD_INDEX);
            row = 0;
            bad |= 1u << u;
          }
        }
        v[u] = value8<SRC, W>(src, row, c);
      }
    }
    __syncthreads();   // the previous tile is consumed
#pragma unroll
    for (int u = 0; u < 4; ++u) tile[(r + 32 * u) * 16 + (tid & 15)] = v[u];
    if (out.codes)
      tile_rows(v, t, src.cols, out, [&](int u) {
        return make_int2((bad >> u) & 1u ? 128 : r + 32 * u, c);
      });
    __syncthreads();
    Columns cols;
    cols.read(tile, tid, s_max);
    __syncthreads();
    cols.write(tid, s_max, t.c0, 0, src.cols, src.cols, t.kb, out, nullptr);
  }
  griddep_launch();
}

// Rows on 16 bytes.  A piece of a tile is fetched (cp.async), read and turned into its result by
// one thread.  Rows: the next tile is on its way into the other of two buffers while this one's
// columns are worked on.  SwiGLU: a and b, read by their own threads alone, make room for the next
// tile's as soon as h stands in a buffer of its own.  Backward: da, db and h overwrite a, b and
// dh.  A tile's column codes overwrite the tile once it is in registers.  So one CTA takes 64,
// 96 or 96 KB, and three or two CTAs to an SM work while another waits (the backward in one CTA of
// 1024 threads with the next tile under way took 118 us at 16383 x 1408).
template <int SRC>
struct TileGeo {
  static constexpr int PER = FT_TILE / FT_THREADS;      // pieces of a tile per thread
  static constexpr int CTAS = SRC == SRC_ROWS ? 3 : 2;  // per SM
  static constexpr int BUFS = SRC == SRC_ROWS ? 2 : 3;
  static constexpr int SMEM = BUFS * FT_TILE * 16 + 1024;
};

// tm, tm_b, tm_h: codes_t of rows, h or da; of db; of the backward's h.
template <int SRC>
__global__ void __launch_bounds__(FT_THREADS, TileGeo<SRC>::CTAS)
fp8_tokens_kernel(const __grid_constant__ CUtensorMap tm, const __grid_constant__ CUtensorMap tm_b,
                  const __grid_constant__ CUtensorMap tm_h, const Source src,
                  const int32_t* __restrict__ src_tok, long long src_rows,
                  const int32_t* __restrict__ offsets, int G, long long rows, const QuantOut out,
                  const QuantOut out_h, int* err) {
  griddep_wait();   // see common.cuh: dependent launches
  using GE = TileGeo<SRC>;
  constexpr int PER = GE::PER;
  constexpr bool BWD = SRC == SRC_SWIGLU_BWD;
  extern __shared__ uint4 dyn[];   // [BUFS][128][16] after the next 1 KB boundary
  uint4* bufs = reinterpret_cast<uint4*>(
      (reinterpret_cast<uintptr_t>(dyn) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ uint32_t s_max[BWD ? 24 : 8][64];
  __shared__ Blocks blocks;
  if (!count_blocks(blocks, offsets, G, rows, err)) return;
  const int tid = threadIdx.x;
  const int width = BWD ? src.f : src.cols;
  const int gx = (width + 127) / 128;
  const long long total = static_cast<long long>(blocks.first[G]) * gx;
  const int r = tid >> 4, ch = tid & 15;   // pieces (r + 32 u, ch)
  auto fetch = [&](const TileAt& t, uint4* dst) {
    const int c = t.c0 + 8 * ch;
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const int rr = r + 32 * u, at = rr * 16 + ch;
      const bool in = rr < t.nr && c < width;
      int row = in ? t.r0 + rr : 0;
      if (SRC == SRC_ROWS && src_tok && in) {
        row = __ldg(src_tok + row);
        if (row < 0 || row >= src_rows) {
          flag_error(err, MOE_DEVERR_BAD_INDEX);
          row = 0;
        }
      }
      const int cc = in ? c : 0;
      if constexpr (SRC == SRC_ROWS) {
        cp_async16(dst + at, src.x + row * src.ld + cc, in);
      } else {
        const __nv_bfloat16* a = src.x + static_cast<long long>(row) * (2 * src.f) + cc;
        cp_async16(dst + at, a, in);
        cp_async16(dst + FT_TILE + at, a + src.f, in);
        if constexpr (BWD)
          cp_async16(dst + 2 * FT_TILE + at, src.dh + static_cast<long long>(row) * src.f + cc, in);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  Walk walk(blockIdx.x, gridDim.x, gx);
  TileAt next;
  if (blockIdx.x < total) {
    next = walk.at(blocks);
    fetch(next, bufs);
  }
  int buf = 0;
  for (long long item = blockIdx.x; item < total; item += gridDim.x, buf ^= 1) {
    const TileAt t = next;
    const bool more = item + gridDim.x < total;
    uint4* raw = bufs + (SRC == SRC_ROWS ? buf * FT_TILE : 0);
    uint4* tile = SRC == SRC_SWIGLU ? bufs + 2 * FT_TILE : raw;
    asm volatile("cp.async.wait_all;" ::: "memory");   // this thread's pieces of this tile
    const int c = t.c0 + 8 * ch;
    uint4 v[4];
    if constexpr (BWD) {
#pragma unroll 1
      for (int u = 0; u < PER; u += 2) {   // two rows at a time
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int rr = r + 32 * (u + i);
          uint4* at = raw + rr * 16 + ch;
          const uint4 a = at[0], b = at[FT_TILE], d = at[2 * FT_TILE];
          uint32_t x[4] = {0u, 0u, 0u, 0u}, y[4] = {0u, 0u, 0u, 0u}, z[4] = {0u, 0u, 0u, 0u};
          if (rr < t.nr && c < width) {
            const uint32_t *pa = &a.x, *pb = &b.x, *pd = &d.x;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const Swiglu2 w = swiglu_bwd2(pa[k], pb[k], pd[k]);
              x[k] = w.da;
              y[k] = w.db;
              z[k] = w.h;
            }
          }
          v[i] = make_uint4(x[0], x[1], x[2], x[3]);
          v[2 + i] = make_uint4(y[0], y[1], y[2], y[3]);
          at[0] = v[i];
          at[FT_TILE] = v[2 + i];
          at[2 * FT_TILE] = make_uint4(z[0], z[1], z[2], z[3]);
        }
        if (out.codes)
          tile_rows(v, t, src.cols, out, [&](int i) {
            return make_int2(r + 32 * (u + (i & 1)), c + (i >> 1) * src.f);
          });
      }
    } else {
#pragma unroll
      for (int u = 0; u < PER; ++u) {
        const uint4* at = raw + (r + 32 * u) * 16 + ch;
        if constexpr (SRC == SRC_ROWS) v[u] = at[0];
        else v[u] = r + 32 * u < t.nr && c < width ? silu_mul8(at[0], at[FT_TILE])
                                                   : make_uint4(0u, 0u, 0u, 0u);
      }
      if (out.codes) {
        if (SRC == SRC_ROWS && src_tok) {
          // rows without a source (read as row 0) get no row codes; on a path of its own, since the
          // question costs rows in order 1% on theirs
          uint32_t bad = 0u;
#pragma unroll
          for (int u = 0; u < PER; ++u)
            if (r + 32 * u < t.nr) {
              const int row = __ldg(src_tok + t.r0 + r + 32 * u);
              if (row < 0 || row >= src_rows) bad |= 1u << u;
            }
          tile_rows(v, t, src.cols, out, [&](int i) {
            return make_int2((bad >> i) & 1u ? 128 : r + 32 * i, c);
          });
        } else {
          tile_rows(v, t, src.cols, out, [&](int i) { return make_int2(r + 32 * i, c); });
        }
      }
      if (tid == 0) bulk_wait_group_read<0>();   // the last tile's codes have left their buffer
    }
    __syncthreads();
    if constexpr (SRC == SRC_SWIGLU) {
#pragma unroll
      for (int u = 0; u < PER; ++u) tile[(r + 32 * u) * 16 + ch] = v[u];
      __syncthreads();
    }
    if (!BWD && more) {
      walk.next();
      next = walk.at(blocks);
      fetch(next, SRC == SRC_ROWS ? bufs + (buf ^ 1) * FT_TILE : raw);
    }
    uint8_t* box = reinterpret_cast<uint8_t*>(tile);
    constexpr int BOX = FT_TILE * 16;   // from one tile's to the next one's
    Columns cols;
    cols.read(tile, tid, s_max);
    if constexpr (BWD) {
      Columns cols_b;
      cols_b.read(tile + FT_TILE, tid, s_max + 8);
      __syncthreads();
      cols.write(tid, s_max, t.c0, 0, src.f, src.cols, t.kb, out, box);
      cols_b.write(tid, s_max + 8, t.c0, src.f, src.f, src.cols, t.kb, out, box + BOX);
      if (out_h.codes_t) {
        cols.read(tile + 2 * FT_TILE, tid, s_max + 16);
        __syncthreads();
        cols.write(tid, s_max + 16, t.c0, 0, src.f, src.f, t.kb, out_h, box + 2 * BOX);
      }
    } else {
      __syncthreads();
      cols.write(tid, s_max, t.c0, 0, src.cols, src.cols, t.kb, out, box);
    }
    fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
      const uint32_t at = smem_u32(box);
      tma_store_2d(&tm, at, 128 * t.kb, t.c0);
      if (BWD) {
        tma_store_2d(&tm_b, at + BOX, 128 * t.kb, t.c0);
        if (out_h.codes_t) tma_store_2d(&tm_h, at + 2 * BOX, 128 * t.kb, t.c0);
      }
      bulk_commit_group();
      if (BWD) bulk_wait_group_read<0>();
    }
    if (BWD && more) {
      walk.next();
      next = walk.at(blocks);
      __syncthreads();   // the codes have left the buffers
      fetch(next, raw);
    }
  }
  if (tid == 0) bulk_wait_group_all();   // stores done before exit
  griddep_launch();
}

// ------------------------------------------------------------------ weights
// One CTA per 128 x 128 block of W [G][N][K]: one scale, the codes row-major and, for the data
// gradient's product, transposed (its block scales transposed with them).
template <int W>
__global__ void __launch_bounds__(FQ_THREADS)
fp8_weights_kernel(const __nv_bfloat16* __restrict__ w, int N, int K, int nb, int kb,
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
    if (n < N && c < K) v[u] = load8<W>(w + (g * N + n) * K + c, K - c);
    m = max2(m, max_mag8(v[u]));
  }
  m = max(m & 0xffffu, m >> 16);
  m = __reduce_max_sync(FULL_MASK, m);
  if ((tid & 31) == 0) s_max[tid >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, s_max[i]);
  const float r = block_quotient(m, pow2, 0);
  if (tid == 0) {
    const float s = block_quotient(m, pow2, 1);
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

bool on(const void* p, unsigned bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

template <int SRC, int W>
cudaError_t launch_rows(const Source& s, const Fp8QuantArgs& a, const QuantOut& o,
                        cudaStream_t st) {
  const long long want = (a.rows + FQ_THREADS / 32 - 1) / (FQ_THREADS / 32);
  auto grid = [&](int per_sm) {
    const long long most = static_cast<long long>(fq_sms()) * per_sm;
    return dim3(static_cast<unsigned>(want < most ? want : most));
  };
  if constexpr (SRC == SRC_ROWS && W == 8) {
    const cudaError_t e = cudaFuncSetAttribute(
        fp8_rows_ring_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, FR_SMEM);
    if (e != cudaSuccess) return e;
    return launch_pdl(fp8_rows_ring_kernel, grid(4 * FR_CTAS), dim3(FQ_THREADS), FR_SMEM, st, 1, s,
                      a.src_tok, a.src_rows, a.offsets, a.G, a.rows, o, a.err);
  } else if constexpr (SRC == SRC_SWIGLU && W == 8) {
    if ((s.f + 255) / 256 % 4 == 0)   // (see fp8_swiglu_rows_kernel)
      return launch_pdl(fp8_rows_kernel<SRC, W>, grid(8), dim3(FQ_THREADS), 0, st, 1, s, a.src_tok,
                        a.src_rows, a.offsets, a.G, a.rows, o, a.err);
    return launch_pdl(fp8_swiglu_rows_kernel, grid(8), dim3(FQ_THREADS), 0, st, 1, s, a.offsets,
                      a.G, a.rows, o, a.err);
  } else {
    return launch_pdl(fp8_rows_kernel<SRC, W>, grid(8), dim3(FQ_THREADS), 0, st, 1, s, a.src_tok,
                      a.src_rows, a.offsets, a.G, a.rows, o, a.err);
  }
}

template <int SRC, int W>
cudaError_t launch_tokens(const Source& s, const Fp8QuantArgs& a, const QuantOut& o,
                          const QuantOut& oh, cudaStream_t st) {
  constexpr bool BWD = SRC == SRC_SWIGLU_BWD;
  const int width = BWD && W == 8 ? s.f : s.cols;
  const long long items = fp8_token_blocks(a.rows, a.G) * ((width + 127) / 128);
  auto grid = [&](int per_sm) {
    const long long most = static_cast<long long>(fq_sms()) * per_sm;
    return dim3(static_cast<unsigned>(items < most ? items : most));
  };
  if constexpr (W == 8) {
    using GE = TileGeo<SRC>;
    auto kern = fp8_tokens_kernel<SRC>;
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, GE::SMEM);
    if (e != cudaSuccess) return e;
    CUtensorMap tm, tm_b, tm_h;
    const uint64_t len = 128ull * static_cast<uint64_t>(o.kb_cap);
    // `width` rows: what the last box has past them is not written
    auto map = [&](CUtensorMap* m, uint8_t* codes) {
      return fp8_codes_map(m, codes, len, len, static_cast<uint64_t>(width), 128);
    };
    if (!map(&tm, o.codes_t)) return cudaErrorInvalidValue;
    tm_b = tm_h = tm;
    if (BWD && (!map(&tm_b, o.codes_t + static_cast<uint64_t>(s.f) * len) ||
                (oh.codes_t && !map(&tm_h, oh.codes_t))))
      return cudaErrorInvalidValue;
    return launch_pdl(kern, grid(GE::CTAS), dim3(FT_THREADS), GE::SMEM, st, 1, tm, tm_b, tm_h, s,
                      a.src_tok, a.src_rows, a.offsets, a.G, a.rows, o, oh, a.err);
  } else {
    return launch_pdl(fp8_tokens_any_kernel<SRC, W>, grid(2), dim3(FT_THREADS), 0, st, 1, s,
                      a.src_tok, a.src_rows, a.offsets, a.G, a.rows, o, a.err);
  }
}

// One kernel where all that is asked for can come from it.
template <int SRC, int W>
cudaError_t launch_quant(const Source& s, const Fp8QuantArgs& a, const QuantOut& o,
                         const QuantOut& oh, cudaStream_t st) {
  return o.codes_t ? launch_tokens<SRC, W>(s, a, o, oh, st) : launch_rows<SRC, W>(s, a, o, st);
}

// The backward reads a, b and dh once for da, db and h.  Where the blocks of da and db share one (f
// no multiple of 128) the tiles of 128 columns do not hold whole blocks of a row: the row codes
// come from a launch of their own (84 of 174 us at 16383 x 1376).
cudaError_t launch_bwd8(const Source& s, const Fp8QuantArgs& a, QuantOut o, const QuantOut& oh,
                        cudaStream_t st) {
  const bool whole = s.f % 128 == 0;
  if (o.codes_t) {
    QuantOut ot = o;
    if (!whole) ot.codes = nullptr;
    const cudaError_t e = launch_tokens<SRC_SWIGLU_BWD, 8>(s, a, ot, oh, st);
    if (e != cudaSuccess || whole) return e;
  }
  return whole ? launch_rows<SRC_SWIGLU_BWD, 128>(s, a, o, st)
               : launch_rows<SRC_SWIGLU_BWD, 8>(s, a, o, st);
}

// Calls go(integral constant) with what can be loaded at once: 8, 2 or 1 values.
template <typename Go>
cudaError_t by_width(bool eight, bool two, Go go) {
  if (eight) return go(std::integral_constant<int, 8>());
  return two ? go(std::integral_constant<int, 2>()) : go(std::integral_constant<int, 1>());
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
  QuantOut oh = o;
  oh.codes = nullptr;
  oh.codes_t = static_cast<uint8_t*>(a.h_codes_t);
  oh.scales_t = a.h_scales_t;
  if (a.src == FP8_SRC_ROWS)
    return by_width(on(a.x, 16) && a.ldx % 8 == 0 && a.C % 8 == 0,
                    on(a.x, 4) && a.ldx % 2 == 0 && a.C % 2 == 0, [&](auto w) {
                      return launch_quant<SRC_ROWS, decltype(w)::value>(s, a, o, oh, st);
                    });
  auto swiglu = [&](const Source& src, const QuantOut& out) {
    return by_width(a.f % 8 == 0, a.f % 2 == 0, [&](auto w) {
      return launch_quant<SRC_SWIGLU, decltype(w)::value>(src, a, out, oh, st);
    });
  };
  if (a.src == FP8_SRC_SWIGLU) return swiglu(s, o);
  if (a.f % 8 == 0) return launch_bwd8(s, a, o, oh, st);
  // other widths: h apart
  const cudaError_t e = a.f % 2 == 0 ? launch_quant<SRC_SWIGLU_BWD, 2>(s, a, o, oh, st)
                                     : launch_quant<SRC_SWIGLU_BWD, 1>(s, a, o, oh, st);
  if (e != cudaSuccess || !a.h_codes_t) return e;
  s.cols = a.f;
  return swiglu(s, oh);
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
  return by_width(on(W, 16) && K % 8 == 0, on(W, 4) && K % 2 == 0, [&](auto w) {
    return go(fp8_weights_kernel<decltype(w)::value>);
  });
}

}  // namespace moe
