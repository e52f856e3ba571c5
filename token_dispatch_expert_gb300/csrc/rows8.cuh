// rows8.cuh -- how the normalisation and the 8-bit checkpoints read and write rows: element types,
// vectors, codes, rows fetched ahead, sums over a row.
//
// A warp takes a row in chunks of 256 columns, eight to a lane, as vectors of V adjacent
// elements: element j of a lane is column
//     chunk + (j / V) * 32 V + lane * V + j % V.
// V = 8 makes 16-byte accesses of bf16 and 8-byte ones of codes; rows off that alignment, or of
// another width, take V = 2 or 1, whose accesses of a warp are still contiguous.  A block of 128
// columns is half a chunk: lanes 0-15 or 16-31 with V = 8, elements 0-3 or 4-7 of every lane with
// V = 2 and 1.  Bytes are kept as they were loaded (Raw8) until they are used, so that the loads
// of several rows or chunks can be under way together whatever their type; types are arguments,
// the same for a whole launch, so their branches are uniform.
#pragma once

#include <cuda_fp8.h>

#include <atomic>

#include "common.cuh"
#include "internal.h"

namespace moe {

constexpr int CHUNK = 256;

// Element types of rows: the public ones, then codes.
enum RowType : int { ROW_BF16 = MOE_OUT_BF16, ROW_FP32 = MOE_OUT_FP32, ROW_INT8 = 2, ROW_E4M3 = 3 };
__host__ __device__ inline int code_type(int format) {
  return format == MOE_CKPT_INT8 ? ROW_INT8 : ROW_E4M3;
}

struct Raw8 {
  uint32_t w[8];
};

template <int V>
__device__ __forceinline__ int elem_col(int chunk, int lane, int j) {
  return chunk + (j / V) * 32 * V + lane * V + j % V;
}

// The bytes of a lane's eight elements of the row at `row`; columns from C on are zeros.  Whole
// chunks, which most are, are read without a condition on every vector.
template <int V, bool ALL>
__device__ __forceinline__ void load_vectors(Raw8& r, const uint8_t* p, int type, int chunk, int C,
                                             int lane) {
#pragma unroll
  for (int i = 0; i < 8 / V; ++i) {
    const int c = elem_col<V>(chunk, lane, i * V);
    if (V == 2) {
      if (type == ROW_FP32) {
        uint2 v = make_uint2(0, 0);
        if (ALL || c < C) v = *reinterpret_cast<const uint2*>(p + 4 * static_cast<int64_t>(c));
        r.w[2 * i] = v.x;
        r.w[2 * i + 1] = v.y;
      } else {
        r.w[i] = 0;
        if (ALL || c < C)
          r.w[i] = type == ROW_BF16
                       ? *reinterpret_cast<const uint32_t*>(p + 2 * static_cast<int64_t>(c))
                       : static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(p + c));
      }
    } else {
      r.w[i] = 0;
      if (ALL || c < C)
        r.w[i] = type == ROW_BF16 ? static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(p + 2 * static_cast<int64_t>(c)))
                 : type == ROW_FP32 ? *reinterpret_cast<const uint32_t*>(p + 4 * static_cast<int64_t>(c))
                                    : static_cast<uint32_t>(p[c]);
    }
  }
}
template <int V>
__device__ __forceinline__ void load_raw(Raw8& r, const void* row, int type, int chunk, int C,
                                         int lane) {
  const uint8_t* p = static_cast<const uint8_t*>(row);
  if (V < 8) {
    if (chunk + CHUNK <= C) load_vectors<V, true>(r, p, type, chunk, C, lane);
    else load_vectors<V, false>(r, p, type, chunk, C, lane);
    return;
  }
  const int c = chunk + 8 * lane;
  uint4 v = make_uint4(0, 0, 0, 0), u = v;
  if (type == ROW_BF16) {
    if (c < C) v = *reinterpret_cast<const uint4*>(p + 2 * static_cast<int64_t>(c));
  } else if (type == ROW_FP32) {
    if (c < C) {
      const uint4* q = reinterpret_cast<const uint4*>(p + 4 * static_cast<int64_t>(c));
      v = q[0];
      u = q[1];
    }
    r.w[4] = u.x; r.w[5] = u.y; r.w[6] = u.z; r.w[7] = u.w;
  } else {
    if (c < C) {
      const uint2 t = *reinterpret_cast<const uint2*>(p + c);
      v.x = t.x;
      v.y = t.y;
    }
  }
  r.w[0] = v.x; r.w[1] = v.y;
  if (type == ROW_BF16 || type == ROW_FP32) { r.w[2] = v.z; r.w[3] = v.w; }
}

// Byte i of w as a number: with the sign bit flipped it is a whole number from 0 to 255 above
// 128, which as the low byte of 2^23 makes 2^23 + code + 128, so that one addition gives the code.
__device__ __forceinline__ float int8_value(uint32_t flipped, int i) {
  return __uint_as_float(__byte_perm(flipped, 0x4B000000u, 0x7440u | static_cast<uint32_t>(i))) -
         8388736.0f;
}
__device__ __forceinline__ float2 e4m3_values(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two & 0xffffu),
                                                   __NV_E4M3);
  return __half22float2(__half2(h));
}

// The values of a lane's eight elements (of codes: the numbers they are, without the scale).
template <int V>
__device__ __forceinline__ void unpack_raw(const Raw8& r, int type, float* f) {
  if (type == ROW_FP32) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(r.w[j]);
  } else if (type == ROW_BF16) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      f[j] = V == 1 ? bf16_lo(r.w[j]) : (j & 1) ? bf16_hi(r.w[j / 2]) : bf16_lo(r.w[j / 2]);
  } else if (type == ROW_INT8) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t w = V == 8 ? r.w[j / 4] : V == 2 ? r.w[j / 2] : r.w[j];
      f[j] = int8_value(w ^ 0x80808080u, V == 8 ? j % 4 : V == 2 ? j % 2 : 0);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const uint32_t two = V == 8 ? r.w[j / 4] >> (8 * (j % 4))
                                  : V == 2 ? r.w[j / 2] : r.w[j] | (r.w[j + 1] << 8);
      const float2 v = e4m3_values(two);
      f[j] = v.x; f[j + 1] = v.y;
    }
  }
}

template <int V>
__device__ __forceinline__ void load_values(float* f, const void* row, int type, int chunk, int C,
                                            int lane) {
  Raw8 r;
  load_raw<V>(r, row, type, chunk, C, lane);
  unpack_raw<V>(r, type, f);
}

// Store a lane's eight values, rounded to nearest where the type is bf16.
template <int V, bool ALL>
__device__ __forceinline__ void store_vectors(uint8_t* p, int type, int chunk, int C, int lane,
                                              const float* f) {
#pragma unroll
  for (int i = 0; i < 8 / V; ++i) {
    const int c = elem_col<V>(chunk, lane, i * V);
    if (!ALL && c >= C) continue;
    if (V == 2) {
      if (type == ROW_BF16)
        *reinterpret_cast<uint32_t*>(p + 2 * static_cast<int64_t>(c)) = pack_bf16x2(f[2 * i], f[2 * i + 1]);
      else
        *reinterpret_cast<float2*>(p + 4 * static_cast<int64_t>(c)) = make_float2(f[2 * i], f[2 * i + 1]);
    } else {
      if (type == ROW_BF16)
        *reinterpret_cast<__nv_bfloat16*>(p + 2 * static_cast<int64_t>(c)) = __float2bfloat16_rn(f[i]);
      else
        *reinterpret_cast<float*>(p + 4 * static_cast<int64_t>(c)) = f[i];
    }
  }
}
template <int V>
__device__ __forceinline__ void store_values(void* row, int type, int chunk, int C, int lane,
                                             const float* f) {
  uint8_t* p = static_cast<uint8_t*>(row);
  if (V < 8) {
    if (chunk + CHUNK <= C) store_vectors<V, true>(p, type, chunk, C, lane, f);
    else store_vectors<V, false>(p, type, chunk, C, lane, f);
    return;
  }
  const int c = chunk + 8 * lane;
  if (c >= C) return;
  if (type == ROW_BF16) {
    *reinterpret_cast<uint4*>(p + 2 * static_cast<int64_t>(c)) = pack8(f);
  } else {
    float4* q = reinterpret_cast<float4*>(p + 4 * static_cast<int64_t>(c));
    q[0] = make_float4(f[0], f[1], f[2], f[3]);
    q[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
}

// Multiply a lane's codes by their blocks' scales.  `first` is the column of the checkpoint's row
// at which the chunk's column 0 lies (blocks count from the row's start, so a part of a row that
// does not start at a block's border has blocks that end inside a vector's neighbours, but never
// inside a vector: V divides `first` and 128).
template <int V>
__device__ __forceinline__ void load_scales(float* s, const float* row_scales, int first, int chunk,
                                            int C, int lane) {
#pragma unroll
  for (int i = 0; i < 8 / V; ++i) {
    const int c = elem_col<V>(chunk, lane, i * V);
    s[i] = c < C ? row_scales[(first + c) >> 7] : 0.0f;
  }
}
// the same where the chunk starts at a block's border: two blocks at most to a lane
template <int V>
__device__ __forceinline__ void load_chunk_scales(float* s, const float* row_scales, int chunk, int C,
                                                  int lane) {
  if (V == 8) {
    load_scales<V>(s, row_scales, 0, chunk, C, lane);
    return;
  }
  const float lo = row_scales[chunk >> 7], hi = chunk + 128 < C ? row_scales[(chunk >> 7) + 1] : 0.0f;
#pragma unroll
  for (int i = 0; i < 8 / V; ++i) s[i] = i < 4 / V ? lo : hi;
}
template <int V>
__device__ __forceinline__ void scale_values(float* f, const float* s) {
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const float2 p = __fmul2_rn(make_float2(f[j], f[j + 1]), make_float2(s[j / V], s[(j + 1) / V]));
    f[j] = p.x;
    f[j + 1] = p.y;
  }
}

// ------------------------------------------------------------------ rows through shared memory
// A kernel that goes from row to row fetches the next rows while it works on one: every thread
// copies (cp.async) just the bytes that it will read itself into slots of its own, so the copies
// need no barrier, and as many rows are under way as there are slots, whatever the registers.
// Eight adjacent columns to a lane (V = 8).  A chunk's bytes in a slot: 512 for bf16, 1024 for
// fp32 (the lanes' first 16 bytes, then their second ones: no bank conflicts), 256 for codes.
__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// until at most `n` of the thread's newest groups are under way (0 <= n <= 3)
__device__ __forceinline__ void copy_wait(int n) {
  if (n == 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
  else if (n == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else if (n == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
  else asm volatile("cp.async.wait_group 3;" ::: "memory");
}

__device__ __forceinline__ void copy_chunk(uint8_t* slot, const void* row, int type, int chunk, int C,
                                           int lane) {
  const int c = chunk + 8 * lane;
  if (c >= C) return;
  const uint8_t* p = static_cast<const uint8_t*>(row);
  const uint32_t at = smem_u32(slot);
  if (type == ROW_BF16) {
    copy_async16(at + 16 * lane, p + 2 * static_cast<int64_t>(c));
  } else if (type == ROW_FP32) {
    copy_async16(at + 16 * lane, p + 4 * static_cast<int64_t>(c));
    copy_async16(at + 512 + 16 * lane, p + 4 * static_cast<int64_t>(c) + 16);
  } else {
    copy_async8(at + 8 * lane, p + c);
  }
}
// The bytes of a lane whose columns lie past the row's end are never copied: they are made zeros
// once.
__device__ __forceinline__ void clear_chunk(uint8_t* slot, int type, int lane) {
  if (type == ROW_BF16 || type == ROW_FP32)
    *reinterpret_cast<uint4*>(slot + 16 * lane) = make_uint4(0, 0, 0, 0);
  if (type == ROW_FP32) *reinterpret_cast<uint4*>(slot + 512 + 16 * lane) = make_uint4(0, 0, 0, 0);
  if (type != ROW_BF16 && type != ROW_FP32)
    *reinterpret_cast<uint2*>(slot + 8 * lane) = make_uint2(0, 0);
}
// a lane's eight values in a slot, as pairs (of codes: without the scale)
__device__ __forceinline__ void slot_values(float2* v, const uint8_t* slot, int type, int lane) {
  if (type == ROW_BF16) {
    const uint4 r = *reinterpret_cast<const uint4*>(slot + 16 * lane);
    v[0] = make_float2(bf16_lo(r.x), bf16_hi(r.x));
    v[1] = make_float2(bf16_lo(r.y), bf16_hi(r.y));
    v[2] = make_float2(bf16_lo(r.z), bf16_hi(r.z));
    v[3] = make_float2(bf16_lo(r.w), bf16_hi(r.w));
  } else if (type == ROW_FP32) {
    const float4 a = *reinterpret_cast<const float4*>(slot + 16 * lane);
    const float4 b = *reinterpret_cast<const float4*>(slot + 512 + 16 * lane);
    v[0] = make_float2(a.x, a.y);
    v[1] = make_float2(a.z, a.w);
    v[2] = make_float2(b.x, b.y);
    v[3] = make_float2(b.z, b.w);
  } else {
    const uint2 r = *reinterpret_cast<const uint2*>(slot + 8 * lane);
    Raw8 raw;
    raw.w[0] = r.x;
    raw.w[1] = r.y;
    float f[8];
    if (type == ROW_INT8) unpack_raw<8>(raw, ROW_INT8, f);
    else unpack_raw<8>(raw, ROW_E4M3, f);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = make_float2(f[2 * j], f[2 * j + 1]);
  }
}
// a lane's eight values of a vector at `p` (the parameters), as pairs; c < C
__device__ __forceinline__ void vector_values(float2* v, const void* p, int type, int c) {
  if (type == ROW_BF16) {
    const uint4 r = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + 2 * static_cast<int64_t>(c));
    v[0] = make_float2(bf16_lo(r.x), bf16_hi(r.x));
    v[1] = make_float2(bf16_lo(r.y), bf16_hi(r.y));
    v[2] = make_float2(bf16_lo(r.z), bf16_hi(r.z));
    v[3] = make_float2(bf16_lo(r.w), bf16_hi(r.w));
  } else {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const uint8_t*>(p) + 4 * static_cast<int64_t>(c));
    const float4 a = q[0], b = q[1];
    v[0] = make_float2(a.x, a.y);
    v[1] = make_float2(a.z, a.w);
    v[2] = make_float2(b.x, b.y);
    v[3] = make_float2(b.z, b.w);
  }
}
__device__ __forceinline__ void store_pairs(void* row, int type, int c, const float2* v) {
  if (type == ROW_BF16) {
    *reinterpret_cast<uint4*>(static_cast<uint8_t*>(row) + 2 * static_cast<int64_t>(c)) =
        make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y),
                   pack_bf16x2(v[2].x, v[2].y), pack_bf16x2(v[3].x, v[3].y));
  } else {
    float4* q = reinterpret_cast<float4*>(static_cast<uint8_t*>(row) + 4 * static_cast<int64_t>(c));
    q[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    q[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
  }
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// ------------------------------------------------------------------ saving a block
// s = amax / top, r = top / amax with amax = max(max |v|, 2^-110), each one correctly rounded
// quotient; int8 codes are the whole number nearest to v * r (ties to even), the product rounded
// once; E4M3 codes are E4M3(fp32(v * r)), as the quantisers of the products' operands make them.
constexpr float CKPT_AMAX_FLOOR = 0x1p-110f;
__device__ __forceinline__ float ckpt_top(int format) {
  return format == MOE_CKPT_INT8 ? 127.0f : 448.0f;
}
// of two magnitudes the larger, of three numbers the largest magnitude; a NaN wins
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max_mag3(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// The largest magnitudes of a lane's block(s): m[0] for V = 8 (the lane's half), m[0] and m[1]
// for V = 2 and 1; complete after the exchange over the warp.
template <int V>
__device__ __forceinline__ void lane_max(const float* f, float* m) {
  if (V == 8) {
    m[0] = max_mag3(max_mag3(f[0], f[1], f[2]), f[3], f[4]);
    m[0] = m[1] = max_mag3(max_mag3(m[0], f[5], f[6]), f[7], 0.0f);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      m[h] = max_mag3(max_mag3(f[4 * h], f[4 * h + 1], f[4 * h + 2]), f[4 * h + 3], 0.0f);
  }
}

// scale and factor of a block
__device__ __forceinline__ void block_scale(float amax, int format, float& scale, float& factor) {
  const float top = ckpt_top(format);
  if (amax < CKPT_AMAX_FLOOR) amax = CKPT_AMAX_FLOOR;
  scale = __fdiv_rn(amax, top);
  factor = __fdiv_rn(top, amax);
}

// The low byte of the result is the code: 1.5 * 2^23 + v * r, rounded once, holds the product's
// nearest whole number in its low bits (|v * r| < 127.5, so no code passes 127).
__device__ __forceinline__ uint32_t int8_code(float v, float r) {
  return __float_as_uint(fmaf(v, r, 12582912.0f));
}
__device__ __forceinline__ uint32_t e4m3_code2(float a, float b) {   // a in the low byte
  return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE,
                                                        __NV_E4M3));
}

// Store a lane's eight codes; r: the factor of elements 0-3 and of 4-7.  A factor that is not a
// positive number (a block with a NaN or an infinity) makes int8 codes of zero, which the block's
// scale then turns into NaN.
template <int V>
__device__ __forceinline__ void store_codes(void* row, int format, int chunk, int C, int lane,
                                            const float* f, const float* r) {
  uint8_t* p = static_cast<uint8_t*>(row);
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float* g = f + 4 * h;
    if (format == MOE_CKPT_INT8) {
      const uint32_t lo = __byte_perm(int8_code(g[0], r[h]), int8_code(g[1], r[h]), 0x0040);
      const uint32_t hi = __byte_perm(int8_code(g[2], r[h]), int8_code(g[3], r[h]), 0x0040);
      w[h] = r[h] > 0.0f ? __byte_perm(lo, hi, 0x5410) : 0u;
    } else {
      w[h] = e4m3_code2(g[0] * r[h], g[1] * r[h]) | (e4m3_code2(g[2] * r[h], g[3] * r[h]) << 16);
    }
  }
  if (V == 8) {
    const int c = chunk + 8 * lane;
    if (c < C) *reinterpret_cast<uint2*>(p + c) = make_uint2(w[0], w[1]);
  } else if (V == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = elem_col<V>(chunk, lane, 2 * i);
      if (c < C) *reinterpret_cast<uint16_t*>(p + c) = static_cast<uint16_t>(w[i / 2] >> (16 * (i % 2)));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = elem_col<V>(chunk, lane, j);
      if (c < C) p[c] = static_cast<uint8_t>(w[j / 4] >> (8 * (j % 4)));
    }
  }
}

// Quantise N chunks that the warp holds (f[i]: the lane's values of chunk[i] of the row whose codes
// and scales are at codes[i] and scales[i]; columns from C on are zeros, a chunk that starts at C
// is none).  With V = 8 the maxima of four chunks go through one set of shuffles: lanes exchange
// all but a share of the chunks at each step, so that each lane ends with one block, divides once
// for it, and the factors are handed back.
template <int V, int N>
__device__ __forceinline__ void save_chunks(void* const* codes, float* const* scales, int format,
                                            const int* chunk, int C, int lane,
                                            const float (*f)[8]) {
  float m[N][2];
#pragma unroll
  for (int i = 0; i < N; ++i) lane_max<V>(f[i], m[i]);
  if (V == 8) {
    float sc, fa, r[N];
    if (N == 4 || N == 2) {
      const bool b3 = lane & 8, b2 = lane & 4;
      float q;
      if (N == 4) {
        float a = b3 ? m[2 % N][0] : m[0][0], b = b3 ? m[3 % N][0] : m[1 % N][0];
        a = max_nan(a, __shfl_xor_sync(FULL_MASK, b3 ? m[0][0] : m[2 % N][0], 8));
        b = max_nan(b, __shfl_xor_sync(FULL_MASK, b3 ? m[1 % N][0] : m[3 % N][0], 8));
        q = max_nan(b2 ? b : a, __shfl_xor_sync(FULL_MASK, b2 ? a : b, 4));
      } else {
        q = max_nan(b3 ? m[1 % N][0] : m[0][0],
                    __shfl_xor_sync(FULL_MASK, b3 ? m[0][0] : m[1 % N][0], 8));
        q = max_nan(q, __shfl_xor_sync(FULL_MASK, q, 4));
      }
      q = max_nan(q, __shfl_xor_sync(FULL_MASK, q, 2));
      q = max_nan(q, __shfl_xor_sync(FULL_MASK, q, 1));
      block_scale(q, format, sc, fa);
      int c = b3 ? chunk[N == 4 ? 2 % N : 1 % N] : chunk[0];
      float* to = b3 ? scales[N == 4 ? 2 % N : 1 % N] : scales[0];
      if (N == 4 && b2) {
        c = b3 ? chunk[3 % N] : chunk[1 % N];
        to = b3 ? scales[3 % N] : scales[1 % N];
      }
      c += 128 * (lane >> 4);
      if ((lane & (N == 4 ? 3 : 7)) == 0 && c < C) to[c >> 7] = sc;
#pragma unroll
      for (int i = 0; i < N; ++i)
        r[i] = __shfl_sync(FULL_MASK, fa, (lane & 16) | (N == 4 ? i / 2 * 8 + i % 2 * 4 : i * 8));
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float q = m[i][0];
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) q = max_nan(q, __shfl_xor_sync(FULL_MASK, q, o));
        block_scale(q, format, sc, r[i]);
        const int c = chunk[i] + 128 * (lane >> 4);
        if ((lane & 15) == 0 && c < C) scales[i][c >> 7] = sc;
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float r2[2] = {r[i], r[i]};
      store_codes<V>(codes[i], format, chunk[i], C, lane, f[i], r2);
    }
  } else {
    // blocks 0 and 1 of a chunk: after the first exchange a lane keeps one of them
    const bool up = lane & 16;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float q = max_nan(up ? m[i][1] : m[i][0],
                        __shfl_xor_sync(FULL_MASK, up ? m[i][0] : m[i][1], 16));
      float sc, fa;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) q = max_nan(q, __shfl_xor_sync(FULL_MASK, q, o));
      block_scale(q, format, sc, fa);
      const int c = chunk[i] + 128 * (lane >> 4);
      if ((lane & 15) == 0 && c < C) scales[i][c >> 7] = sc;
      const float r[2] = {__shfl_sync(FULL_MASK, fa, 0), __shfl_sync(FULL_MASK, fa, 16)};
      store_codes<V>(codes[i], format, chunk[i], C, lane, f[i], r);
    }
  }
}
template <int V, int N>
__device__ __forceinline__ void save_row_chunks(void* codes, float* scales, int format,
                                                const int* chunk, int C, int lane,
                                                const float (*f)[8]) {
  void* c[N];
  float* s[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    c[i] = codes;
    s[i] = scales;
  }
  save_chunks<V, N>(c, s, format, chunk, C, lane, f);
}

// Whole rows through shared memory by bulk copies.  Eight adjacent columns of a lane (V = 8: the row
// starts at 16 bytes), or 32 columns apart (V = 1: rows at any element).
__device__ __forceinline__ float int8_number(uint32_t byte) {   // (see int8_value)
  return __uint_as_float((byte ^ 0x80u) | 0x4B000000u) - 8388736.0f;
}
template <int TYPE, int V>
__device__ __forceinline__ void smem_row_values(float2* v, const uint8_t* row, int chunk, int C, int lane) {
  if constexpr (V == 1) {
    const bool all = chunk + CHUNK <= C;
    const int c0 = chunk + lane;
    uint32_t r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = c0 + 32 * j;
      r[j] = 0;
      if (all || c < C) {
        if constexpr (TYPE == ROW_BF16) r[j] = *reinterpret_cast<const uint16_t*>(row + 2 * c);
        else if constexpr (TYPE == ROW_FP32) r[j] = *reinterpret_cast<const uint32_t*>(row + 4 * c);
        else r[j] = row[c];
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (TYPE == ROW_BF16) v[j] = make_float2(bf16_lo(r[2 * j]), bf16_lo(r[2 * j + 1]));
      else if constexpr (TYPE == ROW_FP32) v[j] = make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
      else if constexpr (TYPE == ROW_INT8) v[j] = make_float2(int8_number(r[2 * j]), int8_number(r[2 * j + 1]));
      else v[j] = e4m3_values(__byte_perm(r[2 * j], r[2 * j + 1], 0x0040));
    }
    return;
  }
  const int col = chunk + 8 * lane;
  if constexpr (TYPE == ROW_BF16) {
    const uint4 r = *reinterpret_cast<const uint4*>(row + 2 * col);
    v[0] = make_float2(bf16_lo(r.x), bf16_hi(r.x));
    v[1] = make_float2(bf16_lo(r.y), bf16_hi(r.y));
    v[2] = make_float2(bf16_lo(r.z), bf16_hi(r.z));
    v[3] = make_float2(bf16_lo(r.w), bf16_hi(r.w));
  } else if constexpr (TYPE == ROW_FP32) {
    const float4 a = *reinterpret_cast<const float4*>(row + 4 * col);
    const float4 b = *reinterpret_cast<const float4*>(row + 4 * col + 16);
    v[0] = make_float2(a.x, a.y);
    v[1] = make_float2(a.z, a.w);
    v[2] = make_float2(b.x, b.y);
    v[3] = make_float2(b.z, b.w);
  } else {
    const uint2 r = *reinterpret_cast<const uint2*>(row + col);
    if constexpr (TYPE == ROW_INT8) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t u = (j < 2 ? r.x : r.y) ^ 0x80808080u;
        v[j] = __fadd2_rn(make_float2(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440u | (j % 2 * 2))),
                                      __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440u | (j % 2 * 2 + 1)))),
                          both(-8388736.0f));
      }
    } else {
      v[0] = e4m3_values(r.x);
      v[1] = e4m3_values(r.x >> 16);
      v[2] = e4m3_values(r.y);
      v[3] = e4m3_values(r.y >> 16);
    }
  }
}
// The bytes [p, p + n) of rows that lie in [first, end), into shared memory at `to`, a 16-byte address
// that stands for p's rounded down: whole 16-byte pieces by the caller's bulk copy, bulk_span says
// which; what the tensor's own ends cut off a piece by plain copies, span_ends (ordered by the caller's
// arrival on the copy's barrier).  One thread.
struct Span {
  uint64_t lo, hi;
};
__device__ __forceinline__ Span bulk_span(const void* p, uint32_t n, const void* first, const void* end) {
  const uint64_t a = reinterpret_cast<uint64_t>(p), f = reinterpret_cast<uint64_t>(first);
  const uint64_t e = reinterpret_cast<uint64_t>(end);
  Span s{a & ~15ull, (a + n + 15) & ~15ull};
  if (s.lo < f) s.lo = (f + 15) & ~15ull;
  if (s.hi > e) s.hi = e & ~15ull;
  if (s.hi < s.lo) s.hi = s.lo;
  return s;
}
__device__ __forceinline__ void span_ends(uint8_t* to, const void* p, uint32_t n, const Span& s) {
  const uint8_t* a = static_cast<const uint8_t*>(p);
  const uint64_t at = reinterpret_cast<uint64_t>(p), low = at & ~15ull;
  for (uint64_t i = at; i < at + n; ++i) {
    if (i >= s.lo && i < s.hi) i = s.hi;
    if (i < at + n) to[i - low] = a[i - at];
  }
}

// The 16-byte pieces that the bytes [p, p + n) touch, copied by a warp to `to`, which stands for p rounded
// down; at most 32 * ROUNDS + 1 of them.  Where they pass an end of their tensor, [first, end), the bytes
// themselves are read.
template <int ROUNDS>
__device__ __forceinline__ void copy_pieces(uint8_t* to, const void* p, int n, const void* first,
                                            const void* end, int lane) {
  const uint64_t low = reinterpret_cast<uint64_t>(p) & ~15ull;
  const int skip = static_cast<int>(reinterpret_cast<uint64_t>(p)) & 15, want = skip + n;   // bytes from low
  if (low >= reinterpret_cast<uint64_t>(first) &&
      low + ((want + 15) & ~15) <= reinterpret_cast<uint64_t>(end)) {
    const uint32_t dst = smem_u32(to);
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r)
      if (512 * r + 16 * lane < want)
        copy_async16(dst + 512 * r + 16 * lane, reinterpret_cast<const uint8_t*>(low) + 512 * r + 16 * lane);
    if (lane == 0 && 512 * ROUNDS < want)
      copy_async16(dst + 512 * ROUNDS, reinterpret_cast<const uint8_t*>(low) + 512 * ROUNDS);
    return;
  }
  // (a tensor's first and last rows)
  for (int i = skip + lane; i < want; i += 32) to[i] = reinterpret_cast<const uint8_t*>(low)[i];
}
// untiled bulk copy global -> shared of a multiple of 16 bytes between 16-byte addresses
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// ------------------------------------------------------------------ sums over a row
constexpr int MAX_WARPS = 16;   // of a row that stays in registers: 16 * 4 chunks of 256 columns

struct RowSums {
  float part[2][2][MAX_WARPS];   // [buffer][which sum][warp]
};
// Before the first sum: the parts that no warp writes are zeros, so that they are read by fours.
__device__ __forceinline__ void row_sum_init(RowSums& sh) {
  for (int i = threadIdx.x; i < 4 * MAX_WARPS; i += blockDim.x) (&sh.part[0][0][0])[i] = 0.0f;
  __syncthreads();
}
__device__ __forceinline__ float row_total(const float* part, int nw) {
  float s = 0.0f;
  for (int i = 0; i < nw; i += 4) {
    const float4 p = *reinterpret_cast<const float4*>(part + i);
    s += (p.x + p.y) + (p.z + p.w);
  }
  return s;
}
// Sums over the nw warps that share a row: every thread gets them, added in one order.  `turn`
// alternates between two buffers, so that one barrier a sum is enough.
__device__ __forceinline__ float row_sum1(float a, RowSums& sh, int turn, int warp, int nw) {
  a = warp_sum(a);
  if (nw == 1) return a;
  if ((threadIdx.x & 31) == 0) sh.part[turn][0][warp] = a;
  __syncthreads();
  return row_total(sh.part[turn][0], nw);
}
// of two numbers at once: the halves of the warp take one each after the first exchange.  `barrier`:
// the group of nw warps' own one, where a CTA holds several.
__device__ __forceinline__ float2 row_sum2(float a, float b, RowSums& sh, int turn, int warp, int nw,
                                           int barrier = 0) {
  const int lane = threadIdx.x & 31;
  const bool up = lane & 16;
  float v = (up ? b : a) + __shfl_xor_sync(FULL_MASK, up ? a : b, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(FULL_MASK, v, o);
  if (nw == 1) return make_float2(__shfl_sync(FULL_MASK, v, 0), __shfl_sync(FULL_MASK, v, 16));
  if ((lane & 15) == 0) sh.part[turn][lane >> 4][warp] = v;
  if (barrier == 0) __syncthreads();
  else asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(32 * nw) : "memory");
  return make_float2(row_total(sh.part[turn][0], nw), row_total(sh.part[turn][1], nw));
}
__device__ __forceinline__ const void* row_at(const void* p, int64_t row, int64_t ld, int size) {
  return static_cast<const uint8_t*>(p) + row * ld * size;
}
__device__ __forceinline__ void* row_at(void* p, int64_t row, int64_t ld, int size) {
  return static_cast<uint8_t*>(p) + row * ld * size;
}

// ------------------------------------------------------------------ columns that stay
// What has no sums over a row goes down the columns: a warp keeps one chunk of 256 columns and takes
// every `groups`-th row, so that the columns' conditions and parameters are found once and a row's
// address is the last one's plus a constant.
constexpr int WALK_THREADS = 256, WALK_WARPS = WALK_THREADS / 32;
struct Walk {
  int chunk;
  int64_t row, groups;
  bool any;
};
__device__ __forceinline__ Walk walk_start(int per, int groups) {
  const unsigned gw = blockIdx.x * WALK_WARPS + (threadIdx.x >> 5);
  Walk w;
  w.row = gw / static_cast<unsigned>(per);
  w.chunk = static_cast<int>(gw - static_cast<unsigned>(w.row) * per) * CHUNK;
  w.groups = groups;
  w.any = w.row < groups;
  return w;
}
// How much shared memory a kernel may be launched with: all there is, said once for each device.
template <auto KERNEL>
inline cudaError_t allow_smem(int bytes) {
  static std::atomic<uint64_t> said{0};
  if (bytes <= 40 * 1024) return cudaSuccess;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (said.load(std::memory_order_relaxed) & bit && dev < 64) return cudaSuccess;
  cudaFuncAttributes f;
  e = cudaFuncGetAttributes(&f, KERNEL);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             227 * 1024 - static_cast<int>(f.sharedSizeBytes));
  if (e == cudaSuccess) said.fetch_or(bit, std::memory_order_relaxed);
  return e;
}
// how many groups of warps: enough for `warps` to an SM, no more than rows
struct WalkGrid {
  int per, groups;
  dim3 grid;
};
inline int row_sms() {
  int dev = 0, sms = 152;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}
// CTAs of a kernel that an SM holds by its registers
template <auto KERNEL>
inline int ctas_by_registers(int threads) {
  static const int regs = [] {   // (of this kernel, whatever the device: one architecture)
    cudaFuncAttributes f;
    return cudaFuncGetAttributes(&f, KERNEL) == cudaSuccess ? (f.numRegs + 7) / 8 * 8 : 128;
  }();
  int n = 65536 / (regs * threads);
  if (n > 2048 / threads) n = 2048 / threads;
  return n < 1 ? 1 : n;
}
inline WalkGrid walk_grid(int64_t rows, int C, int warps) {
  WalkGrid g;
  g.per = (C + CHUNK - 1) / CHUNK;
  // (not so many that a warp has fewer than 16 rows, down to what runs at once)
  const int64_t most = rows * g.per / (16 * static_cast<int64_t>(row_sms()));
  if (warps > most) warps = static_cast<int>(most < 32 ? 32 : most);
  int64_t n = (static_cast<int64_t>(row_sms()) * warps + g.per - 1) / g.per;
  if (n > rows) n = rows;
  g.groups = static_cast<int>(n < 1 ? 1 : n);
  g.grid = dim3(static_cast<unsigned>((static_cast<int64_t>(g.groups) * g.per + WALK_WARPS - 1) / WALK_WARPS));
  return g;
}

// ------------------------------------------------------------------ host: which V
// Rows at p, `ld` elements of `size` bytes apart.
inline bool rows_fit(const void* p, int64_t ld, int size, int v) {
  const int64_t a = v == 8 ? (size == 1 ? 8 : 16) : static_cast<int64_t>(v) * size;
  return !p || (reinterpret_cast<uintptr_t>(p) % a == 0 && (ld * size) % a == 0);
}
__host__ __device__ inline int row_size(int type) { return type == ROW_BF16 ? 2 : type == ROW_FP32 ? 4 : 1; }

constexpr int ROW_SMEM = 216 * 1024;   // of an SM's shared memory, for the rows in flight

}  // namespace moe
