// router.cu -- group-limited routing: scores (softmax over all experts, or sigmoid), a
// balance bias that only the choice sees, the best groups of experts, the top-k inside
// them, weights renormalised over the chosen or not; and the gradient of the weights.
//
// For token t with logits l (NaN counts as -inf and sets MOE_DEVERR_NAN_LOGIT, +inf as the
// largest finite value; an expert at -inf is out of service and never chosen):
//   score   s_e = sigma(l_e)  or  exp(l_e - m) / sum_i exp(l_i - m)
//   key     c_e = s_e + b_e with a bias, else l_e (the same order, and no ties by rounding)
//   group   its best c, or the sum of its two best (of s without a bias); the top_groups
//           best groups stay
//   choice  the k largest keys among them, in descending order; every tie goes to the
//           lower index.  Slots that nothing is left for: expert -1, weight 0, dropped.
//   weight  route_scale * s_e, or route_scale * s_e / sum of the chosen s
//
// Keys with a bias are numbers of their own, so their order is defined in 64 bits: two
// experts whose keys differ by less than the fp32 rounding error would otherwise be ordered
// by the accident of an implementation.  The kernel computes fp32 keys, takes the choice
// from them, and checks that every decision it made had a margin above the keys' error bound.
// Where neighbours in the order are closer (one token in some thousand with 256 sigmoid scores),
// the few candidates' 64-bit keys decide, one lane each; where two groups are, the whole choice
// is made again from 64-bit keys.  (Doing the latter for all of them took 20 us, most of it
// fetching the instructions of code that nothing else runs.)
//
// One warp per token, one CTA per 32-token chunk (32 warps).  A lane sorts its E / 32 keys; the
// choice is k rounds of a warp maximum over the lanes' heads (redux.sync on order-preserving
// 32-bit keys, then on the id among equals), whose lane moves its list up.  The chunk's histogram
// and the ranks inside it are bit masks (as in route.cu); order_count (a warp per expert) and
// order_assign follow; a single chunk (T <= 32) does their work itself, in one launch.
// Not bound by bytes: 4 MB of logits for 4096 tokens are 0.6 us of bandwidth.  One token over 256
// experts takes 3.8 us on the device and 7.7 us with the call, which the host bounds.  4096 tokens
// take 13.4 to 14.4 us in three launches: about 1640 warp instructions a token on 128 SMs, 67% of
// their issue slots, then two launches that wait for all chunks of the one before.  The gradient for
// 8192 tokens of 128 softmax scores takes 5.5 us with the call, most of it the launch.
#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int RG_CHUNK = 32;
constexpr int RG_THREADS = 1024;
constexpr float F32_MAX = 3.402823466e38f;

__device__ __forceinline__ uint32_t key32(float x) {   // order-preserving; 0 below every real
  uint32_t u = __float_as_uint(x);
  if (x == 0.0f) u = 0u;   // +0 and -0 compare equal
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float unkey32(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
__device__ __forceinline__ unsigned long long key64(double x) {
  unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(x));
  if (x == 0.0) u = 0ull;
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

__device__ __forceinline__ unsigned long long warp_max(unsigned long long v) {
  const uint32_t hi = static_cast<uint32_t>(v >> 32);
  const uint32_t top = __reduce_max_sync(FULL_MASK, hi);
  const uint32_t lo = hi == top ? static_cast<uint32_t>(v) : 0u;
  return (static_cast<unsigned long long>(top) << 32) | __reduce_max_sync(FULL_MASK, lo);
}
__device__ __forceinline__ float warp_fmax(float v) {
  return unkey32(__reduce_max_sync(FULL_MASK, key32(v)));
}

// e^x and 1 / d for the keys, off by two ulp and one ulp (the weights use expf and divisions)
__device__ __forceinline__ float fast_exp(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 0x1.715476p+0f));
  return r;
}
__device__ __forceinline__ float fast_rcp(float d) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  return r;
}

// the best 64-bit key left in the warp (0: none) and its expert (the lowest id among equals);
// the winner is taken out of its lane's keys
template <int VPL>
__device__ __forceinline__ void take_best(unsigned long long* key, int lane, int& e) {
  unsigned long long mine = key[0];
#pragma unroll
  for (int s = 1; s < VPL; ++s) mine = key[s] > mine ? key[s] : mine;
  const unsigned long long top = warp_max(mine);
  e = -1;
  if (top == 0) return;
  uint32_t id = 0xffffffffu;
#pragma unroll
  for (int s = VPL - 1; s >= 0; --s)
    if (key[s] == top) id = lane + 32 * s;
  id = __reduce_min_sync(FULL_MASK, id);
#pragma unroll
  for (int s = 0; s < VPL; ++s)
    if (id == static_cast<uint32_t>(lane + 32 * s)) key[s] = 0;
  e = static_cast<int>(id);
}

// This lane's keys in descending order, equal ones by ascending id (id = lane + 32 s).
template <int VPL>
struct SortedKeys {
  uint32_t key[VPL];
  int id[VPL];
  __device__ __forceinline__ void order(int i, int j) {   // i < j: the larger (lower id) first
    const bool swap = key[j] > key[i] || (key[j] == key[i] && id[j] < id[i]);
    const uint32_t k = swap ? key[j] : key[i];
    const int d = swap ? id[j] : id[i];
    key[j] = swap ? key[i] : key[j];
    id[j] = swap ? id[i] : id[j];
    key[i] = k;
    id[i] = d;
  }
  __device__ __forceinline__ void sort(int lane) {
#pragma unroll
    for (int s = 0; s < VPL; ++s) id[s] = lane + 32 * s;
    // Batcher's merge exchange
#pragma unroll
    for (int p = 1; p < VPL; p *= 2)
#pragma unroll
      for (int k = p; k >= 1; k /= 2)
#pragma unroll
        for (int j = k % p; j + k < VPL; j += 2 * k)
#pragma unroll
          for (int i = 0; i < k; ++i)
            if ((i + j) / (2 * p) == (i + j + k) / (2 * p) && i + j + k < VPL)
              order(i + j, i + j + k);
  }
  // the best one left in the warp (0: none) and its expert
  __device__ __forceinline__ uint32_t take(int lane, int& e) {
    const uint32_t top = __reduce_max_sync(FULL_MASK, key[0]);
    e = static_cast<int>(__reduce_min_sync(
        FULL_MASK, key[0] == top ? static_cast<uint32_t>(id[0]) : 0xffffffffu));
    if ((e & 31) == lane) {
#pragma unroll
      for (int s = 0; s + 1 < VPL; ++s) {
        key[s] = key[s + 1];
        id[s] = id[s + 1];
      }
      key[VPL - 1] = 0u;
    }
    if (top == 0u) e = -1;
    return top;
  }
};

struct RouterParams {
  const float* logits;
  const float* bias;
  int64_t T;
  int E, k, G, per, top_groups, top2, sigmoid, renorm, cap;
  int per_magic;           // ceil(2^16 / per): e / per = e * per_magic >> 16 for e < 256
  int lanes_log2, turns;   // 2^lanes_log2 lanes scan a group, in `turns` steps
  float scale;
};
__device__ __forceinline__ int group_of(const RouterParams& p, int e) {
  return (e * p.per_magic) >> 16;
}

// Worth of every group: the L = 2^lanes_log2 lanes g L .. of group g each scan part of its values
// (staged in shared memory) and are joined.  The scan starts at a place that depends on g, so that
// the groups of one step read different banks.  -inf: nothing in service.
template <typename F>
__device__ __forceinline__ F group_worth(const F* val, const RouterParams& p, int lane) {
  const int L = 1 << p.lanes_log2, g = lane >> p.lanes_log2, sub = lane & (L - 1);
  const F none = -static_cast<F>(INFINITY);
  F m1 = none, m2 = none;
  if (g < p.G) {
    int i = sub + L * (g < p.turns ? g : 0);
    for (int n = 0; n < p.turns; ++n) {
      if (i < p.per) {
        const F v = val[g * p.per + i];
        const F lo = v < m1 ? v : m1;
        m1 = v > m1 ? v : m1;
        m2 = lo > m2 ? lo : m2;
      }
      i += L;
      if (i >= L * p.turns) i = sub;
    }
  }
  for (int o = 1; o < L; o <<= 1) {
    const F a = __shfl_xor_sync(FULL_MASK, m1, o), b = __shfl_xor_sync(FULL_MASK, m2, o);
    const F lo = a < m1 ? a : m1;
    m1 = a > m1 ? a : m1;
    m2 = b > m2 ? b : m2;
    m2 = lo > m2 ? lo : m2;
  }
  return (p.top2 && m2 != none) ? m1 + m2 : m1;
}

// Bit g set for each of the top_groups best groups; margin: the least worth that stays minus
// the best that goes (+inf where nothing goes).
template <typename F>
__device__ __forceinline__ uint32_t choose_groups(F worth, const RouterParams& p, int lane,
                                                  F& margin) {
  const int g = lane >> p.lanes_log2;
  int rank = 0;
  for (int j = 0; j < p.G; ++j) {
    const F o = __shfl_sync(FULL_MASK, worth, j << p.lanes_log2);
    rank += (o > worth || (o == worth && j < g)) ? 1 : 0;
  }
  const bool head = g < p.G && (lane & ((1 << p.lanes_log2) - 1)) == 0;
  const bool in = head && rank < p.top_groups;
  // the last one in and the first one out
  const uint32_t heads = __ballot_sync(FULL_MASK, in);
  const uint32_t last = __ballot_sync(FULL_MASK, head && rank == p.top_groups - 1);
  const uint32_t first = __ballot_sync(FULL_MASK, head && rank == p.top_groups);
  margin = __shfl_sync(FULL_MASK, worth, __ffs(last) - 1) -
           __shfl_sync(FULL_MASK, worth, __ffs(first) - 1);
  uint32_t mask = 0u;
  for (int j = 0; j < p.G; ++j) mask |= ((heads >> (j << p.lanes_log2)) & 1u) << j;
  return mask;
}

// The choice from 64-bit keys.  val: the token's logits (NaN already -inf), wide: room for as
// many doubles, both this warp's own.  Lane j gets the j-th choice.
template <int VPL>
__device__ __noinline__ int choose_exact(const RouterParams p, const float* val, double* wide,
                                         int lane) {
  double m = 0.0, z = 0.0;
  if (!p.sigmoid) {
    float mf = -F32_MAX;
#pragma unroll
    for (int s = 0; s < VPL; ++s)
      if (lane + 32 * s < p.E) mf = fmaxf(mf, val[lane + 32 * s]);
    m = static_cast<double>(warp_fmax(mf));
  }
  double sc[VPL];   // unrolled: one 64-bit exponential's latency hides behind the others'
#pragma unroll
  for (int s = 0; s < VPL; ++s) {
    const double l = lane + 32 * s < p.E ? static_cast<double>(val[lane + 32 * s]) : -INFINITY;
    const double x = exp(p.sigmoid ? -l : l - m);
    sc[s] = p.sigmoid ? 1.0 / (1.0 + x) : x;
    z += sc[s];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(FULL_MASK, z, o);
  unsigned long long key[VPL];
#pragma unroll
  for (int s = 0; s < VPL; ++s) {
    const int e = lane + 32 * s;
    key[s] = 0ull;
    if (e >= p.E) continue;
    const bool live = val[e] > -INFINITY;
    const double l = static_cast<double>(val[e]);
    double c = p.sigmoid ? sc[s] : sc[s] / z;
    if (p.bias) c += static_cast<double>(__ldg(p.bias + e));
    // without a bias the experts' own order is that of the logits
    if (live) key[s] = key64(p.bias ? c : l);
    wide[e] = !live ? -INFINITY : (!p.bias && !p.top2) ? l : c;
  }
  if (p.G > 1) {
    __syncwarp();
    double margin;
    const uint32_t mask = choose_groups(group_worth(wide, p, lane), p, lane, margin);
#pragma unroll
    for (int s = 0; s < VPL; ++s)
      if (lane + 32 * s < p.E && !((mask >> group_of(p, lane + 32 * s)) & 1u)) key[s] = 0ull;
  }
  int sel = -1;
  for (int j = 0; j < p.k; ++j) {
    int e;
    take_best<VPL>(key, lane, e);
    if (lane == j) sel = e;
  }
  return sel;
}

// Lane j < n holds candidate my_e: the candidates in the order of their 64-bit keys.
__device__ __noinline__ double exp64(double x) { return exp(x); }
__device__ __noinline__ int order_exact(const RouterParams p, const float* val, int* list, int my_e,
                                        int n, int lane) {
  double m = 0.0, z = 1.0;
  if (!p.sigmoid) {   // the sum over all experts
    float mf = -F32_MAX;
    for (int e = lane; e < p.E; e += 32) mf = fmaxf(mf, val[e]);
    m = static_cast<double>(warp_fmax(mf));
    z = 0.0;
    for (int e = lane; e < p.E; e += 32) z += exp64(static_cast<double>(val[e]) - m);
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(FULL_MASK, z, o);
  }
  const int e = lane < n ? my_e : 0;
  const double l = static_cast<double>(val[e]);
  const double x = exp64(p.sigmoid ? -l : l - m);
  const double c = (p.sigmoid ? 1.0 / (1.0 + x) : x / z) + static_cast<double>(__ldg(p.bias + e));
  int rank = 0;
  for (int j = 0; j < n; ++j) {
    const double o = __shfl_sync(FULL_MASK, c, j);
    const int oe = __shfl_sync(FULL_MASK, e, j);
    rank += (o > c || (o == c && oe < e)) ? 1 : 0;
  }
  __syncwarp();
  if (lane < n) list[rank] = e;
  __syncwarp();
  return lane < n ? list[lane] : -1;
}

template <int VPL>
__global__ void __launch_bounds__(RG_THREADS, 1)
route_groups_kernel(const RouterParams p, int32_t* __restrict__ topk_idx,
                    float* __restrict__ topk_w, int32_t* __restrict__ dest_row,
                    int32_t* __restrict__ chunk_cnt, int64_t nch, int32_t* __restrict__ counts,
                    int32_t* __restrict__ kept, int32_t* __restrict__ offsets,
                    int32_t* __restrict__ src_tok, int32_t* __restrict__ src_slot,
                    uint8_t* __restrict__ drop_mask, int* err) {
  griddep_wait();   // see common.cuh: dependent launches
  // per warp: room for 64-bit keys (the exact choice), the values that its groups are judged by,
  // and the logits
  extern __shared__ double s_dyn[];
  __shared__ int s_idx[RG_CHUNK][8];
  __shared__ uint32_t s_bits[256];
  __shared__ int s_off[257];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int warps = blockDim.x >> 5;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * RG_CHUNK + warp;
  const int E = p.E, k = p.k;
  double* s_dbl = s_dyn + warp * 32 * VPL;
  float* s_val = reinterpret_cast<float*>(s_dyn + warps * 32 * VPL) + warp * 64 * VPL;
  float* s_log = s_val + 32 * VPL;
  for (int e = threadIdx.x; e < E; e += blockDim.x) s_bits[e] = 0u;
  if (threadIdx.x < RG_CHUNK * 8) (&s_idx[0][0])[threadIdx.x] = -1;
  float v[VPL];
#pragma unroll
  for (int s = 0; s < VPL; ++s) {
    const int e = lane + 32 * s;
    v[s] = (t < p.T && e < E) ? p.logits[t * E + e] : -INFINITY;
  }
  __syncthreads();

  int my_e = -1;
  if (t < p.T) {
    bool redo = false;
    bool nan_here = false;
    float top = -F32_MAX, z = 0.0f;   // softmax over all experts: maximum and sum
#pragma unroll
    for (int s = 0; s < VPL; ++s) {
      if (v[s] != v[s]) {
        nan_here = true;
        v[s] = -INFINITY;
      }
      v[s] = fminf(v[s], F32_MAX);
      s_log[lane + 32 * s] = v[s];
      top = fmaxf(top, v[s]);
    }
    if (__any_sync(FULL_MASK, nan_here) && lane == 0) flag_error(err, MOE_DEVERR_NAN_LOGIT);
    const bool keyed = p.bias != nullptr;               // keys are scores + bias
    const bool scored = keyed || (p.G > 1 && p.top2);   // scores enter the choice
    float sc[VPL];
#pragma unroll
    for (int s = 0; s < VPL; ++s) sc[s] = 0.0f;
    if (!p.sigmoid && (scored || !p.renorm)) {
      top = warp_fmax(top);
#pragma unroll
      for (int s = 0; s < VPL; ++s) {
        // without renorm z also divides the weights, as in the gradient: expf
        sc[s] = p.renorm ? fast_exp(v[s] - top) : expf(v[s] - top);
        z += sc[s];
      }
      z = fmaxf(warp_sum(z), 1e-37f);
      const float inv = 1.0f / z;
#pragma unroll
      for (int s = 0; s < VPL; ++s) sc[s] *= inv;
    } else if (scored) {
#pragma unroll
      for (int s = 0; s < VPL; ++s) sc[s] = fast_rcp(1.0f + fast_exp(-v[s]));
    }
    SortedKeys<VPL> keys;
    float big = 0.0f;
#pragma unroll
    for (int s = 0; s < VPL; ++s) {
      const int e = lane + 32 * s;
      keys.key[s] = 0u;
      const bool live = v[s] > -INFINITY;
      const float c = keyed && e < E ? sc[s] + __ldg(p.bias + e) : sc[s];
      if (live) {
        keys.key[s] = key32(keyed ? c : v[s]);
        big = fmaxf(big, fabsf(c));
      }
      if (p.G > 1) s_val[e] = !live ? -INFINITY : scored ? c : v[s];
    }
    // Error bound of an fp32 key.  sigma = 1 / (1 + e^-x): the exponential is off by 2^-22 and by
    // its argument's rounding, |x| 2^-24, of which sigma (1 - sigma) <= 1/4 reaches the result
    // (x sigma (1 - sigma) < 0.23); the sum and the reciprocal by 0.75 * 2^-22 of it: below
    // 2^-22.  softmax: e^x is off by 2^-22 and |x| 2^-24 of itself, the sum of 256 terms by 13
    // roundings more, the quotient by two: below 2^-19.  Adding the bias rounds once more,
    // relative to the key.
    const float largest = scored ? warp_fmax(big) : 0.0f;
    const float tol = scored ? (p.sigmoid ? 0x1p-22f : 0x1p-19f) + 0x1p-24f * largest : 0.0f;
    if (p.G > 1) {
      __syncwarp();
      float margin;
      const uint32_t mask = choose_groups(group_worth(s_val, p, lane), p, lane, margin);
      // On either side two keys, tol each, and the rounding of their sum, which is at most twice the
      // largest key: 2 * 2^-24 of that.  NaN: -inf on both.
      if (scored && margin <= 4.0f * tol + 0x1p-22f * largest) redo = true;
#pragma unroll
      for (int s = 0; s < VPL; ++s)
        if (lane + 32 * s < E && !((mask >> group_of(p, lane + 32 * s)) & 1u)) keys.key[s] = 0u;
    }
    keys.sort(lane);
    __syncwarp();
    // the k best, and with scores in the keys every further one that may belong to them: lane j
    // gets the j-th
    uint32_t last = 0u;
    int last_e = -1, found = 0;
    bool close = false;
    for (;; ++found) {
      if (found == (keyed ? 32 : k)) {
        redo |= keyed;   // more candidates than lanes
        break;
      }
      int e;
      const uint32_t got = keys.take(lane, e);
      if (got == 0u) break;
      if (keyed && found > 0) {
        // too close to tell, unless they are made of the same logit and the same bias
        const bool near = unkey32(last) - unkey32(got) <= 2.0f * tol;
        if (found >= k && !near) break;
        if (near && (s_log[e] != s_log[last_e] || __ldg(p.bias + e) != __ldg(p.bias + last_e)))
          close = true;
      }
      if (lane == found) my_e = e;
      last = got;
      last_e = e;
    }
    if (redo) my_e = choose_exact<VPL>(p, s_log, s_dbl, lane);
    else if (close) my_e = order_exact(p, s_log, reinterpret_cast<int*>(s_val), my_e, found, lane);
    if (lane >= k) my_e = -1;

    // weights of the chosen, one lane each
    const float my_l = my_e >= 0 ? s_log[my_e] : -INFINITY;
    const bool live = lane < k && my_e >= 0;
    float w = 0.0f;
    if (p.renorm) {
      // quotients of scores that may all underflow: divided by e^m first, m = min(0, the
      // largest chosen logit) for sigma (sigma(l) = e^l / (1 + e^l)), that logit for softmax
      const float lm = warp_fmax(live ? my_l : -F32_MAX);
      if (live) {
        if (!p.sigmoid) w = expf(my_l - lm);
        else if (lm >= 0.0f)
          w = my_l >= 0.0f ? 1.0f / (1.0f + expf(-my_l)) : expf(my_l) / (1.0f + expf(my_l));
        else
          w = expf(my_l - lm) / (1.0f + expf(my_l));
      }
      const float sum = warp_sum(w);
      if (live) w = p.scale * (w / sum);
    } else if (live) {
      w = p.scale * (p.sigmoid ? 1.0f / (1.0f + expf(-my_l)) : expf(my_l - top) / z);
    }
    if (lane < k) {
      topk_idx[t * k + lane] = my_e;
      topk_w[t * k + lane] = w;
      if (my_e < 0) dest_row[t * k + lane] = -1;
    }
  }
  if (t < p.T && lane < k) s_idx[warp][lane] = my_e;
  __syncthreads();

  // chunk histogram as per-expert token bit masks (OR is order-free: deterministic)
  const int tok = threadIdx.x >> 3, j = threadIdx.x & 7;
  int e = -1;
  if (threadIdx.x < RG_CHUNK * 8) {
    e = s_idx[tok][j];
    if (e >= 0) atomicOr(&s_bits[e], 1u << tok);
  }
  __syncthreads();
  const int rank = e >= 0 ? __popc(s_bits[e] & ((1u << tok) - 1u)) : -1;
  const int64_t slot = (static_cast<int64_t>(blockIdx.x) * RG_CHUNK + tok) * k + j;
  if (nch > 1) {
    if (e >= 0) dest_row[slot] = rank;
    for (int x = threadIdx.x; x < E; x += blockDim.x)
      chunk_cnt[static_cast<int64_t>(x) * nch + blockIdx.x] = __popc(s_bits[x]);
    griddep_launch();
    return;
  }
  // a single chunk: counts, offsets and the side arrays here (route.cu's scan and assign)
  if (warp == 0) {
    int sum = 0, kp[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int x = lane * 8 + i;
      const int c = x < E ? __popc(s_bits[x]) : 0;
      kp[i] = (p.cap > 0 && c > p.cap) ? p.cap : c;
      sum += kp[i];
      if (x < E) {
        counts[x] = c;
        kept[x] = kp[i];
      }
    }
    const int incl = warp_incl_scan(sum);
    int run = incl - sum;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int x = lane * 8 + i;
      if (x < E) {
        s_off[x] = run;
        offsets[x] = run;
      }
      run += kp[i];
    }
    if (lane == 31) {
      s_off[E] = incl;
      offsets[E] = incl;
    }
  }
  __syncthreads();
  if (threadIdx.x < RG_CHUNK * 8 && j < k && tok < p.T) {
    const bool stays = e >= 0 && (p.cap == 0 || rank < p.cap);
    const int d = stays ? s_off[e] + rank : -1;
    dest_row[slot] = d;
    drop_mask[slot] = stays ? 0 : 1;
    if (stays) {
      src_tok[d] = tok;
      src_slot[d] = static_cast<int32_t>(slot);
    }
  }
  for (int i = threadIdx.x; i < p.T * k; i += blockDim.x)
    if (i >= s_off[E]) {
      src_tok[i] = -1;
      src_slot[i] = -1;
    }
  griddep_launch();
}

// One warp per expert: its chunks' counts to their exclusive sums, its total and what is kept.
__global__ void __launch_bounds__(256)
order_count_kernel(int32_t* __restrict__ chunk_cnt, int64_t nch, int E, int cap,
                   int32_t* __restrict__ counts, int32_t* __restrict__ kept) {
  griddep_wait();   // see common.cuh: dependent launches
  const int lane = threadIdx.x & 31;
  const int e = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (e < E) {
    int32_t* col = chunk_cnt + static_cast<int64_t>(e) * nch;
    int running = 0;
    // 256 chunks at a time, the eight loads before any store
    for (int64_t base = 0; base < nch; base += 256) {
      int v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t c = base + 32 * i + lane;
        v[i] = c < nch ? col[c] : 0;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t c = base + 32 * i + lane;
        const int incl = warp_incl_scan(v[i]);
        if (c < nch) col[c] = running + incl - v[i];
        running += __shfl_sync(FULL_MASK, incl, 31);
      }
    }
    if (lane == 0) {
      counts[e] = running;
      kept[e] = cap > 0 && running > cap ? cap : running;
    }
  }
  griddep_launch();
}

// A thread per slot; every CTA sums the kept rows to the segments' offsets itself.
__global__ void __launch_bounds__(256)
order_assign_kernel(const int32_t* __restrict__ topk_idx, int64_t T, int k, int E, int cap,
                    const int32_t* __restrict__ chunk_base, int64_t nch,
                    const int32_t* __restrict__ kept, int32_t* __restrict__ offsets,
                    int32_t* __restrict__ dest_row, int32_t* __restrict__ src_tok,
                    int32_t* __restrict__ src_slot, uint8_t* __restrict__ drop_mask) {
  griddep_wait();   // see common.cuh: dependent launches
  __shared__ int s_off[257];
  __shared__ int s_sum[8];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + tid;
  const bool in = i < T * k;
  const int in_chunk = in ? dest_row[i] : -1;   // rank inside the chunk, or -1: not routed
  const int e = in ? topk_idx[i] : -1;
  const int n = tid < E ? kept[tid] : 0;
  const int base =
      in_chunk >= 0 ? chunk_base[static_cast<int64_t>(e) * nch + i / k / RG_CHUNK] : 0;
  const int incl = warp_incl_scan(n);
  if (lane == 31) s_sum[warp] = incl;
  __syncthreads();
  int before = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) before += w < warp ? s_sum[w] : 0;
  if (tid < E) s_off[tid] = before + incl - n;
  if (tid == E - 1) s_off[E] = before + incl;
  __syncthreads();
  if (blockIdx.x == 0)
    for (int x = tid; x <= E; x += 256) offsets[x] = s_off[x];
  if (in) {
    if (i >= s_off[E]) {
      src_tok[i] = -1;
      src_slot[i] = -1;
    }
    const int r = in_chunk < 0 ? -1 : base + in_chunk;
    const bool stays = r >= 0 && (cap == 0 || r < cap);
    const int d = stays ? s_off[e] + r : -1;
    dest_row[i] = d;
    drop_mask[i] = stays ? 0 : 1;
    if (stays) {
      src_tok[d] = static_cast<int32_t>(i / k);
      src_slot[d] = static_cast<int32_t>(i);
    }
  }
  griddep_launch();
}

// dlogits from dw, one warp per token.  With u the chosen experts' renormalised scores and
// dw the gradient of the weights:
//   renormalised:      dl_j = scale u_j sum_i u_i (dw_j - dw_i)  (times sigma(-l_j) for sigma)
//   sigma, as it is:   dl_j = scale dw_j sigma(l_j) sigma(-l_j)
//   softmax, as it is: dl_e = p_e (g_e - sum_i p_i g_i) for every expert, g = scale dw at the
//                      chosen ones and 0 elsewhere
// summed as differences, sum_i u_i (x_j - x_i), which keeps its precision when one score
// carries almost all the weight.  Bound by the T E * 4 bytes written (and read, in the dense
// form).
constexpr int RB_THREADS = 256;

template <int VPL>
__global__ void __launch_bounds__(RB_THREADS)
route_groups_bwd_kernel(const RouterParams p, const int32_t* __restrict__ topk_idx,
                        const float* __restrict__ dw, float* __restrict__ dlogits, int* err) {
  griddep_wait();   // see common.cuh: dependent launches
  const int lane = threadIdx.x & 31;
  const int64_t t = (static_cast<int64_t>(blockIdx.x) * RB_THREADS + threadIdx.x) >> 5;
  if (t >= p.T) return;
  const int E = p.E, k = p.k;
  const bool dense = !p.sigmoid && !p.renorm;
  const float* row = p.logits + t * E;
  int e = -1;
  float g = 0.0f;
  if (lane < k) {
    e = __ldg(topk_idx + t * k + lane);
    if (e >= E || e < -1) {
      flag_error(err, MOE_DEVERR_BAD_INDEX);
      e = -1;
    }
    if (e >= 0) g = p.scale * __ldg(dw + t * k + lane);
  }
  auto clean = [](float l) { return l != l ? -INFINITY : fminf(l, F32_MAX); };
  float v[VPL];
  float l = -INFINITY;
  float top = -F32_MAX, z = 1.0f, rest = 0.0f;
  if (dense) {
#pragma unroll
    for (int s = 0; s < VPL; ++s) {
      v[s] = lane + 32 * s < E ? clean(row[lane + 32 * s]) : -INFINITY;
      top = fmaxf(top, v[s]);
    }
    top = warp_fmax(top);
    if (e >= 0) l = clean(__ldg(row + e));
    // bit s: this lane's s-th expert is chosen
    uint32_t chosen = 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int ej = __shfl_sync(FULL_MASK, e, j);
      if ((ej & 31) == lane && ej >= 0) chosen |= 1u << (ej >> 5);
    }
    float zz = 0.0f;
#pragma unroll
    for (int s = 0; s < VPL; ++s) {
      v[s] = expf(v[s] - top);
      zz += v[s];
      if (!((chosen >> s) & 1u)) rest += v[s];
    }
    z = fmaxf(warp_sum(zz), 1e-37f);
    rest = warp_sum(rest) / z;
  } else if (e >= 0) {
    l = clean(__ldg(row + e));
  }
  // u: this lane's normalised score
  float u = 0.0f;
  const bool live = e >= 0 && l > -INFINITY;
  if (dense) {
    if (live) u = expf(l - top) / z;
  } else if (p.renorm) {
    const float lm = warp_fmax(live ? l : -F32_MAX);
    if (live) {
      if (!p.sigmoid) u = expf(l - lm);
      else if (lm >= 0.0f) u = l >= 0.0f ? 1.0f / (1.0f + expf(-l)) : expf(l) / (1.0f + expf(l));
      else u = expf(l - lm) / (1.0f + expf(l));
    }
    const float sum = warp_sum(u);
    if (live) u = u / sum;
  }
  float d = 0.0f, dot = 0.0f;
  if (!p.renorm && p.sigmoid) {
    if (live) d = g * (1.0f / (1.0f + expf(-l))) * (1.0f / (1.0f + expf(l)));
  } else {
    float acc = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float uj = __shfl_sync(FULL_MASK, u, j), gj = __shfl_sync(FULL_MASK, g, j);
      acc = fmaf(uj, g - gj, acc);
      dot = fmaf(uj, gj, dot);
    }
    if (dense) acc = fmaf(rest, g, acc);
    if (live) d = u * acc * (p.sigmoid ? 1.0f / (1.0f + expf(l)) : 1.0f);
  }
  // the whole row first, then the chosen experts' places
  const float each = dense ? -dot / z : 0.0f;
#pragma unroll
  for (int s = 0; s < VPL; ++s)
    if (lane + 32 * s < E) dlogits[t * E + lane + 32 * s] = dense ? v[s] * each : 0.0f;
  __syncwarp();
  if (e >= 0) dlogits[t * E + e] = d;
  griddep_launch();
}

RouterParams router_params(const moe_config_t* c, const moe_router_t* r, const float* logits) {
  RouterParams p;
  p.logits = logits;
  p.bias = r->bias;
  p.T = c->T;
  p.E = c->E;
  p.k = c->k;
  p.G = r->groups;
  p.per = c->E / r->groups;
  p.top_groups = r->top_groups;
  p.top2 = r->group_top == 2;
  p.sigmoid = r->score == MOE_SCORE_SIGMOID;
  p.renorm = r->renorm;
  p.cap = c->capacity;
  p.scale = c->route_scale;
  if (p.top_groups == p.G) p.G = 1;   // every group stays: nothing to choose
  p.per_magic = (65536 + p.per - 1) / p.per;
  p.lanes_log2 = 0;
  while ((2 << p.lanes_log2) * p.G <= 32 && (1 << p.lanes_log2) < p.per) ++p.lanes_log2;
  p.turns = (p.per + (1 << p.lanes_log2) - 1) >> p.lanes_log2;
  return p;
}

}  // namespace

cudaError_t launch_route_groups(const moe_config_t* c, const moe_router_t* r, const float* logits,
                                int32_t* topk_idx, float* topk_w, int32_t* counts, int32_t* kept,
                                int32_t* offsets, int32_t* dest_row, int32_t* src_tok,
                                int32_t* src_slot, uint8_t* drop_mask, void* scratch, int* err,
                                cudaStream_t st) {
  const RouterParams p = router_params(c, r, logits);
  const int64_t nch = route_chunks(c->T);
  int32_t* chunk_cnt = static_cast<int32_t*>(scratch);
  // a short single chunk: a warp per token, at least the 256 threads of its histogram
  const unsigned warps = nch > 1 ? 32u : static_cast<unsigned>(c->T < 8 ? 8 : c->T);
  const dim3 grid(static_cast<unsigned>(nch)), block(32 * warps);
  auto go = [&](auto kern, int vpl) {
    const size_t smem = static_cast<size_t>(warps) * 32 * vpl * 16;
    if (smem > 48 * 1024) {
      const cudaError_t a = cudaFuncSetAttribute(
          kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
      if (a != cudaSuccess) return a;
    }
    return launch_pdl(kern, grid, block, smem, st, 1, p, topk_idx, topk_w, dest_row, chunk_cnt, nch,
                      counts, kept, offsets, src_tok, src_slot, drop_mask, err);
  };
  cudaError_t e;
  if (c->E <= 32) e = go(route_groups_kernel<1>, 1);
  else if (c->E <= 64) e = go(route_groups_kernel<2>, 2);
  else if (c->E <= 128) e = go(route_groups_kernel<4>, 4);
  else e = go(route_groups_kernel<8>, 8);
  if (e != cudaSuccess || nch == 1) return e;
  e = launch_pdl(order_count_kernel, dim3(static_cast<unsigned>((c->E + 7) / 8)), dim3(256), 0, st,
                 1, chunk_cnt, nch, c->E, c->capacity, counts, kept);
  if (e != cudaSuccess) return e;
  return launch_pdl(order_assign_kernel, dim3(static_cast<unsigned>((c->T * c->k + 255) / 256)),
                    dim3(256), 0, st, 1, topk_idx, c->T, c->k, c->E, c->capacity, chunk_cnt, nch,
                    kept, offsets, dest_row, src_tok, src_slot, drop_mask);
}

cudaError_t launch_route_groups_bwd(const moe_config_t* c, const moe_router_t* r,
                                    const float* logits, const int32_t* topk_idx, const float* dw,
                                    float* dlogits, int* err, cudaStream_t st) {
  const RouterParams p = router_params(c, r, logits);
  const dim3 grid(static_cast<unsigned>((c->T + RB_THREADS / 32 - 1) / (RB_THREADS / 32)));
#define MOE_RB_LAUNCH(V)                                                                       \
  launch_pdl(route_groups_bwd_kernel<V>, grid, dim3(RB_THREADS), 0, st, 1, p, topk_idx, dw,     \
             dlogits, err)
  if (c->E <= 32) return MOE_RB_LAUNCH(1);
  if (c->E <= 64) return MOE_RB_LAUNCH(2);
  if (c->E <= 128) return MOE_RB_LAUNCH(4);
  return MOE_RB_LAUNCH(8);
#undef MOE_RB_LAUNCH
}

}  // namespace moe
