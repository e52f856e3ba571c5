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
// from them, and checks that every decision it made had a margin above the keys' error bound;
// a token without that margin (measured: 0.1 - 0.3 % of tokens with 256 sigmoid scores) is
// chosen again from 64-bit keys.
//
// One warp per token, one CTA per 32-token chunk (32 warps).  The choice is k rounds of a
// warp maximum (redux.sync on order-preserving 32-bit keys, then on the id among equals).
// The chunk's histogram and the ranks inside it are bit masks as in route.cu, whose scan
// and assign kernels follow; a single chunk (T <= 32) does their work itself, in one
// launch.
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

__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(FULL_MASK, v); }
__device__ __forceinline__ unsigned long long warp_max(unsigned long long v) {
  const uint32_t hi = static_cast<uint32_t>(v >> 32);
  const uint32_t top = __reduce_max_sync(FULL_MASK, hi);
  const uint32_t lo = hi == top ? static_cast<uint32_t>(v) : 0u;
  return (static_cast<unsigned long long>(top) << 32) | __reduce_max_sync(FULL_MASK, lo);
}
__device__ __forceinline__ float warp_fmax(float v) {
  return unkey32(__reduce_max_sync(FULL_MASK, key32(v)));
}

// the best key left in the warp (0: none) and its expert (the lowest id among equals);
// the winner is taken out of its lane's keys
template <int VPL, typename K>
__device__ __forceinline__ K take_best(K* key, int lane, int& e) {
  K mine = key[0];
#pragma unroll
  for (int s = 1; s < VPL; ++s) mine = key[s] > mine ? key[s] : mine;
  const K top = warp_max(mine);
  if (top == 0) {
    e = -1;
    return top;
  }
  uint32_t id = 0xffffffffu;
#pragma unroll
  for (int s = VPL - 1; s >= 0; --s)
    if (key[s] == top) id = lane + 32 * s;
  id = __reduce_min_sync(FULL_MASK, id);
#pragma unroll
  for (int s = 0; s < VPL; ++s)
    if (id == static_cast<uint32_t>(lane + 32 * s)) key[s] = 0;
  e = static_cast<int>(id);
  return top;
}

// Worth of every group: lane g * L + sub scans part of group g's values (staged in shared
// memory) and the L lanes of a group are joined.  The scan starts at a place that depends on
// g, so that the groups of one step read different banks.  -inf: nothing in service.
template <typename F>
__device__ __forceinline__ F group_worth(const F* val, int G, int per, int top2, int lane, int& g,
                                         int& L) {
  L = 1;
  while (2 * L * G <= 32 && L < per) L *= 2;
  g = lane / L;
  const int sub = lane - g * L;
  const F none = -static_cast<F>(INFINITY);
  F m1 = none, m2 = none;
  if (g < G) {
    const int nj = (per + L - 1) / L;
    int j = g % nj;
    for (int n = 0; n < nj; ++n) {
      const int i = sub + L * j;
      if (i < per) {
        const F v = val[g * per + i];
        if (v > m1) {
          m2 = m1;
          m1 = v;
        } else if (v > m2) {
          m2 = v;
        }
      }
      if (++j == nj) j = 0;
    }
  }
  for (int o = 1; o < L; o <<= 1) {
    const F a = __shfl_xor_sync(FULL_MASK, m1, o), b = __shfl_xor_sync(FULL_MASK, m2, o);
    const F lo = a < m1 ? a : m1;
    m1 = a > m1 ? a : m1;
    m2 = b > m2 ? b : m2;
    m2 = lo > m2 ? lo : m2;
  }
  return (top2 && m2 != none) ? m1 + m2 : m1;
}

// Bit g set for each of the top_groups best groups; margin: the least worth that stays minus
// the best that goes (+inf where nothing goes).
template <typename F>
__device__ __forceinline__ uint32_t choose_groups(F worth, int g, int L, int G, int top_groups,
                                                  int lane, F& margin) {
  int rank = 0;
  for (int j = 0; j < G; ++j) {
    const F o = __shfl_sync(FULL_MASK, worth, j * L);
    rank += (o > worth || (o == worth && j < g)) ? 1 : 0;
  }
  const bool head = g < G && lane == g * L;
  const bool in = head && rank < top_groups;
  F lo = in ? worth : static_cast<F>(INFINITY);
  F hi = (head && !in) ? worth : -static_cast<F>(INFINITY);
  for (int o = 16; o > 0; o >>= 1) {
    const F a = __shfl_xor_sync(FULL_MASK, lo, o), b = __shfl_xor_sync(FULL_MASK, hi, o);
    lo = a < lo ? a : lo;
    hi = b > hi ? b : hi;
  }
  margin = hi == -static_cast<F>(INFINITY) ? static_cast<F>(INFINITY) : lo - hi;
  uint32_t mask = 0u;
  const uint32_t heads = __ballot_sync(FULL_MASK, in);
  for (int j = 0; j < G; ++j) mask |= ((heads >> (j * L)) & 1u) << j;
  return mask;
}

struct RouterParams {
  const float* logits;
  const float* bias;
  int64_t T;
  int E, k, G, per, top_groups, top2, sigmoid, renorm, cap;
  float scale;
};

// The choice from 64-bit keys.  val: the token's logits (NaN already -inf), wide: room for as
// many doubles, both this warp's own.  Lane j gets the j-th choice.
template <int VPL>
__device__ __noinline__ int choose_exact(const RouterParams p, const float* val, double* wide,
                                         int lane) {
  double m = 0.0, z = 0.0;
  if (!p.sigmoid) {
    float mf = -F32_MAX;
#pragma unroll 1
    for (int e = lane; e < p.E; e += 32) mf = fmaxf(mf, val[e]);
    m = static_cast<double>(warp_fmax(mf));
  }
#pragma unroll 1
  for (int e = lane; e < p.E; e += 32) {
    const double l = static_cast<double>(val[e]);
    wide[e] = p.sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - m);
    z += wide[e];
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
    double c = p.sigmoid ? wide[e] : wide[e] / z;
    if (p.bias) c += static_cast<double>(__ldg(p.bias + e));
    // without a bias the experts' own order is that of the logits
    if (live) key[s] = key64(p.bias ? c : l);
    wide[e] = !live ? -INFINITY : (!p.bias && !p.top2) ? l : c;
  }
  if (p.G > 1) {
    __syncwarp();
    int g, L;
    const double worth = group_worth(wide, p.G, p.per, p.top2, lane, g, L);
    double margin;
    const uint32_t mask = choose_groups(worth, g, L, p.G, p.top_groups, lane, margin);
#pragma unroll
    for (int s = 0; s < VPL; ++s)
      if (lane + 32 * s < p.E && !((mask >> ((lane + 32 * s) / p.per)) & 1u)) key[s] = 0ull;
  }
  int sel = -1;
  for (int j = 0; j < p.k; ++j) {
    int e;
    take_best<VPL>(key, lane, e);
    if (lane == j) sel = e;
  }
  return sel;
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
  // per warp: room for 64-bit keys (the exact choice), and the fp32 values that its groups are
  // judged by
  extern __shared__ double s_dyn[];
  __shared__ int s_idx[RG_CHUNK][8];
  __shared__ uint32_t s_bits[256];
  __shared__ int s_off[257];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * RG_CHUNK + warp;
  const int E = p.E, k = p.k;
  double* s_dbl = s_dyn + warp * 32 * VPL;
  float* s_val = reinterpret_cast<float*>(s_dyn + RG_CHUNK * 32 * VPL) + warp * 32 * VPL;
  for (int e = threadIdx.x; e < E; e += RG_THREADS) s_bits[e] = 0u;
  float v[VPL];
#pragma unroll
  for (int s = 0; s < VPL; ++s) {
    const int e = lane + 32 * s;
    v[s] = (t < p.T && e < E) ? p.logits[t * E + e] : -INFINITY;
  }
  __syncthreads();

  int my_e = -1;
  bool redo = false;
  float top = -F32_MAX, z = 0.0f;   // softmax over all experts: maximum and sum
  if (t < p.T) {
    bool nan_here = false;
    float top_here = -F32_MAX;
#pragma unroll
    for (int s = 0; s < VPL; ++s) {
      if (v[s] != v[s]) {
        nan_here = true;
        v[s] = -INFINITY;
      }
      v[s] = fminf(v[s], F32_MAX);
      top_here = fmaxf(top_here, v[s]);
    }
    if (__any_sync(FULL_MASK, nan_here) && lane == 0) flag_error(err, MOE_DEVERR_NAN_LOGIT);
    const bool keyed = p.bias != nullptr;               // keys are scores + bias
    const bool scored = keyed || (p.G > 1 && p.top2);   // scores enter the choice
    float sc[VPL];
#pragma unroll
    for (int s = 0; s < VPL; ++s) sc[s] = 0.0f;
    if (!p.sigmoid && (scored || !p.renorm)) {
      top = warp_fmax(top_here);
#pragma unroll
      for (int s = 0; s < VPL; ++s) {
        sc[s] = expf(v[s] - top);
        z += sc[s];
      }
      z = warp_sum(z);
      const float inv = 1.0f / fmaxf(z, 1e-37f);
#pragma unroll
      for (int s = 0; s < VPL; ++s) sc[s] *= inv;
    } else if (scored) {
#pragma unroll
      for (int s = 0; s < VPL; ++s) sc[s] = 1.0f / (1.0f + expf(-v[s]));
    }
    uint32_t key[VPL];
    float big = 0.0f;
#pragma unroll
    for (int s = 0; s < VPL; ++s) {
      const int e = lane + 32 * s;
      key[s] = 0u;
      const bool live = v[s] > -INFINITY;
      const float c = keyed && e < E ? sc[s] + __ldg(p.bias + e) : sc[s];
      if (live) {
        key[s] = key32(keyed ? c : v[s]);
        big = fmaxf(big, fabsf(c));
      }
      if (p.G > 1 && e < E) s_val[e] = !live ? -INFINITY : scored ? c : v[s];
    }
    // error bound of an fp32 key.  sigma: one ulp of expf and two roundings, below 2^-21 of a
    // score <= 1.  softmax: the argument's rounding |x| 2^-24 times e^x is below 2^-25, the
    // sum of 256 terms adds 13 roundings, the quotient two: below 2^-19.  Adding the bias
    // rounds once more, relative to the key.
    const float tol = scored ? (p.sigmoid ? 0x1p-21f : 0x1p-19f) + 0x1p-23f * warp_fmax(big) : 0.0f;
    if (p.G > 1) {
      __syncwarp();
      int g, L;
      const float worth = group_worth(s_val, p.G, p.per, p.top2, lane, g, L);
      float margin;
      const uint32_t mask = choose_groups(worth, g, L, p.G, p.top_groups, lane, margin);
      // two keys a group and the rounding of their sum, on both sides
      if (scored && !(margin > 5.0f * tol)) redo = true;
#pragma unroll
      for (int s = 0; s < VPL; ++s)
        if (lane + 32 * s < E && !((mask >> ((lane + 32 * s) / p.per)) & 1u)) key[s] = 0u;
    }
    uint32_t last = 0u;
    for (int j = 0; j < k; ++j) {
      int e;
      const uint32_t got = take_best<VPL>(key, lane, e);
      if (lane == j) my_e = e;
      if (keyed && j > 0 && got != 0u && !(unkey32(last) - unkey32(got) > 2.0f * tol)) redo = true;
      last = got;
    }
    if (keyed && last != 0u) {   // the first one left out
      int e;
      const uint32_t got = take_best<VPL>(key, lane, e);
      if (got != 0u && !(unkey32(last) - unkey32(got) > 2.0f * tol)) redo = true;
    }
    if (redo) {
      __syncwarp();
#pragma unroll
      for (int s = 0; s < VPL; ++s)
        if (lane + 32 * s < E) s_val[lane + 32 * s] = v[s];
      my_e = choose_exact<VPL>(p, s_val, s_dbl, lane);
    }

    // weights of the chosen, one lane each
    float my_l = -INFINITY;
    const int at = my_e < 0 ? 0 : my_e;
#pragma unroll
    for (int s = 0; s < VPL; ++s) {
      const float o = __shfl_sync(FULL_MASK, v[s], at & 31);
      if (s == (at >> 5)) my_l = o;
    }
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
  if (lane < 8) s_idx[warp][lane] = (t < p.T && lane < k) ? my_e : -1;
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
    for (int x = threadIdx.x; x < E; x += RG_THREADS)
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
  for (int i = threadIdx.x; i < p.T * k; i += RG_THREADS)
    if (i >= s_off[E]) {
      src_tok[i] = -1;
      src_slot[i] = -1;
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
    float zz = 0.0f;
#pragma unroll
    for (int s = 0; s < VPL; ++s) {
      bool chosen = false;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        chosen |= __shfl_sync(FULL_MASK, e, j) == lane + 32 * s;
      v[s] = expf(v[s] - top);
      zz += v[s];
      if (!chosen) rest += v[s];
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
#pragma unroll
  for (int s = 0; s < VPL; ++s) {
    const int x = lane + 32 * s;
    float val = dense ? -(v[s] / z) * dot : 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int ej = __shfl_sync(FULL_MASK, e, j);
      const float dj = __shfl_sync(FULL_MASK, d, j);
      if (ej == x) val = dj;
    }
    if (x < E) dlogits[t * E + x] = val;
  }
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
  const dim3 grid(static_cast<unsigned>(nch)), block(RG_THREADS);
#define MOE_RG_LAUNCH(V)                                                                       \
  (e = cudaFuncSetAttribute(route_groups_kernel<V>, cudaFuncAttributeMaxDynamicSharedMemorySize, \
                            RG_CHUNK * 32 * V * 12)) != cudaSuccess                             \
      ? e                                                                                       \
      : launch_pdl(route_groups_kernel<V>, grid, block, RG_CHUNK * 32 * V * 12, st, 1, p,       \
                   topk_idx, topk_w, dest_row, chunk_cnt, nch, counts, kept, offsets, src_tok,  \
                   src_slot, drop_mask, err)
  cudaError_t e;
  if (c->E <= 32) e = MOE_RG_LAUNCH(1);
  else if (c->E <= 64) e = MOE_RG_LAUNCH(2);
  else if (c->E <= 128) e = MOE_RG_LAUNCH(4);
  else e = MOE_RG_LAUNCH(8);
#undef MOE_RG_LAUNCH
  if (e != cudaSuccess || nch == 1) return e;
  return launch_route_order(c->T, c->E, c->k, c->capacity, topk_idx, chunk_cnt, counts, kept,
                            offsets, dest_row, src_tok, src_slot, drop_mask, st);
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
