// Routing by scores (moe_route_scores), its gradient and the balance bias's
// step: softmax or sigmoid scores, a bias that only the choice sees, groups of
// experts, top-k, renormalised weights.
//
// One warp per token.  The choice is that of 64-bit arithmetic, in three steps of
// rising care.  Every expert's value is formed with the hardware's exponential
// and reciprocal together with a bound on its error, which gives an interval that
// holds the true value; the top_k-th largest lower end over the lanes is a
// threshold that every chosen expert's upper end reaches.  The few experts that
// reach it (a dozen for top_k = 8) go to a lane each and are formed again, to
// a few units in the last place, and ranked against one another.  Only where two
// neighbours of that order are nearer than their errors (once in some thousand
// tokens) are the candidates' values formed in 64 bits.  GB300 has two 64-bit
// lanes per SM and clock, so that forming all of them so would take a
// hundred times as long as reading them.
#include <math_constants.h>

#include "../../include/moe_block.h"
#include "router.cuh"
#include "train.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr uint32_t kAll = 0xffffffffu;

struct RouteParams {
  const void* logits;
  const float* bias;
  void* ids;
  float* weights;
  const int32_t* num_tokens;
  int64_t M, ld;
  int E, top_k, groups, topk_groups, group_size;
  int lanes;        // lanes per group, a power of two: lane = group * lanes + part
  int per;          // experts per lane
  int pair, score, renormalize, dtype, id_bits;
  float scale;
};

__device__ __forceinline__ float warp_max(float v) {   // NaN has no part
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// A logit as FP32 (exact).
__device__ __forceinline__ float logit_at(const void* p, int dtype, int64_t i) {
  if (dtype == MOE_TYPE_FP32) return __ldg(static_cast<const float*>(p) + i);
  const uint16_t b = __ldg(static_cast<const unsigned short*>(p) + i);
  if (dtype == MOE_TYPE_BF16) return __uint_as_float(static_cast<uint32_t>(b) << 16);
  return __half2float(__ushort_as_half(b));
}

// Unsigned keys in the order of the values; NaN above everything, -0 as 0.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return v != v ? 0xffffffffu : b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint64_t order_key(double v) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
  return v != v ? ~uint64_t(0) : b ^ (static_cast<uint64_t>(static_cast<int64_t>(b) >> 63) | (uint64_t(1) << 63));
}

__device__ __forceinline__ float sigmoid_precise(float l) {
  const float e = expf(-fabsf(l));
  return __fdiv_rn(l >= 0.f ? 1.f : e, 1.f + e);
}
__device__ __forceinline__ double sigmoid64(float l) {
  const double e = exp(-fabs(static_cast<double>(l)));
  return (l >= 0.f ? 1.0 : e) / (1.0 + e);
}

// The expert of this lane's i-th place, or -1.
__device__ __forceinline__ int expert_at(const RouteParams& p, int i, int lane) {
  const int off = lane % p.lanes + p.lanes * i, g = lane / p.lanes;
  return g < p.groups && off < p.group_size ? g * p.group_size + off : -1;
}

// What a token's selection leaves with lane j < n: its j-th expert and logit.
struct Chosen {
  int n, e;
  float l;
};

// exp(l - m) summed over the token's experts, in 64 bits.
__device__ __noinline__ double softmax_total(const RouteParams& p, int64_t t, double m) {
  double part = 0.0;
  for (int e = threadIdx.x % 32; e < p.E; e += 32) part += exp(static_cast<double>(logit_at(p.logits, p.dtype, t * p.ld + e)) - m);
  return warp_sum(part);
}

// The ranks of the n candidates (one a lane) in 64 bits.
template <int kMode>
__device__ __noinline__ int rank_exactly(const RouteParams& p, int64_t t, int n, int e, float l, float b, float m) {
  double v = static_cast<double>(b);
  if (kMode == 1)
    v += sigmoid64(l);
  else
    v += exp(static_cast<double>(l) - m) / softmax_total(p, t, m);
  const uint64_t key = order_key(v);
  int rank = 0;
  for (int j = 0; j < n; ++j) {
    const uint64_t other = __shfl_sync(kAll, key, j);
    const int oe = __shfl_sync(kAll, e, j);
    rank += other > key || (other == key && oe < e);
  }
  return rank;
}

// The two largest of a group, over its lanes (key 0: none).
struct TopTwo {
  uint64_t k1 = 0, k2 = 0;
  double a1 = 0.0, a2 = 0.0;
  __device__ __forceinline__ void take(double a) {
    const uint64_t k = order_key(a);
    if (k > k1) {
      k2 = k1, a2 = a1, k1 = k, a1 = a;
    } else if (k > k2) {
      k2 = k, a2 = a;
    }
  }
  __device__ __forceinline__ void merge(int lanes) {
    for (int o = 1; o < lanes; o <<= 1) {
      const uint64_t o1 = __shfl_xor_sync(kAll, k1, o), o2 = __shfl_xor_sync(kAll, k2, o);
      const double b1 = __shfl_xor_sync(kAll, a1, o), b2 = __shfl_xor_sync(kAll, a2, o);
      // (equal values count as two)
      if (o1 > k1) {
        if (o2 > k1) k2 = o2, a2 = b2; else k2 = k1, a2 = a1;
        k1 = o1, a1 = b1;
      } else if (o1 > k2) {
        k2 = o1, a2 = b1;
      }
    }
  }
};

// Whether this lane's group is among those that stay, from its two largest values.
__device__ __forceinline__ bool group_stays(const RouteParams& p, const TopTwo& top) {
  const int g = (threadIdx.x % 32) / p.lanes;
  const uint64_t key = top.k1 == 0 ? 0 : p.pair && top.k2 != 0 ? order_key(top.a1 + top.a2) : top.k1;
  int rank = 0;
  for (int j = 0; j < p.groups; ++j) {
    const uint64_t other = __shfl_sync(kAll, key, j * p.lanes);
    rank += other > key || (other == key && j < g);
  }
  return g < p.groups && rank < p.topk_groups;
}

// The groups in 64 bits, from the places `some` of this lane (the others cannot count).
template <int kMode>
__device__ __noinline__ bool groups_exactly(const RouteParams& p, int64_t t, uint64_t some, float m) {
  const int lane = threadIdx.x % 32;
  const double total = kMode == 2 ? softmax_total(p, t, m) : 1.0;
  TopTwo top;
  while (some) {
    const int e = expert_at(p, __ffsll(static_cast<long long>(some)) - 1, lane);
    some &= some - 1;
    const float l = logit_at(p.logits, p.dtype, t * p.ld + e);
    const double s = kMode == 1 ? sigmoid64(l) : exp(static_cast<double>(l) - m) / total;
    top.take(s + (p.bias ? static_cast<double>(__ldg(p.bias + e)) : 0.0));
  }
  __syncwarp();
  top.merge(p.lanes);
  return group_stays(p, top);
}

// Lane r gets the lane whose rank is r (ranks are distinct).
__device__ __forceinline__ int place(int16_t* at, int rank, int lane) {
  __syncwarp();
  at[rank & 31] = static_cast<int16_t>(lane);
  __syncwarp();
  return at[lane];
}

// Everything in 64 bits, for any values: a NaN, or many experts too near to tell apart.
// Every expert's key once, then groups, then top_k rounds of a warp-wide maximum.
__device__ __noinline__ Chosen choose_exactly(const RouteParams& p, int64_t t, int by_score) {
  const int lane = threadIdx.x % 32;
  const bool softmax = p.score == MOE_SCORE_SOFTMAX;
  double m = 0.0, total = 1.0;
  if (by_score && softmax) {
    float top = -CUDART_INF_F;
    for (int e = lane; e < p.E; e += 32) top = fmaxf(top, logit_at(p.logits, p.dtype, t * p.ld + e));
    m = static_cast<double>(warp_max(top));
    total = softmax_total(p, t, m);
  }
  uint64_t keys[64];                            // 0: left out (p.per <= 64)
  TopTwo top;
  for (int i = 0; i < p.per; ++i) {
    keys[i] = 0;
    const int e = expert_at(p, i, lane);
    if (e < 0) continue;
    const float l = logit_at(p.logits, p.dtype, t * p.ld + e), b = p.bias ? __ldg(p.bias + e) : 0.f;
    if (l == -CUDART_INF_F || b == -CUDART_INF_F) continue;
    double v = static_cast<double>(l);
    if (by_score) v = (softmax ? exp(v - m) / total : sigmoid64(l)) + static_cast<double>(b);
    top.take(v);
    // (without a bias experts go by their logits)
    keys[i] = order_key(p.bias ? v : static_cast<double>(l));
  }
  __syncwarp();
  bool kept = true;
  if (p.groups > 1) {
    top.merge(p.lanes);
    kept = group_stays(p, top);
  }
  Chosen c = {0, -1, 0.f};
  for (int j = 0; j < p.top_k; ++j) {
    uint64_t key = 0;
    int at = 0x7fffffff, place = -1;
    for (int i = 0; i < p.per && kept; ++i)
      if (keys[i] > key) key = keys[i], at = expert_at(p, i, lane), place = i;
    const uint64_t own = key;
    const int mine = at;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const uint64_t ok = __shfl_xor_sync(kAll, key, o);
      const int oa = __shfl_xor_sync(kAll, at, o);
      if (ok > key || (ok == key && oa < at)) key = ok, at = oa;
    }
    if (key == 0) break;                        // none left
    if (own == key && mine == at) keys[place] = 0;
    if (lane == j) {
      c.e = at;
      c.l = logit_at(p.logits, p.dtype, t * p.ld + at);
    }
    c.n = j + 1;
  }
  return c;
}

// The careful value of an expert's choice: FP32, within `err` of the true one.
template <int kMode>
__device__ __forceinline__ float careful_value(const RouteParams& p, bool biased, float l, float b, float m, float total,
                                               float& err) {
  err = 0.f;
  if (kMode == 0 || !biased) return l;
  // in units of 2^-23 of the score: the sigmoid's exponential, sum and divide; for softmax the
  // exponential, |x| / 2 for the rounding of x = l - m, the divide and the total's own
  // (an average of 3 and half a unit for each of its additions)
  const float x = l - m;
  const float s = kMode == 1 ? sigmoid_precise(l) : __fdiv_rn(expf(x), total);
  const float rel = kMode == 1 ? 4.f : fmaf(fabsf(x), 0.5f, 9.f + 0.5f * static_cast<float>(p.per));
  const float v = s + b;
  err = fmaf(fabsf(v), 0x1p-23f, fmaf(s, rel * 0x1p-23f, 0x1p-120f));
  return v;
}

// The choice where more experts reach the threshold than a warp has lanes (many
// equal logits, as of a router's first step): top_k rounds of a warp-wide maximum over
// the careful values.  n = -1: two of them are too near to tell.
template <int kMode>
__device__ __noinline__ Chosen choose_of_many(const RouteParams& p, int64_t t, bool kept, float m, float total) {
  const int lane = threadIdx.x % 32;
  const bool biased = kMode != 0 && p.bias != nullptr;
  Chosen c = {0, -1, 0.f};
  float cv = 0.f, cb = 0.f, worst_err = 0.f;
  uint64_t last = ~uint64_t(0);
  auto at = [&](int i, int& e, float& l, float& b, float& v, float& err) {
    e = kept ? expert_at(p, i, lane) : -1;
    if (e < 0) return false;
    l = logit_at(p.logits, p.dtype, t * p.ld + e);
    b = biased ? __ldg(p.bias + e) : 0.f;
    if (l == -CUDART_INF_F || b == -CUDART_INF_F) return false;
    v = careful_value<kMode>(p, biased, l, b, m, total, err);
    return true;
  };
  int e;
  float l, b, v, err;
  for (int j = 0; j < p.top_k; ++j) {
    uint64_t best = 0;
    float bl = 0.f, bb = 0.f, bv = 0.f;
    for (int i = 0; i < p.per; ++i) {
      if (!at(i, e, l, b, v, err)) continue;
      worst_err = fmaxf(worst_err, err);
      const uint64_t key = (static_cast<uint64_t>(order_key(v)) << 32) | static_cast<uint32_t>(~e);
      if (key < last && key > best) best = key, bl = l, bb = b, bv = v;
    }
    const uint32_t hi = __reduce_max_sync(kAll, static_cast<uint32_t>(best >> 32));
    if (hi == 0) break;                           // none left (values' keys are above 0)
    const uint32_t lo = __reduce_max_sync(kAll, (best >> 32) == hi ? static_cast<uint32_t>(best) : 0u);
    const uint64_t won = (static_cast<uint64_t>(hi) << 32) | lo;
    const int owner = __ffs(static_cast<int>(__ballot_sync(kAll, best == won))) - 1;
    bl = __shfl_sync(kAll, bl, owner);
    bb = __shfl_sync(kAll, bb, owner);
    bv = __shfl_sync(kAll, bv, owner);
    last = won;
    if (lane == j) c.e = static_cast<int>(~lo), c.l = bl, cv = bv, cb = bb;
    c.n = j + 1;
  }
  if (!biased || c.n == 0) return c;
  const float near = 2.f * warp_max(worst_err);
  const float pv = __shfl_up_sync(kAll, cv, 1), pl = __shfl_up_sync(kAll, c.l, 1), pb = __shfl_up_sync(kAll, cb, 1);
  bool close = lane > 0 && lane < c.n && !(pv - cv > near) && !(pl == c.l && pb == cb);
  const float kv = __shfl_sync(kAll, cv, c.n - 1), kl = __shfl_sync(kAll, c.l, c.n - 1), kb = __shfl_sync(kAll, cb, c.n - 1);
  for (int i = 0; i < p.per; ++i)
    if (at(i, e, l, b, v, err)) {
      const uint64_t key = (static_cast<uint64_t>(order_key(v)) << 32) | static_cast<uint32_t>(~e);
      close |= key < last && !(kv - v > near) && !(l == kl && b == kb);
    }
  if (__any_sync(kAll, close)) c.n = -1;
  return c;
}

// Whether all of the token's experts have one logit and one bias: their values are then
// equal, whatever their error.
__device__ __noinline__ bool all_equal(const RouteParams& p, int64_t t) {
  const int lane = threadIdx.x % 32;
  const float l0 = logit_at(p.logits, p.dtype, t * p.ld), b0 = p.bias ? __ldg(p.bias) : 0.f;
  bool same = true;
  for (int e = lane; e < p.E; e += 32)
    same &= logit_at(p.logits, p.dtype, t * p.ld + e) == l0 && (p.bias ? __ldg(p.bias + e) : 0.f) == b0;
  return __all_sync(kAll, same);
}

// kMode: what the choice compares.  0: the logits; 1: sigmoid scores (and
// bias); 2: softmax scores (and bias).
template <int kPer, int kMode>
__global__ void __launch_bounds__(32 * kWarps) route_scores_kernel(const __grid_constant__ RouteParams p) {
  __shared__ uint64_t s_key[kWarps][32];
  __shared__ int16_t s_cand[kWarps][32];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int g = lane / p.lanes, part = lane % p.lanes;
  const int mine = g < p.groups ? (p.group_size - part + p.lanes - 1) / p.lanes : 0;   // experts of this lane
  const int64_t first = static_cast<int64_t>(g) * p.group_size + part;
  const int64_t live = p.num_tokens ? min(static_cast<int64_t>(max(*p.num_tokens, 0)), p.M) : p.M;
  const bool softmax = p.score == MOE_SCORE_SOFTMAX;
  const bool biased = kMode != 0 && p.bias != nullptr;
  // error of the coarse score, relative to it, in units of 2^-23: the fast exponential's
  // 2 + 1.173 |x|, the divide's 2 and the sum's half; for softmax |x| / 2 more from the
  // rounding of x = l - m, and the total's: half a unit for each of its kPer + 5 additions
  // and an average of its terms' own (exp(-x) (2 + 1.7 x) <= 3)
  constexpr float kUnit = 0x1p-23f;
  constexpr float kBase = (kMode == 1 ? 5.f : 9.f + kPer / 2) * kUnit, kSlope = (kMode == 1 ? 1.2f : 1.7f) * kUnit;

  constexpr bool kHold = kMode != 0 && kPer <= 16;   // the bias stays in registers
  float held[kHold ? kPer : 1];
  if (kHold) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) held[i] = biased && i < mine ? __ldg(p.bias + first + i * p.lanes) : 0.f;
  }

  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp; t < p.M;
       t += static_cast<int64_t>(gridDim.x) * kWarps) {
    Chosen c = {0, -1, 0.f};
    float m = 0.f, total = 1.f;
    if (t < live) {
      // hi: the upper end of each value's interval (-inf: left out), low: the largest lower end
      float hi[kPer];
      const int64_t at = t * p.ld + first;
      if (p.dtype == MOE_TYPE_FP32) {
        const float* src = static_cast<const float*>(p.logits) + at;
#pragma unroll
        for (int i = 0; i < kPer; ++i) hi[i] = i < mine ? __ldcs(src + i * p.lanes) : -CUDART_INF_F;
      } else {
        const unsigned short* src = static_cast<const unsigned short*>(p.logits) + at;
        const bool bf16 = p.dtype == MOE_TYPE_BF16;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const uint32_t b = i < mine ? __ldcs(src + i * p.lanes) : bf16 ? 0xff80u : 0xfc00u;
          hi[i] = bf16 ? __uint_as_float(b << 16) : __half2float(__ushort_as_half(static_cast<unsigned short>(b)));
        }
      }
      float low = -CUDART_INF_F;
      bool nan = false;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        low = fmaxf(low, hi[i]);
        nan |= hi[i] != hi[i];
      }
      if (softmax && (kMode == 2 || !p.renormalize)) {
        m = warp_max(low);
        float sum = 0.f;
        if (kMode == 0) {
#pragma unroll
          for (int i = 0; i < kPer; ++i) sum += __expf(hi[i] - m);
          total = warp_sum(sum);
        }
      }
      float a1 = low, a2 = -CUDART_INF_F, slack = 0.f;      // the group's two largest, and its largest error
      if (kMode != 0) {
        float inv = 1.f;
        if (kMode == 2) {
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < kPer; ++i) sum += __expf(hi[i] - m);
          total = warp_sum(sum);
          inv = __frcp_rn(total);
        }
        a1 = low = -CUDART_INF_F;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const float x = kMode == 1 ? hi[i] : hi[i] - m;
          const float s = kMode == 1 ? __fdividef(1.f, 1.f + __expf(-x)) : __expf(x) * inv;
          const float b = kHold ? held[kHold ? i : 0] : biased && i < mine ? __ldg(p.bias + first + i * p.lanes) : 0.f;
          const float v = s + b;
          const bool out = hi[i] == -CUDART_INF_F || b == -CUDART_INF_F;
          const float err = fmaf(fabsf(v), 0x1p-22f, fmaf(s, fmaf(fabsf(x), kSlope, kBase), 0x1p-120f));
          nan |= v != v && !out;
          hi[i] = out ? -CUDART_INF_F : v + err;
          low = fmaxf(low, out ? -CUDART_INF_F : v - err);
          if (p.groups > 1) {
            const float in = out ? -CUDART_INF_F : v;
            a2 = fmaxf(a2, fminf(a1, in));
            a1 = fmaxf(a1, in);
            slack = fmaxf(slack, out ? 0.f : err);
          }
        }
      }
      int way = __any_sync(kAll, nan) ? 2 : 0;              // 1: many candidates, 2: in 64 bits
      bool stays = true;                                    // this lane's group
      if (p.groups > 1 && way == 0) {
        for (int o = 1; o < p.lanes; o <<= 1) {
          const float b1 = __shfl_xor_sync(kAll, a1, o);
          if (kMode != 0) {
            const float b2 = __shfl_xor_sync(kAll, a2, o);
            a2 = fmaxf(fmaxf(a2, b2), fminf(a1, b1));
            slack = fmaxf(slack, __shfl_xor_sync(kAll, slack, o));
          }
          a1 = fmaxf(a1, b1);
        }
        const float v = kMode != 0 && p.pair && a2 != -CUDART_INF_F ? a1 + a2 : a1;
        const float err = kMode != 0 ? fmaf(fabsf(v), 0x1p-22f, p.pair ? 2.f * slack : slack) : 0.f;
        int rank = 0;
        for (int j = 0; j < p.groups; ++j) {
          const float other = __shfl_sync(kAll, v, j * p.lanes);
          rank += other > v || (other == v && j < g);
        }
        bool kept = g < p.groups && rank < p.topk_groups;
        if (kMode != 0) {
          // a group that stays and one that goes nearer than their errors (an infinite
          // value has an infinite error: its difference is NaN)
          const float worst = -warp_max(kept ? -(v - err) : -CUDART_INF_F);
          const float best = warp_max(!kept && g < p.groups && v != -CUDART_INF_F ? v + err : -CUDART_INF_F);
          if (best != -CUDART_INF_F && !(worst > best) && !all_equal(p, t)) {
            // the experts that may be among the two largest of their group, in 64 bits
            const float floor = (p.pair && a2 != -CUDART_INF_F ? a2 : a1) - slack;
            uint64_t some = 0;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
              if (hi[i] != -CUDART_INF_F && !(hi[i] < floor)) some |= uint64_t(1) << i;
            kept = groups_exactly<kMode>(p, t, some, m);
          }
        }
        stays = kept;
        if (!kept) {
          low = -CUDART_INF_F;
#pragma unroll
          for (int i = 0; i < kPer; ++i) hi[i] = -CUDART_INF_F;
        }
      }
      if (way == 0) {
        // the threshold: the top_k-th largest of the lanes' lower ends
        float cur = low, thr = -CUDART_INF_F;
        for (int j = 0; j < p.top_k; ++j) {
          thr = warp_max(cur);
          if (thr == -CUDART_INF_F) break;
          if (cur == thr) cur = -CUDART_INF_F;
        }
        uint64_t cand = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (hi[i] >= thr && hi[i] != -CUDART_INF_F) cand |= uint64_t(1) << i;
        int n = 0;
        __syncwarp();                                       // (the last token's reads of s_cand are done)
        for (uint32_t some = __ballot_sync(kAll, cand != 0); some; some = __ballot_sync(kAll, cand != 0)) {
          const int pos = n + __popc(some & ((1u << lane) - 1));
          if (cand) {
            const int i = __ffsll(static_cast<long long>(cand)) - 1;
            cand &= cand - 1;
            if (pos < 32) s_cand[warp][pos] = static_cast<int16_t>(first + i * p.lanes);
          }
          n += __popc(some);
          if (n > 32) break;
        }
        __syncwarp();
        if (n > 32) {
          way = 1;
        } else {
          const int e = lane < n ? s_cand[warp][lane] : 0;
          const bool here = lane < n && MOE_IN_BOUNDS(e >= 0 && e < p.E);
          const float l = here ? logit_at(p.logits, p.dtype, t * p.ld + e) : 0.f;
          const float b = here && biased ? __ldg(p.bias + e) : 0.f;
          float err;
          const float v = careful_value<kMode>(p, biased, l, b, m, total, err);
          if (!here) err = 0.f;
          // rank: how many are above (equal ones: of lower index)
          uint64_t key = (static_cast<uint64_t>(order_key(v)) << 32) | static_cast<uint32_t>(~e);
          s_key[warp][lane] = key;
          __syncwarp();
          int rank = 0;
          for (int j = 0; j < n; ++j) rank += s_key[warp][j] > key;
          if (!here) rank = lane;
          c.n = min(n, p.top_k);
          int src = place(s_cand[warp], rank, lane);
          c.e = __shfl_sync(kAll, e, src);
          c.l = __shfl_sync(kAll, l, src);
          if (biased) {
            const float sv = __shfl_sync(kAll, v, src), sb = __shfl_sync(kAll, b, src);
            const float near = 2.f * warp_max(err);
            // each chosen one against the next, and the last chosen against all behind it;
            // equal logits of equal biases are equal, whatever their error
            const int ref = lane < p.top_k ? lane - 1 : p.top_k - 1;
            const float rv = __shfl_sync(kAll, sv, max(ref, 0)), rl = __shfl_sync(kAll, c.l, max(ref, 0)),
                        rb = __shfl_sync(kAll, sb, max(ref, 0));
            const bool close = lane > 0 && lane < n && !(rv - sv > near) && !(rl == c.l && rb == sb);
            if (__any_sync(kAll, close)) {
              rank = rank_exactly<kMode>(p, t, n, e, l, b, m);
              src = place(s_cand[warp], here ? rank : lane, lane);
              c.e = __shfl_sync(kAll, e, src);
              c.l = __shfl_sync(kAll, l, src);
            }
          }
        }
      }
      if (way == 1) c = choose_of_many<kMode>(p, t, stays, m, total);
      if (way == 2 || c.n < 0) c = choose_exactly(p, t, kMode != 0);
    }

    // the weights, by the lanes that hold the chosen
    const bool here = lane < c.n;
    float w = 0.f;
    if (p.renormalize) {
      // scores over a common factor that cannot vanish: exp(top), where top is the
      // largest chosen logit (for a sigmoid the smaller of that and 0)
      float top = warp_max(here ? c.l : -CUDART_INF_F);
      if (softmax) {
        w = expf(c.l - top);
      } else {
        top = fminf(top, 0.f);
        w = c.l != c.l ? c.l : __fdiv_rn(expf(fminf(c.l, 0.f) - top), 1.f + expf(-fabsf(c.l)));
      }
      const float sum = warp_sum(here ? w : 0.f);
      w = __fdiv_rn(w, sum) * p.scale;
    } else {
      w = (softmax ? __fdiv_rn(expf(c.l - m), total) : sigmoid_precise(c.l)) * p.scale;
    }
    if (lane < p.top_k) {
      const int64_t o = t * p.top_k + lane;
      p.weights[o] = here ? w : 0.f;
      if (p.id_bits == 64)
        static_cast<int64_t*>(p.ids)[o] = here ? c.e : -1;
      else
        static_cast<int32_t*>(p.ids)[o] = here ? c.e : -1;
    }
  }
}

// The logits' gradient.  One warp per token: the chosen logits go to a lane each, the
// row is written in whole lines (zeros, or for plain softmax every expert's
// -s sum(dw s)), then the chosen places by their lanes, after a warp barrier.
struct RouteGradParams {
  const void* logits;
  const void* ids;
  const float* dweights;
  void* dlogits;
  const int32_t* num_tokens;
  int64_t M, ld, ldd;
  int E, top_k, score, renormalize, id_bits, vec;
  float scale;
};

template <typename T> struct Logit;
template <> struct Logit<float> {
  static constexpr int kDtype = MOE_TYPE_FP32;
  static __device__ __forceinline__ float round(float v) { return v; }
};
template <> struct Logit<__nv_bfloat16> {
  static constexpr int kDtype = MOE_TYPE_BF16;
  static __device__ __forceinline__ __nv_bfloat16 round(float v) { return __float2bfloat16_rn(v); }
};
template <> struct Logit<__half> {
  static constexpr int kDtype = MOE_TYPE_FP16;
  static __device__ __forceinline__ __half round(float v) { return __float2half_rn(v); }
};

// kPer: logits a lane of a dense row (softmax, not renormalised; 0: the others)
template <typename T, int kPer>
__global__ void __launch_bounds__(32 * kWarps) route_scores_backward_kernel(const __grid_constant__ RouteGradParams p) {
  constexpr int kDtype = Logit<T>::kDtype;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x % 32;
  const int64_t live = p.num_tokens ? min(static_cast<int64_t>(max(*p.num_tokens, 0)), p.M) : p.M;
  const bool softmax = p.score == MOE_SCORE_SOFTMAX;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32; t < p.M;
       t += static_cast<int64_t>(gridDim.x) * kWarps) {
    T* row = static_cast<T*>(p.dlogits) + t * p.ldd;
    int64_t e = -1;
    float l = 0.f, dw = 0.f;
    if (t < live && lane < p.top_k) {
      const int64_t o = t * p.top_k + lane;
      e = p.id_bits == 64 ? __ldg(static_cast<const long long*>(p.ids) + o) : __ldg(static_cast<const int32_t*>(p.ids) + o);
      dw = __ldg(p.dweights + o);
    }
    bool here = e >= 0 && e < p.E;
    if (here) {
      l = logit_at(p.logits, kDtype, t * p.ld + e);
      here = l != -CUDART_INF_F;
    }
    // an expert listed more than once counts by all of its terms: their sum and number
    const uint32_t same = __match_any_sync(kAll, here ? static_cast<int>(e) : -1 - lane);
    float sum_dw = dw, terms = 1.f;
    if (__any_sync(kAll, __popc(same) > 1)) {
      sum_dw = terms = 0.f;
      for (int j = 0; j < p.top_k; ++j) {
        const float x = __shfl_sync(kAll, dw, j);
        if ((same >> j) & 1) sum_dw += x, terms += 1.f;
      }
    }
    float own;                                      // the gradient at this lane's expert
    if (kPer == 0) {
      if (p.renormalize) {
        // scores over a common factor that cannot vanish, as in the forward pass
        float top = warp_max(here ? l : -CUDART_INF_F), x;
        if (softmax) {
          x = expf(l - top);
        } else {
          top = fminf(top, 0.f);
          x = l != l ? l : __fdiv_rn(expf(fminf(l, 0.f) - top), 1.f + expf(-fabsf(l)));
        }
        const float share = __fdiv_rn(x, warp_sum(here ? x : 0.f));
        const float mean = warp_sum(here ? dw * share : 0.f);
        own = p.scale * share * (sum_dw - terms * mean) * (softmax ? 1.f : sigmoid_precise(-l));
      } else {
        own = p.scale * sum_dw * sigmoid_precise(l) * sigmoid_precise(-l);
      }
      // zeros, 16 bytes a lane where the rows allow it
      if (p.vec) {
        constexpr int kVec = 16 / static_cast<int>(sizeof(T));
        for (int i = lane; i * kVec < p.E; i += 32) reinterpret_cast<uint4*>(row)[i] = make_uint4(0, 0, 0, 0);
      } else {
        for (int i = lane; i < p.E; i += 32) row[i] = Logit<T>::round(0.f);
      }
    } else {
      constexpr int kHeld = kPer == 0 ? 1 : kPer;
      float s[kHeld];
      float m = -CUDART_INF_F, sum = 0.f;
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        s[i] = t < live && lane + 32 * i < p.E ? logit_at(p.logits, kDtype, t * p.ld + lane + 32 * i) : -CUDART_INF_F;
        m = fmaxf(m, s[i]);
      }
      m = warp_max(m);
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        s[i] = s[i] == -CUDART_INF_F ? 0.f : expf(s[i] - m);     // (a row of -inf has no gradient)
        sum += s[i];
      }
      const float inv = __frcp_rn(warp_sum(sum));
      const float mine = expf(l - m) * inv;
      const float mean = warp_sum(here ? dw * mine : 0.f);
#pragma unroll
      for (int i = 0; i < kHeld; ++i)
        if (lane + 32 * i < p.E) row[lane + 32 * i] = Logit<T>::round(s[i] == 0.f ? 0.f : -p.scale * (s[i] * inv) * mean);
      own = p.scale * mine * (sum_dw - mean);
    }
    __syncwarp();
    if (here && (same & ((1u << lane) - 1)) == 0 && MOE_IN_BOUNDS(e >= 0 && e < p.E)) row[e] = Logit<T>::round(own);
    __syncwarp();
  }
}

// out[e] = bias[e] + rate sign(sum - E load[e]); one CTA.
__global__ void __launch_bounds__(1024)
    route_balance_kernel(const int32_t* __restrict__ load, const float* bias, float* out, int E, float rate) {
  __shared__ long long s_part[32];
  pdl_wait();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
  long long sum = 0;
  for (int e = threadIdx.x; e < E; e += blockDim.x) sum += load[e];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
  if (lane == 0) s_part[warp] = sum;
  __syncthreads();
  sum = lane < warps ? s_part[lane] : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    const long long mine = static_cast<long long>(load[e]) * E;
    out[e] = sum == mine ? bias[e] : sum > mine ? bias[e] + rate : bias[e] - rate;
  }
}

unsigned warp_grid(int64_t tokens, int sms) {
  const int64_t want = ceil_div(tokens, kWarps), most = static_cast<int64_t>(sms) * 32;
  return static_cast<unsigned>(want < 1 ? 1 : want > most ? most : want);
}

template <int kMode>
auto route_kernel_of(int per) {
  return per <= 2    ? route_scores_kernel<2, kMode>
         : per <= 4  ? route_scores_kernel<4, kMode>
         : per <= 8  ? route_scores_kernel<8, kMode>
         : per <= 10 ? route_scores_kernel<10, kMode>
         : per <= 16 ? route_scores_kernel<16, kMode>
         : per <= 32 ? route_scores_kernel<32, kMode>
                     : route_scores_kernel<64, kMode>;
}

template <typename T>
auto route_grad_kernel_of(bool dense, int per) {
  return !dense      ? route_scores_backward_kernel<T, 0>
         : per <= 2  ? route_scores_backward_kernel<T, 2>
         : per <= 4  ? route_scores_backward_kernel<T, 4>
         : per <= 10 ? route_scores_backward_kernel<T, 10>
         : per <= 16 ? route_scores_backward_kernel<T, 16>
                     : route_scores_backward_kernel<T, 64>;
}

// Checks that both directions share: types, sizes, choices.
moe_status check_route(int dtype, int id_bits, int score, int64_t M, int E, int top_k, int64_t ld, float scale) {
  if (!is_type(dtype) || (id_bits != 32 && id_bits != 64)) return MOE_ERR_DTYPE;
  if (!ok_routes(M, top_k < 1 ? 1 : top_k) || top_k < 1 || top_k > kRouteMaxTopK || E < 1 || E > kRouteMaxE || ld < E ||
      ld > kMostElements || (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) || !(scale - scale == 0.f))
    return MOE_ERR_SHAPE;
  return MOE_OK;
}

bool aligned_to(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes) == 0; }

}  // namespace
}  // namespace moe

extern "C" {

moe_status moe_route_scores(const moe_route_scores_args* a, moe_stream_t stream) {
  using namespace moe;
  if (!a) return MOE_ERR_NULL;
  const moe_status bad = check_route(a->dtype, a->id_bits, a->score, a->M, a->E, a->top_k, a->ldlogits, a->routed_scale);
  if (bad != MOE_OK) return bad;
  if (a->groups < 1 || a->groups > 32 || a->E % a->groups || a->topk_groups < 1 || a->topk_groups > a->groups ||
      (a->group_score != MOE_GROUP_MAX && a->group_score != MOE_GROUP_TOP2) || a->top_k > a->topk_groups * (a->E / a->groups))
    return MOE_ERR_SHAPE;
  if (a->M == 0) return MOE_OK;
  if (!a->logits || !a->topk_ids || !a->topk_weights) return MOE_ERR_NULL;
  const int eb = type_bytes(a->dtype), ib = a->id_bits / 8;
  if (!aligned_to(a->logits, eb) || !aligned_to(a->topk_ids, ib) || !aligned4(a->topk_weights, a->bias, a->num_tokens))
    return MOE_ERR_ALIGN;
  const int64_t routes = a->M * a->top_k, in = extent_bytes(a->M, a->ldlogits, a->E, eb);
  const struct { const void* p; int64_t n; } outs[] = {{a->topk_ids, routes * ib}, {a->topk_weights, routes * 4}},
      ins[] = {{a->logits, in}, {a->bias, a->bias ? a->E * int64_t(4) : 0}, {a->num_tokens, a->num_tokens ? 4 : 0}};
  if (overlap(outs[0].p, outs[0].n, outs[1].p, outs[1].n)) return MOE_ERR_SHAPE;
  for (const auto& o : outs)
    for (const auto& i : ins)
      if (overlap(o.p, o.n, i.p, i.n)) return MOE_ERR_SHAPE;
  DeviceInfo dev;
  if (current_device(&dev) != MOE_OK) return MOE_ERR_CUDA;
  const void* ptrs[] = {a->logits, a->bias, a->topk_ids, a->topk_weights, a->num_tokens};
  for (const void* p : ptrs)
    if (p && !on_device(p, dev.device)) return MOE_ERR_DEVICE;
  RouteParams p;
  p.logits = a->logits;
  p.bias = a->bias;
  p.ids = a->topk_ids;
  p.weights = a->topk_weights;
  p.num_tokens = a->num_tokens;
  p.M = a->M;
  p.ld = a->ldlogits;
  p.E = a->E;
  p.top_k = a->top_k;
  // (all groups staying is no grouping)
  p.groups = a->topk_groups == a->groups ? 1 : a->groups;
  p.topk_groups = p.groups == 1 ? 1 : a->topk_groups;
  p.group_size = a->E / p.groups;
  p.lanes = 32;
  while (p.lanes * p.groups > 32) p.lanes /= 2;
  p.per = static_cast<int>(ceil_div(p.group_size, p.lanes));
  p.pair = a->group_score == MOE_GROUP_TOP2;
  p.score = a->score;
  p.renormalize = a->renormalize;
  p.dtype = a->dtype;
  p.id_bits = a->id_bits;
  p.scale = a->routed_scale;
  // without a bias the scores' order is the logits'; sums of two scores have none such
  const bool scored = a->bias || (p.groups > 1 && p.pair);
  auto kernel = !scored                          ? route_kernel_of<0>(p.per)
                : a->score == MOE_SCORE_SIGMOID ? route_kernel_of<1>(p.per)
                                                : route_kernel_of<2>(p.per);
  MOE_CUDA_TRY(launch_pdl(kernel, dim3(warp_grid(a->M, dev.sms)), dim3(32 * kWarps), 0, stream, 1, p));
  return MOE_OK;
}

moe_status moe_route_scores_backward(const moe_route_scores_backward_args* a, moe_stream_t stream) {
  using namespace moe;
  if (!a) return MOE_ERR_NULL;
  const moe_status bad = check_route(a->dtype, a->id_bits, a->score, a->M, a->E, a->top_k, a->ldlogits, a->routed_scale);
  if (bad != MOE_OK) return bad;
  if (a->lddlogits < a->E || a->lddlogits > kMostElements) return MOE_ERR_SHAPE;
  if (a->M == 0) return MOE_OK;
  if (!a->logits || !a->topk_ids || !a->dweights || !a->dlogits) return MOE_ERR_NULL;
  const int eb = type_bytes(a->dtype), ib = a->id_bits / 8;
  if (!aligned_to(a->logits, eb) || !aligned_to(a->dlogits, eb) || !aligned_to(a->topk_ids, ib) ||
      !aligned4(a->dweights, a->num_tokens))
    return MOE_ERR_ALIGN;
  const Rows in{a->logits, a->M, a->ldlogits, a->E}, out{a->dlogits, a->M, a->lddlogits, a->E};
  const bool in_place = a->dlogits == a->logits && (a->M == 1 || a->lddlogits == a->ldlogits);
  const int64_t routes = a->M * a->top_k, n = extent_bytes(a->M, a->lddlogits, a->E, eb);
  if ((!in_place && overlap(out, in, eb)) || overlap(a->dlogits, n, a->topk_ids, routes * ib) ||
      overlap(a->dlogits, n, a->dweights, routes * 4) || overlap(a->dlogits, n, a->num_tokens, a->num_tokens ? 4 : 0))
    return MOE_ERR_SHAPE;
  DeviceInfo dev;
  if (current_device(&dev) != MOE_OK) return MOE_ERR_CUDA;
  const void* ptrs[] = {a->logits, a->topk_ids, a->dweights, a->dlogits, a->num_tokens};
  for (const void* p : ptrs)
    if (p && !on_device(p, dev.device)) return MOE_ERR_DEVICE;
  RouteGradParams p;
  p.logits = a->logits;
  p.ids = a->topk_ids;
  p.dweights = a->dweights;
  p.dlogits = a->dlogits;
  p.num_tokens = a->num_tokens;
  p.M = a->M;
  p.ld = a->ldlogits;
  p.ldd = a->lddlogits;
  p.E = a->E;
  p.top_k = a->top_k;
  p.score = a->score;
  p.renormalize = a->renormalize;
  p.id_bits = a->id_bits;
  p.scale = a->routed_scale;
  p.vec = aligned16(a->dlogits) && a->lddlogits * eb % 16 == 0 && a->E * eb % 16 == 0;
  const bool dense = a->score == MOE_SCORE_SOFTMAX && !a->renormalize;
  const int per = static_cast<int>(ceil_div(a->E, 32));
  auto kernel = a->dtype == MOE_TYPE_BF16   ? route_grad_kernel_of<__nv_bfloat16>(dense, per)
                : a->dtype == MOE_TYPE_FP16 ? route_grad_kernel_of<__half>(dense, per)
                                            : route_grad_kernel_of<float>(dense, per);
  MOE_CUDA_TRY(launch_pdl(kernel, dim3(warp_grid(a->M, dev.sms)), dim3(32 * kWarps), 0, stream, 1, p));
  return MOE_OK;
}

moe_status moe_route_balance(const int32_t* load, const float* bias, float* out, int E, float rate, moe_stream_t stream) {
  using namespace moe;
  if (E < 1 || E > kRouteMaxE || !(rate - rate == 0.f)) return MOE_ERR_SHAPE;
  if (!load || !bias || !out) return MOE_ERR_NULL;
  if (!aligned4(load, bias, out)) return MOE_ERR_ALIGN;
  const int64_t n = int64_t(4) * E;
  if (overlap(out, n, load, n) || (out != bias && overlap(out, n, bias, n))) return MOE_ERR_SHAPE;
  DeviceInfo dev;
  if (current_device(&dev) != MOE_OK) return MOE_ERR_CUDA;
  if (!on_device(load, dev.device) || !on_device(bias, dev.device) || !on_device(out, dev.device)) return MOE_ERR_DEVICE;
  const unsigned threads = static_cast<unsigned>(round_up(E < 1024 ? E : 1024, 32));
  MOE_CUDA_TRY(launch_pdl(route_balance_kernel, dim3(1), dim3(threads), 0, stream, 1, load, bias, out, E, rate));
  return MOE_OK;
}

}  // extern "C"

MOE_BOUNDS_TU()
