// Routing by scores (moe_route_scores), its gradient and the balance bias's
// step: softmax or sigmoid scores, a bias that only the choice sees, groups of
// experts, top-k, renormalised weights.
//
// One warp per token.  The choice is that of 64-bit arithmetic, in steps of rising care.  Every
// expert's value is formed with the hardware's exponential and reciprocal, within a bound that
// holds for all of the token's.  The top_k-th largest of the lanes' two largest values, less
// two such errors, is a threshold that every chosen expert reaches.  The few experts that reach
// it (a dozen for top_k = 8) go to a lane each and are ranked against one another.  Only where
// two neighbours of that order, or a group that stays and one that goes, are nearer than their
// errors (a few tokens in a thousand) are the values in question formed in 64 bits.  GB300 has two
// 64-bit lanes per SM and clock: forming all of them so would take a hundred times as long as
// reading them.
//
// Without a bias the scores' order is the logits' own, which are compared as they are.
//
// Instructions bound it, and of those mostly the ones that a token costs whatever E is: 16-bit
// logits of 257 experts, top 9, take some 470 (65536 tokens: 29.5 us, 1.31 TB/s); sigmoid scores with
// a bias, 8 groups and top 10 of 512 experts some 1080 (8192 tokens: 11.2 to 12.2 us, by their near
// ties).  Two tokens finished side by side by half a warp each (10% fewer instructions, fewer warps) and warps that stay
// for many tokens (40 us) were slower.  The 64 bits count where a token is among the last ones: of
// 8192, two or three have groups too near to tell, which cost 2 us until only the groups in
// question were formed so.
#include <math_constants.h>

#include <type_traits>

#include "../../include/moe_block.h"
#include "route_layout.h"
#include "router.cuh"
#include "train.cuh"

namespace moe {
namespace {

// Warps of a CTA.  Where scores are compared a warp has one token, and small CTAs fill the places that
// finished ones leave (8192 tokens of 512 experts in groups: 12.0 us, 12.3 with eight warps); where logits
// are, a warp takes several of many tokens (65536 tokens of 257 experts: 3% less than with four).
constexpr int kWarps = 8, kWarpsScored = 4;
constexpr uint32_t kAll = 0xffffffffu;

struct RouteParams : RouteLayout {
  const void* logits;
  const float* bias;
  void* ids;
  float* weights;
  const int32_t* num_tokens;
  int64_t M, ld;
  int top_k, topk_groups;
  int pair, score, renormalize, dtype, id_bits;
  float scale;
  float softmax_units;
};

__device__ __forceinline__ float warp_max(float v) {   // NaN has no part
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));   // (all lanes: it may not move into a branch)
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

// Places of a lane as a mask, its lowest one, and how many the careful paths hold beside a kernel of kPer.
template <int kPer>
using PlaceMask = std::conditional_t<(kPer > 64), unsigned __int128, std::conditional_t<(kPer > 32), uint64_t, uint32_t>>;
__device__ __forceinline__ int first_place(uint32_t m) { return __ffs(static_cast<int>(m)) - 1; }
__device__ __forceinline__ int first_place(uint64_t m) { return __ffsll(static_cast<long long>(m)) - 1; }
__device__ __forceinline__ int first_place(unsigned __int128 m) {
  const uint64_t low = static_cast<uint64_t>(m);
  return low ? first_place(low) : 64 + first_place(static_cast<uint64_t>(m >> 64));
}
template <int kPer>
constexpr int kMostPlaces = kPer > 64 ? 128 : 64;

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

// Whether this lane's group is among the `slots` best of those in question, from its two largest values.
__device__ __forceinline__ bool group_stays(const RouteParams& p, const TopTwo& top, bool in_question, int slots) {
  const int g = (threadIdx.x % 32) / p.lanes;
  const uint64_t key = top.k1 == 0 ? 0 : p.pair && top.k2 != 0 ? order_key(top.a1 + top.a2) : top.k1;
  const uint32_t some = __ballot_sync(kAll, in_question);
  int rank = 0;
  for (int j = 0; j < p.groups; ++j) {
    if (!((some >> (j * p.lanes)) & 1)) continue;
    const uint64_t other = __shfl_sync(kAll, key, j * p.lanes);
    rank += other > key || (other == key && j < g);
  }
  return in_question && rank < slots;
}

// The groups in question in 64 bits, from the places `some` of this lane (the others cannot count).
template <int kMode, typename Mask>
__device__ __noinline__ bool groups_exactly(const RouteParams& p, int64_t t, Mask some, float m, bool in_question, int slots) {
  const int lane = threadIdx.x % 32;
  const double total = kMode == 2 ? softmax_total(p, t, m) : 1.0;
  TopTwo top;
  while (some) {
    const int e = route_expert_at(p, first_place(some), lane);
    some &= some - 1;
    const float l = logit_at(p.logits, p.dtype, t * p.ld + e);
    const double s = kMode == 1 ? sigmoid64(l) : exp(static_cast<double>(l) - m) / total;
    top.take(s + (p.bias ? static_cast<double>(__ldg(p.bias + e)) : 0.0));
  }
  __syncwarp();
  top.merge(p.lanes);
  return group_stays(p, top, in_question, slots);
}

// The lane whose rank is this lane's number (ranks are distinct).
__device__ __forceinline__ int place(int16_t* at, int rank, int lane) {
  __syncwarp();
  at[rank & 31] = static_cast<int16_t>(lane);
  __syncwarp();
  return at[lane];
}

// Everything in 64 bits, for any values: a NaN, or many experts too near to tell apart.
// Every expert's key once, then groups, then top_k rounds of a warp-wide maximum.
template <int kMost>
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
  uint64_t keys[kMost];                         // 0: left out
  TopTwo top;
#pragma unroll 4
  for (int i = 0; i < p.per && MOE_IN_BOUNDS(i < kMost); ++i) {
    const int e = route_expert_at(p, i, lane);
    const float l = e >= 0 ? logit_at(p.logits, p.dtype, t * p.ld + e) : -CUDART_INF_F, b = e >= 0 && p.bias ? __ldg(p.bias + e) : 0.f;
    double v = static_cast<double>(l);
    if (by_score) v = (softmax ? exp(v - m) / total : sigmoid64(l)) + static_cast<double>(b);
    const bool in = l != -CUDART_INF_F && b != -CUDART_INF_F;
    if (in) top.take(v);
    // (without a bias experts go by their logits)
    keys[i] = in ? order_key(p.bias ? v : static_cast<double>(l)) : 0;
  }
  __syncwarp();
  bool kept = true;
  if (p.groups > 1) {
    top.merge(p.lanes);
    kept = group_stays(p, top, lane / p.lanes < p.groups, p.topk_groups);
  }
  Chosen c = {0, -1, 0.f};
  for (int j = 0; j < p.top_k; ++j) {
    uint64_t key = 0;
    int at = 0x7fffffff, place = -1;
    for (int i = 0; i < p.per && kept; ++i)
      if (keys[i] > key) key = keys[i], at = route_expert_at(p, i, lane), place = i;
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

// exp(x) by the hardware: 2 + 1.173 |x| units in the last place, 0 below 2^-126.
__device__ __forceinline__ float exp_coarse(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
  return r;
}
// 1 / x to a unit in the last place (0 for x beyond 2^126).
__device__ __forceinline__ float reciprocal_coarse(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// What the choice compares, to the error that the kernel states for it.
template <int kMode>
__device__ __forceinline__ float coarse_value(float l, float b, float m, float inv) {
  if (kMode == 0) return l;
  return (kMode == 1 ? reciprocal_coarse(1.f + exp_coarse(-l)) : exp_coarse(l - m) * inv) + b;
}

// The choice where more experts reach the threshold than a warp has lanes (many
// equal logits, as of a router's first step): top_k rounds of a warp-wide maximum.
// n = -1: two of them are too near to tell.
template <int kMode, int kMost>
__device__ __noinline__ Chosen choose_of_many(const RouteParams& p, int64_t t, bool kept, float m, float inv, float err) {
  const int lane = threadIdx.x % 32;
  const bool by_value = kMode != 0 && p.bias;          // without a bias experts go by their logits
  Chosen c = {0, -1, 0.f};
  using Mask = PlaceMask<kMost>;
  float values[kMost];
  Mask taken = 0;                                      // places that are left out or chosen
#pragma unroll 4
  for (int i = 0; i < p.per && MOE_IN_BOUNDS(i < kMost); ++i) {
    const int e = kept ? route_expert_at(p, i, lane) : -1;
    const float l = e >= 0 ? logit_at(p.logits, p.dtype, t * p.ld + e) : -CUDART_INF_F, b = e >= 0 && by_value ? __ldg(p.bias + e) : 0.f;
    values[i] = by_value ? coarse_value<kMode>(l, b, m, inv) : l;
    if (l == -CUDART_INF_F || b == -CUDART_INF_F) taken |= Mask(1) << i;
  }
  float cv = 0.f, cb = 0.f;
  for (int j = 0; j < p.top_k; ++j) {
    float best = -CUDART_INF_F;
    int at = 0x7fffffff, place = 0;
    for (int i = 0; i < p.per; ++i)
      if (!((taken >> i) & 1) && (values[i] > best || at == 0x7fffffff)) best = values[i], place = i, at = route_expert_at(p, i, lane);
    const bool some = at != 0x7fffffff;
    const float top = warp_max(some ? best : -CUDART_INF_F);
    const int won = __reduce_min_sync(kAll, some && best == top ? at : 0x7fffffff);
    if (won == 0x7fffffff) break;                      // none left
    if (some && at == won) taken |= Mask(1) << place;
    if (lane == j) c.e = won, cv = top;
    c.n = j + 1;
  }
  if (lane < c.n) {
    c.l = logit_at(p.logits, p.dtype, t * p.ld + c.e);
    cb = by_value ? __ldg(p.bias + c.e) : 0.f;
  }
  __syncwarp();
  if (!by_value || c.n == 0) return c;
  const float near = 2.f * err;
  const float pv = __shfl_up_sync(kAll, cv, 1), pl = __shfl_up_sync(kAll, c.l, 1), pb = __shfl_up_sync(kAll, cb, 1);
  bool close = lane > 0 && lane < c.n && !(pv - cv > near) && !(pl == c.l && pb == cb);
  const float kv = __shfl_sync(kAll, cv, c.n - 1), kl = __shfl_sync(kAll, c.l, c.n - 1), kb = __shfl_sync(kAll, cb, c.n - 1);
  for (int i = 0; i < p.per; ++i)
    if (!((taken >> i) & 1) && !(kv - values[i] > near)) {
      const int e = route_expert_at(p, i, lane);
      close |= !(logit_at(p.logits, p.dtype, t * p.ld + e) == kl && __ldg(p.bias + e) == kb);
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

// A token's ids and weights, from the lanes that hold its chosen.
__device__ __forceinline__ void write_routes(const RouteParams& p, uint32_t t, int lane, const Chosen& c, bool softmax, float m, float total) {
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
    w = __fdividef(w, warp_sum(here ? w : 0.f)) * p.scale;
  } else {
    w = (softmax ? __fdividef(expf(c.l - m), total) : sigmoid_precise(c.l)) * p.scale;
  }
  if (lane < p.top_k) {
    const uint32_t o = t * p.top_k + lane;                  // (M top_k is below 2^31)
    p.weights[o] = here ? w : 0.f;
    if (p.id_bits == 64)
      static_cast<int64_t*>(p.ids)[o] = here ? c.e : -1;
    else
      static_cast<int32_t*>(p.ids)[o] = here ? c.e : -1;
  }
}

// The kernels' places a lane are 2, 4, 8, 9, 12, 16, 32, 64 and (groups only) 128.  Without runs of experts a kernel is
// taken for more than the next smaller number, so that every lane has an expert in that many places (without
// groups), and they need no comparison (65536 tokens of 257 experts: 29.3 us, 30.4 with it).
// Steps are by about a third up to 16, then double.  9 is for 256 experts and up to a lane's width more (257 to 288
// in 16 bits, 65536 tokens: 28.8 to 29.6 us, 30.7 to 30.9 with 12 places) and 33 to 36 in each of eight groups (8192
// tokens: 11.0 to 11.5, 11.5 to 11.9).  More than 64 places take all registers: 8192 tokens of 2040 experts in
// 17 groups 250 us, of 2048 in 16 groups 59.
template <int kPer>
constexpr int kPlacesBelow = kPer > 32 ? 32 : kPer > 16 ? 16 : kPer > 12 ? 12 : kPer > 9 ? 9 : kPer > 8 ? 8 : kPer > 4 ? 4 : kPer > 2 ? 2 : 0;

// A lane's places, `none` where it has no expert.  kRun experts in one load where rows allow it.
template <int kPer, bool kGroups, int kRun, typename Load>
__device__ __forceinline__ void load_runs(float (&to)[kPer], const RouteParams& p, int part, bool group, float none, Load load) {
  const int step = (kGroups ? p.lanes : 32) * kRun, first = part * kRun;
  const int left = (!kGroups || group ? p.group_size : 0) - first;      // (a lane without a group has none)
#pragma unroll
  for (int i = 0; i < kPer; i += kRun) {
    if (!kGroups && kRun == 1 && i < kPlacesBelow<kPer>) {
      load(first + i * step, &to[i]);
      continue;
    }
#pragma unroll
    for (int j = 0; j < kRun; ++j) to[i + j] = none;
    if (i / kRun * step < left) load(first + i / kRun * step, &to[i]);
  }
}
// The bias of a lane's experts (in runs: on 16 bytes, too).
template <int kPer, bool kGroups>
__device__ __forceinline__ void load_bias(float (&to)[kPer], const RouteParams& p, int first, int part, bool group) {
  const float* src = p.bias + first;
  auto four = [&](int off, float* f) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(src + off));
    f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
  };
  if constexpr (kPer % 8 == 0) {
    if (p.run == 3) {
      load_runs<kPer, kGroups, 8>(to, p, part, group, 0.f, [&](int off, float* f) { four(off, f), four(off + 4, f + 4); });
      return;
    }
  }
  if constexpr (kPer % 4 == 0) {
    if (p.run == 2) {
      load_runs<kPer, kGroups, 4>(to, p, part, group, 0.f, four);
      return;
    }
  }
  load_runs<kPer, kGroups, 1>(to, p, part, group, 0.f, [&](int off, float* f) { f[0] = __ldg(src + off); });
}
template <int kPer, bool kGroups>
__device__ __forceinline__ void load_logits(float (&to)[kPer], const RouteParams& p, int64_t at, int part, bool group) {
  if (p.dtype == MOE_TYPE_FP32) {
    const float* src = static_cast<const float*>(p.logits) + at;
    if constexpr (kPer % 4 == 0) {
      if (p.run == 2) {
        load_runs<kPer, kGroups, 4>(to, p, part, group, -CUDART_INF_F, [&](int off, float* f) {
          const float4 v = __ldg(reinterpret_cast<const float4*>(src + off));
          f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
        });
        return;
      }
    }
    load_runs<kPer, kGroups, 1>(to, p, part, group, -CUDART_INF_F, [&](int off, float* f) { f[0] = __ldg(src + off); });
    return;
  }
  const unsigned short* src = static_cast<const unsigned short*>(p.logits) + at;
  const bool bf16 = p.dtype == MOE_TYPE_BF16;
  if constexpr (kPer % 8 == 0) {
    if (p.run == 3) {
      load_runs<kPer, kGroups, 8>(to, p, part, group, -CUDART_INF_F, [&](int off, float* f) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(src + off));
        float w[8];
        if (bf16) unpack8<__nv_bfloat16>(v, w); else unpack8<__half>(v, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = w[j];
      });
      return;
    }
  }
  if (bf16)
    load_runs<kPer, kGroups, 1>(to, p, part, group, -CUDART_INF_F, [&](int off, float* f) { f[0] = __uint_as_float(static_cast<uint32_t>(__ldg(src + off)) << 16); });
  else
    load_runs<kPer, kGroups, 1>(to, p, part, group, -CUDART_INF_F, [&](int off, float* f) { f[0] = __half2float(__ushort_as_half(__ldg(src + off))); });
}

// kMode: what the choice compares.  0: the logits; 1: sigmoid scores (and
// bias); 2: softmax scores (and bias).  A lane holds kPer experts at most.
template <int kPer, int kMode, bool kGroups>
__global__ void __launch_bounds__(32 * (kMode == 0 ? kWarps : kWarpsScored), kPer > 16 ? 1 : kMode == 0 ? 6 : 8)
    route_scores_kernel(const __grid_constant__ RouteParams p) {
  constexpr int kTokens = kMode == 0 ? kWarps : kWarpsScored;
  using Mask = PlaceMask<kPer>;
  __shared__ __align__(16) uint64_t s_key[kTokens][32];
  __shared__ int16_t s_cand[kTokens][32];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int lanes = kGroups ? p.lanes : 32, g = kGroups ? lane / p.lanes : 0, part = lane - g * lanes;
  const bool group = g < p.groups;
  const int first = g * p.group_size + (part << p.run), run_step = lanes << p.run, run_mask = (1 << p.run) - 1;
  const uint32_t M = static_cast<uint32_t>(p.M), live = p.num_tokens ? min(static_cast<uint32_t>(max(*p.num_tokens, 0)), M) : M;
  const bool softmax = kMode == 2 || (kMode == 0 && p.score == MOE_SCORE_SOFTMAX);
  const bool biased = kMode != 0 && p.bias != nullptr;

  constexpr bool kHold = kMode != 0 && kPer <= 16;   // the bias stays in registers
  float held[kPer];                                  // (only then)
  float most_bias = 0.f;                             // of the finite ones
  if (kHold) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) held[i] = 0.f;
    if (biased) {
      if constexpr (kHold) load_bias<kPer, kGroups>(held, p, g * p.group_size, part, group);
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (fabsf(held[i]) < CUDART_INF_F) most_bias = fmaxf(most_bias, fabsf(held[i]));
    }
  } else if (biased) {
    for (int e = lane; e < p.E; e += 32)
      if (const float b = fabsf(__ldg(p.bias + e)); b < CUDART_INF_F) most_bias = fmaxf(most_bias, b);
  }
  if (kMode != 0) most_bias = warp_max(most_bias);

  for (uint32_t t = blockIdx.x * kTokens + warp; t < M; t += gridDim.x * kTokens) {
    Chosen c = {0, -1, 0.f};
    float m = 0.f, total = 1.f;
    if (t < live) {
      float inv = 1.f, err = 0.f;
      int n = 0, way = 0;                          // 1: many candidates, 2: in 64 bits
      bool stays = true;                                    // this lane's group
      float v[kPer];                                        // the logits, then the values (-inf: left out)
      const int64_t row = static_cast<int64_t>(t) * static_cast<int32_t>(p.ld);        // (both below 2^31)
      load_logits<kPer, kGroups>(v, p, row + g * p.group_size, part, group);
      float a1 = v[0], a2 = -CUDART_INF_F;                  // the lane's (then group's) two largest
#pragma unroll
      for (int i = 1; i < kPer; ++i) {
        if (kGroups && kMode == 0) a2 = fmaxf(a2, fminf(a1, v[i]));
        a1 = max_nan(a1, v[i]);
      }
      bool nan = a1 != a1;
      // No value is further than `err` from its true one.  In units of 2^-23 a sigmoid is off by the fast
      // exponential's 2 + 1.173 |x| and the divide's and sum's 3, times itself: most at the largest
      // logit, or at 0.  For softmax see route_softmax_units.
      err = 0.f;
      if (kMode != 0 || (softmax && !p.renormalize)) m = warp_max(a1);
      if (kMode == 2 || (kMode == 0 && softmax && !p.renormalize)) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) sum += exp_coarse(v[i] - m);
        total = warp_sum(sum);
      }
      if (kMode != 0) {
        inv = kMode == 2 ? reciprocal_coarse(total) : 1.f;
        err = kMode == 1 ? fmaf(fmaxf(m, 0.f), 1.2f, 5.f) : p.softmax_units * inv;
        err = fmaf(err, 0x1p-23f, fmaf(most_bias + inv, 0x1p-22f, 0x1p-120f));          // (and the addition's half: a score is at most inv)
        a1 = -CUDART_INF_F;
        float any = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const float s = kMode == 1 ? reciprocal_coarse(1.f + exp_coarse(-v[i])) : exp_coarse(v[i] - m) * inv;
          float x = s + (kHold ? held[i] : 0.f);
          if (!kHold && biased) {
            const int e = i < p.per ? route_expert_at(p, i, lane) : -1;
            x = s + (e >= 0 ? __ldg(p.bias + e) : 0.f);
          }
          v[i] = v[i] == -CUDART_INF_F ? v[i] : x;
          any = max_nan(any, v[i]);
          if (kGroups) a2 = fmaxf(a2, fminf(a1, v[i]));
          a1 = fmaxf(a1, v[i]);
        }
        nan |= any != any;
      }
      float low = a1, second = a2;                          // the lane's two largest values
      way = __any_sync(kAll, nan) ? 2 : 0;
      if (kGroups && way == 0) {
        for (int o = 1; o < lanes; o <<= 1) {
          const float b1 = __shfl_xor_sync(kAll, a1, o);
          if (kMode != 0) a2 = fmaxf(fmaxf(a2, __shfl_xor_sync(kAll, a2, o)), fminf(a1, b1));
          a1 = fmaxf(a1, b1);
        }
        const bool pair = kMode != 0 && p.pair && a2 != -CUDART_INF_F;
        // (half of a group's value where scores are compared: sums of two of the type's lowest value stay in range)
        const float x = kMode == 0 ? a1 : pair ? fmaf(0.5f, a1, 0.5f * a2) : 0.5f * a1;
        // the topk_groups largest, one after another, of equal ones the lower
        stays = false;
        float cur = group ? x : -CUDART_INF_F;
        for (int j = 0; j < p.topk_groups; ++j) {
          const float top = warp_max(cur);
          const uint32_t at = __ballot_sync(kAll, cur == top && group && !stays);
          if (at == 0) break;
          if ((lane ^ (__ffs(static_cast<int>(at)) - 1)) < lanes) stays = true, cur = -CUDART_INF_F;      // (lanes is a power of two)
        }
        if (kMode != 0) {
          // a group that stays and one that goes nearer than their errors
          const float worst = -warp_max(stays ? -x : -CUDART_INF_F), best = warp_max(!stays && group ? x : -CUDART_INF_F), near = 2.f * err;
          if (best != -CUDART_INF_F && !(worst - best > near)) {
            // (equal experts, as of a router's first step, are equal whatever their error)
            bool same = true;
#pragma unroll
            for (int i = 0; i < kPer; ++i) same &= v[i] == a1 || v[i] == -CUDART_INF_F;
            if (!(__all_sync(kAll, same) && all_equal(p, t))) {
              // which ones are in question: their experts that may be among their two largest, in 64 bits
              const bool in_question = group && !(stays ? x - best > near : worst - x > near);
              const int sure = __popc(__ballot_sync(kAll, stays && !in_question)) / lanes;
              const float floor = (pair ? a2 : a1) - 2.f * err;
              Mask some = 0;
#pragma unroll
              for (int i = 0; i < kPer; ++i)
                if (v[i] != -CUDART_INF_F && !(v[i] < floor)) some |= Mask(1) << i;
              const bool among = groups_exactly<kMode, Mask>(p, t, in_question ? some : Mask(0), m, in_question, p.topk_groups - sure);
              if (in_question) stays = among;
            }
          }
        }
        if (!stays) low = second = -CUDART_INF_F;
      }
      if (way == 0) {
        // the threshold: what is below the top_k-th largest of the lanes' two largest (one where all
        // lanes are in) by more than two errors has top_k others above it
        float thr = -CUDART_INF_F;
#pragma unroll 2
        for (int j = 0; j < p.top_k; ++j) {
          thr = warp_max(low);
          if (low == thr) low = second, second = -CUDART_INF_F;
        }
        // (what is left out lies below the smallest finite value; a lane whose group goes takes none)
        thr = fmaxf(kMode == 0 ? thr : thr - 2.f * err, -3.402823466e38f);
        if (kGroups && !stays) thr = CUDART_NAN_F;
        Mask cand = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (v[i] >= thr) cand |= Mask(1) << i;
        __syncwarp();                                       // (the last token's reads of s_cand are done)
        const uint32_t below = (1u << lane) - 1;
        for (uint32_t some = __ballot_sync(kAll, cand != 0); some; some = __ballot_sync(kAll, cand != 0)) {
          if (cand) {
            const int pos = n + __popc(some & below);
            const int i = first_place(cand);
            cand &= cand - 1;
            if (pos < 32) s_cand[warp][pos] = static_cast<int16_t>(first + ((i >> p.run) * run_step + (i & run_mask)));
          }
          n += __popc(some);
          if (n > 32) break;
        }
        __syncwarp();
        if (n > 32) {
          way = 1;
        } else {
          // the candidates, one a lane, formed as before
          const int e = lane < n ? s_cand[warp][lane] : -1;
          const bool here = e >= 0 && MOE_IN_BOUNDS(e < p.E);
          const float l = here ? logit_at(p.logits, p.dtype, row + e) : 0.f;
          const float b = here && biased ? __ldg(p.bias + e) : 0.f;
          const float x = biased ? coarse_value<kMode>(l, b, m, inv) : l;
          // rank: how many are above (equal ones, frequent in 16 bits: of lower index); idle lanes' keys are 0
          const uint64_t key = here ? (static_cast<uint64_t>(order_key(x)) << 32) | static_cast<uint32_t>(~e) : 0;
          s_key[warp][lane] = key;
          __syncwarp();
          int rank = 0;
#pragma unroll 1
          for (int j = 0; j < n; j += 4) {
            const ulonglong2 k0 = *reinterpret_cast<const ulonglong2*>(&s_key[warp][j]);
            const ulonglong2 k1 = *reinterpret_cast<const ulonglong2*>(&s_key[warp][j + 2]);
            rank += (k0.x > key) + (k0.y > key) + (k1.x > key) + (k1.y > key);
          }
          int src = place(s_cand[warp], here ? rank : lane, lane);
          c.n = min(n, p.top_k);
          c.e = __shfl_sync(kAll, e, src);
          c.l = __shfl_sync(kAll, l, src);
          if (biased) {
            const float sv = __shfl_sync(kAll, x, src), sb = __shfl_sync(kAll, b, src);
            // each chosen one against the next, and the last chosen against all behind it; equal
            // logits of equal biases are equal, whatever their error
            const int ref = max(lane < p.top_k ? lane - 1 : p.top_k - 1, 0);
            const float rv = __shfl_sync(kAll, sv, ref), rl = __shfl_sync(kAll, c.l, ref), rb = __shfl_sync(kAll, sb, ref);
            const bool close = lane > 0 && lane < n && !(rv - sv > 2.f * err) && !(rl == c.l && rb == sb);
            if (__any_sync(kAll, close)) {
              rank = rank_exactly<kMode>(p, t, n, e, l, b, m);
              src = place(s_cand[warp], here ? rank : lane, lane);
              c.e = __shfl_sync(kAll, e, src);
              c.l = __shfl_sync(kAll, l, src);
            }
          }
        }
      }
      if (way == 1) c = choose_of_many<kMode, kMostPlaces<kPer>>(p, t, stays, m, inv, err);
      if (way == 2 || c.n < 0) c = choose_exactly<kMostPlaces<kPer>>(p, t, kMode != 0);
    }
    write_routes(p, t, lane, c, softmax, m, total);
    if (kMode != 0) break;
  }
}

// The logits' gradient.  One warp per token: the chosen logits go to a lane each, the
// row is written in whole lines (zeros, or for plain softmax every expert's
// -s sum(dw s)), then the chosen places by their lanes, after a warp barrier.
//
// Zeros: the writes bound it (8192 tokens of 512 experts, FP32: 6.0 us, 3.0 TB/s into L2 and
// HBM, launch included).  Dense rows: two loads one after the other (ids, their logits), two
// sums over the warp and 350 instructions a token (65536 tokens of 257 experts in 16 bits: 32.2 us with
// the balance step, 2.2 TB/s); pairs of 16-bit logits, 42 us one at a time.  Loads of the next token ahead and both sums
// in one exchange changed nothing; six CTAs an SM instead of eight 38 us.
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

// The next smaller of the dense kernels' words a lane, which a kernel is taken for more than: words below it
// lie inside the row (but the first pair, which may begin one before it), and need no comparison (32.1 -> 31.3 us).
// 16-bit rows of 256, 512 and 2048 experts need one word more than a power of two, for that pair: 5, 9 and 33.  65536 x 256
// takes 30.4 us, 42.6 with nine words a lane, and 32768 x 512 31.7, 67 with sixteen.
template <int kPer>
constexpr int kWordsBelow = kPer > 33 ? 33 : kPer > 16 ? 16 : kPer > 9 ? 9 : kPer > 5 ? 5 : kPer > 4 ? 4 : kPer > 2 ? 2 : 0;

// (the row may be written in place: plain loads, not those of memory that stays as it is)
template <typename T> struct Logit;
template <> struct Logit<float> {
  static __device__ __forceinline__ float load(const float* p) { return *p; }
  static __device__ __forceinline__ float round(float v) { return v; }
};
template <> struct Logit<__nv_bfloat16> {
  static __device__ __forceinline__ float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  static __device__ __forceinline__ __nv_bfloat16 round(float v) { return __float2bfloat16_rn(v); }
};
template <> struct Logit<__half> {
  static __device__ __forceinline__ float load(const __half* p) { return __half2float(*p); }
  static __device__ __forceinline__ __half round(float v) { return __float2half_rn(v); }
};

// kPer: words of a lane in a dense row (softmax, not renormalised; 0: the others)
template <typename T, int kPer>
__global__ void __launch_bounds__(32 * kWarps, kPer <= 9 ? 8 : 1)
    route_scores_backward_kernel(const __grid_constant__ RouteGradParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x % 32;
  const uint32_t M = static_cast<uint32_t>(p.M), live = p.num_tokens ? min(static_cast<uint32_t>(max(*p.num_tokens, 0)), M) : M;
  const bool softmax = p.score == MOE_SCORE_SOFTMAX;
  for (uint32_t t = blockIdx.x * kWarps + threadIdx.x / 32; t < M; t += gridDim.x * kWarps) {
    T* row = static_cast<T*>(p.dlogits) + static_cast<int64_t>(t) * static_cast<int32_t>(p.ldd);
    // a dense row: kPer words of one or two logits a lane, on their way before the rest
    // (16 bits: words start at even addresses, which may be one before the row)
    constexpr int kEach = 4 / static_cast<int>(sizeof(T)), kWords = kPer == 0 ? 1 : kPer;
    const T* in = static_cast<const T*>(p.logits) + static_cast<int64_t>(t) * static_cast<int32_t>(p.ld);
    const int back = kEach == 2 ? static_cast<int>(reinterpret_cast<uintptr_t>(in) >> 1) & 1 : 0;
    float s[kWords][kEach];
    constexpr int kSure = kWordsBelow<kPer>;
    if constexpr (kPer != 0) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const int at = kEach * (lane + 32 * i) - back;
#pragma unroll
        for (int j = 0; j < kEach; ++j) s[i][j] = -CUDART_INF_F;
        if (t < live) {
          if constexpr (kEach == 1) {
            if (i < kSure || at < p.E) s[i][0] = in[at];
          } else if (((i > 0 && i < kSure) || (at >= 0 && at + 1 < p.E)) && p.vec) {
            const float2 v = Pack2<T>::load(*reinterpret_cast<const unsigned int*>(in + at));
            s[i][0] = v.x, s[i][1] = v.y;
          } else {
#pragma unroll
            for (int j = 0; j < kEach; ++j)
              if (at + j >= 0 && at + j < p.E) s[i][j] = Logit<T>::load(in + at + j);
          }
        }
      }
    }
    int e = -1;
    float l = 0.f, dw = 0.f;
    if (t < live && lane < p.top_k) {
      const uint32_t o = t * p.top_k + lane;                  // (M top_k is below 2^31)
      if (p.id_bits == 64) {
        const long long id = __ldg(static_cast<const long long*>(p.ids) + o);
        e = id >= 0 && id < p.E ? static_cast<int>(id) : -1;
      } else {
        e = __ldg(static_cast<const int32_t*>(p.ids) + o);
      }
      dw = __ldg(p.dweights + o);
    }
    bool here = e >= 0 && e < p.E;
    if (here) {
      l = Logit<T>::load(in + e);
      here = l != -CUDART_INF_F;
    }
    // an expert listed more than once counts by all of its terms: their sum and number
    // (the match goes from one value to the next: idle lanes share theirs)
    const uint32_t same = __match_any_sync(kAll, here ? e : -1);
    float sum_dw = dw, terms = 1.f;
    if (__any_sync(kAll, here && __popc(same) > 1)) {
      sum_dw = terms = 0.f;
      for (int j = 0; j < p.top_k; ++j) {
        const float x = __shfl_sync(kAll, dw, j);
        if ((same >> j) & 1) sum_dw += x, terms += 1.f;
      }
    }
    float own;                                      // the gradient at this lane's expert
    __syncwarp();                                   // (every lane has its logits: the row may be written)
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
      float m = -CUDART_INF_F, sum = 0.f;
#pragma unroll
      for (int i = 0; i < kWords; ++i)
#pragma unroll
        for (int j = 0; j < kEach; ++j) m = fmaxf(m, s[i][j]);
      m = warp_max(m);
      const float ref = m == -CUDART_INF_F ? 0.f : m;              // (a row of -inf has no gradient)
#pragma unroll
      for (int i = 0; i < kWords; ++i)
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
          s[i][j] = exp_coarse(s[i][j] - ref);
          sum += s[i][j];
        }
      sum = warp_sum(sum);
      const float inv = sum == 0.f ? 0.f : __frcp_rn(sum);
      const float mine = here ? exp_coarse(l - ref) * inv : 0.f;
      const float mean = warp_sum(here ? dw * mine : 0.f), factor = -p.scale * mean * inv;
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const int at = kEach * (lane + 32 * i) - back;
        if constexpr (kEach == 1) {
          if (i < kSure || at < p.E) row[at] = Logit<T>::round(s[i][0] * factor);
        } else if (((i > 0 && i < kSure) || (at >= 0 && at + 1 < p.E)) && p.vec) {
          *reinterpret_cast<unsigned int*>(row + at) = Pack2<T>::store(s[i][0] * factor, s[i][1] * factor);
        } else {
#pragma unroll
          for (int j = 0; j < kEach; ++j)
            if (at + j >= 0 && at + j < p.E) row[at + j] = Logit<T>::round(s[i][j] * factor);
        }
      }
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

// (kPlacesBelow has the same numbers)
template <int kMode, bool kGroups>
auto route_kernel_of(int places) {
  if constexpr (kGroups) {
    if (places > 64) return route_scores_kernel<128, kMode, kGroups>;
  }
  return places == 2    ? route_scores_kernel<2, kMode, kGroups>
         : places == 4  ? route_scores_kernel<4, kMode, kGroups>
         : places == 8  ? route_scores_kernel<8, kMode, kGroups>
         : places == 9  ? route_scores_kernel<9, kMode, kGroups>
         : places == 12 ? route_scores_kernel<12, kMode, kGroups>
         : places == 16 ? route_scores_kernel<16, kMode, kGroups>
         : places == 32 ? route_scores_kernel<32, kMode, kGroups>
                        : route_scores_kernel<64, kMode, kGroups>;
}

template <typename T>
auto route_grad_kernel_of(bool dense, int words) {
  return !dense        ? route_scores_backward_kernel<T, 0>
         : words <= 2  ? route_scores_backward_kernel<T, 2>
         : words <= 4  ? route_scores_backward_kernel<T, 4>
         : words <= 5  ? route_scores_backward_kernel<T, 5>
         : words <= 9  ? route_scores_backward_kernel<T, 9>
         : words <= 16 ? route_scores_backward_kernel<T, 16>
         : words <= 33 ? route_scores_backward_kernel<T, 33>
                       : route_scores_backward_kernel<T, 64>;
}

// Checks that both directions share: types, sizes, choices.
moe_status check_route(int dtype, int id_bits, int score, int64_t M, int E, int top_k, int64_t ld, float scale) {
  if (!is_type(dtype) || (id_bits != 32 && id_bits != 64)) return MOE_ERR_DTYPE;
  if (!ok_routes(M, top_k < 1 ? 1 : top_k) || top_k < 1 || top_k > kRouteMaxTopK || E < 1 || E > kRouteMaxE || ld < E ||
      ld >= (int64_t(1) << 31) || (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) || !(scale - scale == 0.f))
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
  // (all groups staying is no grouping)
  const int groups = a->topk_groups == a->groups ? 1 : a->groups;
  RouteParams p;
  static_cast<RouteLayout&>(p) =
      route_layout(a->E, groups, eb, aligned16(a->logits) && aligned16(a->bias) && a->ldlogits * eb % 16 == 0);
  const int places = route_places(p);
  if (p.per > places || (groups == 1 && places > 64)) return MOE_ERR_SHAPE;      // (no size: the layout's test goes through all)
  p.logits = a->logits;
  p.bias = a->bias;
  p.ids = a->topk_ids;
  p.weights = a->topk_weights;
  p.num_tokens = a->num_tokens;
  p.M = a->M;
  p.ld = a->ldlogits;
  p.top_k = a->top_k;
  p.topk_groups = groups == 1 ? 1 : a->topk_groups;
  p.pair = a->group_score == MOE_GROUP_TOP2;
  p.score = a->score;
  p.renormalize = a->renormalize;
  p.dtype = a->dtype;
  p.id_bits = a->id_bits;
  p.scale = a->routed_scale;
  p.softmax_units = route_softmax_units(a->E, places);
  // without a bias the scores' order is the logits'; sums of two scores have none such
  const bool scored = a->bias || (p.groups > 1 && p.pair);
  const int mode = !scored ? 0 : a->score == MOE_SCORE_SIGMOID ? 1 : 2;
  auto kernel = p.groups > 1 ? (mode == 0   ? route_kernel_of<0, true>(places)
                                : mode == 1 ? route_kernel_of<1, true>(places)
                                            : route_kernel_of<2, true>(places))
                             : (mode == 0   ? route_kernel_of<0, false>(places)
                                : mode == 1 ? route_kernel_of<1, false>(places)
                                            : route_kernel_of<2, false>(places));
  const int warps = mode == 0 ? kWarps : kWarpsScored;
  const unsigned grid = mode == 0 ? warp_grid(a->M, dev.sms) : static_cast<unsigned>(ceil_div(a->M, warps));
  MOE_CUDA_TRY(launch_pdl(kernel, dim3(grid), dim3(32 * warps), 0, stream, 1, p));
  return MOE_OK;
}

moe_status moe_route_scores_backward(const moe_route_scores_backward_args* a, moe_stream_t stream) {
  using namespace moe;
  if (!a) return MOE_ERR_NULL;
  const moe_status bad = check_route(a->dtype, a->id_bits, a->score, a->M, a->E, a->top_k, a->ldlogits, a->routed_scale);
  if (bad != MOE_OK) return bad;
  if (a->lddlogits < a->E || a->lddlogits >= (int64_t(1) << 31)) return MOE_ERR_SHAPE;
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
  const bool dense = a->score == MOE_SCORE_SOFTMAX && !a->renormalize;
  // whole rows of zeros in 16-byte stores; dense rows of 16 bits in pairs, where input and output have them alike
  p.vec = dense ? ((reinterpret_cast<uintptr_t>(a->logits) ^ reinterpret_cast<uintptr_t>(a->dlogits)) & 2) == 0 &&
                      (a->M == 1 || (a->ldlogits - a->lddlogits) % 2 == 0)
                : aligned16(a->dlogits) && a->lddlogits * eb % 16 == 0 && a->E * eb % 16 == 0;
  const int words = static_cast<int>(eb == 4 ? ceil_div(a->E, 32) : ceil_div(a->E + 1, 64));
  auto kernel = a->dtype == MOE_TYPE_BF16   ? route_grad_kernel_of<__nv_bfloat16>(dense, words)
                : a->dtype == MOE_TYPE_FP16 ? route_grad_kernel_of<__half>(dense, words)
                                            : route_grad_kernel_of<float>(dense, words);
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
