// One AdamW step over many tensors in one launch (moe_adamw_step).
//
// A device table lists the tensors; each is cut into chunks of 2048 elements
// and the CTAs walk the chunks of all tensors, so that a list of small
// tensors costs one launch.  Per element the step reads the gradient, the
// parameter and both states once and writes the parameter, its 16-bit copy
// and the states once: HBM bounds it.
//
// The arithmetic is FP32.  268 million elements, BF16 gradients and copy: 32-bit
// states 1141 us (28 bytes an element, 6.6 TB/s, the measured copy rate), 8-bit
// states 715 us (16.1 bytes, 6.05 TB/s; some 50 instructions an element keep the
// schedulers busy enough that the loads have to run a chunk ahead).
#include <cfloat>
#include <cmath>
#include <new>
#include <vector>

#include "train.cuh"

namespace moe {
namespace {

constexpr int kChunk = 2048;   // elements per chunk
constexpr int kThreads = 128;
constexpr int kSteps = kChunk / (4 * kThreads);  // four elements per thread and step

struct AdamEntry {
  float* param;
  uint16_t* model;
  const void* grad;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  int64_t n;
  int64_t first_chunk;
  float weight_decay;
  int32_t kind;   // the gradients' type, and kEightBits (a kernel for other states would write past this tensor's)
  int32_t model_dtype;
};
constexpr int32_t kEightBits = 4;

struct AdamParams {
  const AdamEntry* table;
  const float* grad_scale;
  const int32_t* skip;
  int64_t chunks;
  float lr;
  float beta1, one_minus_beta1, beta2, one_minus_beta2;
  float step_size;   // lr / (1 - beta1^step)
  float root_scale;  // 1 / sqrt(1 - beta2^step)
  float eps;
  uint32_t seed;
  int count;
};

// The new m, v, root of v and parameter of one element.  m and v are rounded
// once per written operation; the quotient of the update comes from the
// hardware's reciprocal (within 2 units of the last place of the update, far
// below the parameter's own rounding).  Two elements at a time: the packed FP32 instructions round each half as the
// scalar ones do.
struct Elem2 {
  float2 m, v, r, p;
};
__device__ __forceinline__ float rsqrt_fast(float v) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp_fast(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
// The sum of two packed products, each rounded on its own: a packed addition
// would be contracted with them (and a state's last bit decides, now and then,
// about an 8-bit code).
__device__ __forceinline__ float2 add_unfused(float2 a, float2 b) {
  return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y));
}
__device__ __forceinline__ float2 neg(float2 v) { return make_float2(-v.x, -v.y); }

// The states' codes are to be those of the formula, so roots and quotients are
// rounded correctly: an approximation and its exact residual, corrected once
// (Markstein's method).  Of all floats from 2^-102 on, every root is the
// correctly rounded one.  Below, the residual underflows: the root's last bit may be
// off, and from v = 1e-37 down it comes out too small (0.15 of it at 1e-39).
// kSmall: small values are taken 2^100 times as large.  That costs 2.7% with
// 8-bit states (733 us against 715 at 268 million elements) and 0.7% with 32-bit
// ones, so it is chosen by eps, beside which such roots vanish (moe_adamw_step).
template <bool kSmall>
__device__ __forceinline__ float2 root2(float2 u) {
  const bool up_x = kSmall && u.x < 0x1p-100f, up_y = kSmall && u.y < 0x1p-100f;
  const float2 v = kSmall ? __fmul2_rn(u, make_float2(up_x ? 0x1p100f : 1.f, up_y ? 0x1p100f : 1.f)) : u;
  const float2 y = make_float2(rsqrt_fast(fmaxf(v.x, 1e-37f)), rsqrt_fast(fmaxf(v.y, 1e-37f)));
  const float2 s = __fmul2_rn(v, y);
  float2 r = __ffma2_rn(__ffma2_rn(neg(s), s, v), __fmul2_rn(y, both(0.5f)), s);
  if (kSmall) r = __fmul2_rn(r, make_float2(up_x ? 0x1p-50f : 1.f, up_y ? 0x1p-50f : 1.f));
  // (infinity is its own root; the steps above would make it a NaN)
  return make_float2(v.x > FLT_MAX ? v.x : r.x, v.y > FLT_MAX ? v.y : r.y);
}
// a / b, `inv` the correctly rounded reciprocal of b.
__device__ __forceinline__ float2 quotient2(float2 a, float b, float inv) {
  const float2 q = __fmul2_rn(a, both(inv));
  return __ffma2_rn(__ffma2_rn(neg(q), both(b), a), both(inv), q);
}
__device__ __forceinline__ float2 second_moment(const AdamParams& a, float2 g, float2 v) {
  return add_unfused(__fmul2_rn(v, both(a.beta2)), __fmul2_rn(__fmul2_rn(g, g), both(a.one_minus_beta2)));
}
template <bool kSmall>
__device__ __forceinline__ Elem2 adam_elem2(const AdamParams& a, float decay, float2 g, float2 p, float2 m, float2 v) {
  Elem2 e;
  e.m = add_unfused(__fmul2_rn(m, both(a.beta1)), __fmul2_rn(g, both(a.one_minus_beta1)));
  e.v = second_moment(a, g, v);
  e.r = root2<kSmall>(e.v);
  const float2 den = __ffma2_rn(e.r, both(a.root_scale), both(a.eps));
  const float2 upd = __fmul2_rn(__fmul2_rn(e.m, both(-a.step_size)), make_float2(rcp_fast(den.x), rcp_fast(den.y)));
  e.p = __fadd2_rn(__fmul2_rn(p, both(decay)), upd);
  return e;
}

// Four gradients: their bits first (nothing waits for them yet), then the
// values.
// kGrad: the gradients' type, known when a chunk's loop is chosen.
template <int kGrad>
__device__ __forceinline__ uint4 load_grad4(const AdamEntry& t, int64_t i, bool ok) {
  uint4 raw = make_uint4(0, 0, 0, 0);
  if (ok && kGrad == MOE_TYPE_FP32)
    raw = __ldcs(reinterpret_cast<const uint4*>(static_cast<const float*>(t.grad) + i));
  if (ok && kGrad != MOE_TYPE_FP32) {
    const uint2 v = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(t.grad) + i));
    raw.x = v.x;
    raw.y = v.y;
  }
  return raw;
}
template <int kGrad>
__device__ __forceinline__ void grad4(const uint4& raw, float (&g)[4]) {
  if (kGrad == MOE_TYPE_FP32) {
    g[0] = __uint_as_float(raw.x); g[1] = __uint_as_float(raw.y);
    g[2] = __uint_as_float(raw.z); g[3] = __uint_as_float(raw.w);
    return;
  }
  const float2 a = kGrad == MOE_TYPE_BF16 ? Pack2<__nv_bfloat16>::load(raw.x) : Pack2<__half>::load(raw.x);
  const float2 b = kGrad == MOE_TYPE_BF16 ? Pack2<__nv_bfloat16>::load(raw.y) : Pack2<__half>::load(raw.y);
  g[0] = a.x; g[1] = a.y; g[2] = b.x; g[3] = b.y;
}
__device__ __forceinline__ float load_grad1(const AdamEntry& t, int64_t i) {
  const int dtype = t.kind % kEightBits;
  if (dtype == MOE_TYPE_FP32) return static_cast<const float*>(t.grad)[i];
  const uint32_t v = static_cast<const uint16_t*>(t.grad)[i];
  return dtype == MOE_TYPE_BF16 ? Pack2<__nv_bfloat16>::load(v).x : Pack2<__half>::load(v).x;
}
__device__ __forceinline__ uint2 model4(const AdamEntry& t, const float (&p)[4]) {
  if (t.model_dtype == MOE_TYPE_BF16)
    return make_uint2(Pack2<__nv_bfloat16>::store(p[0], p[1]), Pack2<__nv_bfloat16>::store(p[2], p[3]));
  return make_uint2(Pack2<__half>::store(p[0], p[1]), Pack2<__half>::store(p[2], p[3]));
}

// The table entry that holds chunk c (whole warps): 128 entries are compared
// at a time, four a lane, so a list of 128 tensors takes one load's latency and
// one of 16384 two.
__device__ __forceinline__ int find_entry(const AdamParams& a, int64_t c) {
  int lo = 0, n = a.count;   // table[lo].first_chunk <= c; the entry is in [lo, lo + n)
  while (n > 1) {
    const int stride = (n + 127) / 128;
    unsigned le = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = (4 * static_cast<int>(threadIdx.x % 32) + j) * stride;
      if (i < n && a.table[lo + i].first_chunk <= c) ++le;
    }
    const int k = static_cast<int>(__reduce_add_sync(0xffffffffu, le)) - 1;
    lo += k * stride;
    n = min(stride, n - k * stride);
  }
  return lo;
}

// ---------------------------------------------------------------- 32-bit states

// A chunk, four elements a thread and step; steps that pass the tensor's end
// are left out.
template <int kGrad, bool kSmall>
__device__ __forceinline__ void adamw32_chunk(const AdamParams& a, const AdamEntry& t, float decay, float gs,
                                              int64_t i0) {
  // every load of the chunk goes out before the first result is needed
  uint4 raw[kSteps];
  float4 p4[kSteps], m4[kSteps], v4[kSteps];
  float* m = static_cast<float*>(t.m);
  float* v = static_cast<float*>(t.v);
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const int64_t i = i0 + 4 * (threadIdx.x + u * kThreads);
    const bool ok = i + 4 <= t.n;
    raw[u] = load_grad4<kGrad>(t, i, ok);
    if (ok) p4[u] = __ldcs(reinterpret_cast<const float4*>(t.param + i));
    if (ok) m4[u] = __ldcs(reinterpret_cast<const float4*>(m + i));
    if (ok) v4[u] = __ldcs(reinterpret_cast<const float4*>(v + i));
  }
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const int64_t i = i0 + 4 * (threadIdx.x + u * kThreads);
    if (i + 4 > t.n) continue;
    float g[4], p[4];
    grad4<kGrad>(raw[u], g);
    const Elem2 lo = adam_elem2<kSmall>(a, decay, __fmul2_rn(make_float2(g[0], g[1]), both(gs)), make_float2(p4[u].x, p4[u].y),
                                make_float2(m4[u].x, m4[u].y), make_float2(v4[u].x, v4[u].y));
    const Elem2 hi = adam_elem2<kSmall>(a, decay, __fmul2_rn(make_float2(g[2], g[3]), both(gs)), make_float2(p4[u].z, p4[u].w),
                                make_float2(m4[u].z, m4[u].w), make_float2(v4[u].z, v4[u].w));
    p[0] = lo.p.x; p[1] = lo.p.y; p[2] = hi.p.x; p[3] = hi.p.y;
    m4[u] = make_float4(lo.m.x, lo.m.y, hi.m.x, hi.m.y);
    v4[u] = make_float4(lo.v.x, lo.v.y, hi.v.x, hi.v.y);
    __stcs(reinterpret_cast<float4*>(t.param + i), make_float4(p[0], p[1], p[2], p[3]));
    __stcs(reinterpret_cast<float4*>(m + i), m4[u]);
    __stcs(reinterpret_cast<float4*>(v + i), v4[u]);
    if (t.model) *reinterpret_cast<uint2*>(t.model + i) = model4(t, p);
  }
}

template <int kGrad, bool kSmall>
__global__ void __launch_bounds__(kThreads) adamw32_kernel(const __grid_constant__ AdamParams a) {
  pdl_wait();
  if (a.skip && *a.skip) return;
  const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
  for (int64_t c = blockIdx.x; c < a.chunks; c += gridDim.x) {
    const AdamEntry t = a.table[find_entry(a, c)];
    if (t.kind != kGrad) continue;
    const float decay = fmaf(-a.lr, t.weight_decay, 1.0f);
    const int64_t i0 = (c - t.first_chunk) * kChunk;
    if (!MOE_IN_BOUNDS(i0 >= 0)) continue;
    adamw32_chunk<kGrad, kSmall>(a, t, decay, gs, i0);
    // the last one to three elements, in their chunk (past the table's chunks there is none)
    const int64_t k = (t.n & ~int64_t(3)) + threadIdx.x;
    if (k < t.n && static_cast<uint64_t>(k - i0) < kChunk) {
      float* m = static_cast<float*>(t.m);
      float* v = static_cast<float*>(t.v);
      const Elem2 e = adam_elem2<kSmall>(a, decay, both(__fmul_rn(load_grad1(t, k), gs)), both(t.param[k]), both(m[k]), both(v[k]));
      t.param[k] = e.p.x;
      m[k] = e.m.x;
      v[k] = e.v.x;
      const float p[4] = {e.p.x, 0.f, 0.f, 0.f};
      if (t.model) t.model[k] = static_cast<uint16_t>(model4(t, p).x & 0xFFFFu);
    }
  }
}

// ---------------------------------------------------------------- 8-bit states

// Twenty bits for one element: an integer hash of seed, tensor and element;
// `key` is what the elements of 2^32 share.  The two multiply-xorshift rounds
// are the published mixer of C. Wellons ("Prospecting for Hash Functions", 2018).
__device__ __forceinline__ uint32_t random_key(uint32_t seed, uint32_t tensor, int64_t i) {
  return static_cast<uint32_t>(i >> 32) * 0x85EBCA77u + seed + 0x9E3779B9u * (tensor + 1u);
}
__device__ __forceinline__ uint32_t random20(uint32_t key, uint32_t i) {
  uint32_t x = i * 0x9E3779B1u + key;
  x = (x ^ (x >> 16)) * 0x7FEB352Du;
  x = (x ^ (x >> 15)) * 0x846CA68Bu;
  return (x ^ (x >> 16)) >> 12;
}

// The smaller one, or the NaN.
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// E4M3 code of y in [0, 448.x], rounded up with probability (part cut off) /
// (code spacing).  From 2^-6 on the spacing is 2^20 units of the FP32 pattern
// (three mantissa bits stay), so the random bits are added below it and cut
// off; the exponent's bias goes from 127 to 7.  Below, codes are multiples of
// 2^-9.  A positive y stays at least at the smallest code.
constexpr uint32_t kCodeNan = 0x7Fu;
__device__ __forceinline__ uint32_t encode_random_high(float y, uint32_t u20) {
  return min(((__float_as_uint(y) + u20) >> 20) - ((127u - 7u) << 3), 0x7Eu);
}
__device__ __forceinline__ uint32_t encode_random(float y, uint32_t u20) {
  if (y >= 0x1p-6f) return encode_random_high(y, u20);
  return static_cast<uint32_t>(
      __fadd_rn(__fmul_rn(fmaxf(y, 0x1p-9f), 512.f), __fmul_rn(static_cast<float>(u20), 0x1p-20f)));
}

// What a lane holds of its warp's group of 128 elements: four of them.
struct Group8 {
  uint4 graw;
  float p[4];
  uint32_t mw, vw;
  float ms, vs;
};

// The quotients and scales of a group (a whole warp's) that holds infinities or
// whose largest values are so small that a residual could underflow, or that
// root2's misses would count.  An infinite scale would make the group's other
// elements NaN or infinite at the next step: a v beyond FP32 has a root within it,
// formed here from values 2^-80 times as large, and what has not is held as the
// largest finite value.  (Apart, as its code between the usual groups' cost 3%:
// 268 million elements 737 us against 715.)
struct Scaled8 {
  float4 m, r;
  float m_scale, r_scale;
};
// Four values, divided by their group's scale: the largest times 1/448.
__device__ __forceinline__ float scale_to(float (&x)[4], float largest) {
  const float scale = __fmul_rn(largest, 1.f / 448.f), up = largest > 1e-25f ? 1.f : 0x1p90f;
  const float by = __fmul_rn(scale, up), inv = __frcp_rn(by);
#pragma unroll
  for (int h = 0; h < 4; h += 2) {
    const float2 q = quotient2(__fmul2_rn(make_float2(x[h], x[h + 1]), both(up)), by, inv);
    // (zero, or a NaN, without a scale)
    x[h] = scale > 0.f ? q.x : x[h] * 0.f;
    x[h + 1] = scale > 0.f ? q.y : x[h + 1] * 0.f;
  }
  return scale;
}
__device__ __noinline__ Scaled8 scale_unusual(const AdamParams& a, float4 m4, float4 r4, uint32_t old_codes,
                                              float old_scale, float4 g4, float gs) {
  float m[4] = {m4.x, m4.y, m4.z, m4.w}, r[4] = {r4.x, r4.y, r4.z, r4.w};
  const float g[4] = {g4.x, g4.y, g4.z, g4.w};
  float mmax = 0.f, rmax = 0.f;
#pragma unroll
  for (int h = 0; h < 4; h += 2) {
    const float2 ro = __fmul2_rn(e4m3x2_to_f32(old_codes >> (8 * h) & 0xFFFFu), both(old_scale));
    const float2 gj = __fmul2_rn(make_float2(g[h], g[h + 1]), both(gs));
    const float2 v = second_moment(a, gj, __fmul2_rn(ro, ro));
    const float2 x = __fmul2_rn(ro, both(0x1p-80f)), y = __fmul2_rn(gj, both(0x1p-80f));
    const float2 far = second_moment(a, y, __fmul2_rn(x, x)), near = root2<true>(v);
    // (r is zero past the tensor's end)
    if (r[h] > 0.f) r[h] = v.x > FLT_MAX ? fminf(__fsqrt_rn(far.x) * 0x1p80f, FLT_MAX) : near.x;
    if (r[h + 1] > 0.f) r[h + 1] = v.y > FLT_MAX ? fminf(__fsqrt_rn(far.y) * 0x1p80f, FLT_MAX) : near.y;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (fabsf(m[j]) > FLT_MAX) m[j] = copysignf(FLT_MAX, m[j]);
    mmax = fmaxf(mmax, fabsf(m[j]));
    rmax = fmaxf(rmax, r[j]);
  }
  Scaled8 o;
  o.m_scale = scale_to(m, __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mmax))));
  o.r_scale = scale_to(r, __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(rmax))));
  o.m = make_float4(m[0], m[1], m[2], m[3]);
  o.r = make_float4(r[0], r[1], r[2], r[3]);
  return o;
}

template <bool kWhole, bool kSmall>
__device__ __forceinline__ void adamw8_group(const AdamParams& a, const AdamEntry& t, float decay, float gs,
                                             uint32_t tensor, int64_t group, Group8& x, const float (&g)[4], int have) {
  const int lane = threadIdx.x % 32;
  const int64_t i = group * 128 + 4 * lane;
  uint8_t* mc = static_cast<uint8_t*>(t.m);
  uint8_t* vc = static_cast<uint8_t*>(t.v);
  float m[4], r[4];
  float mmax = 0.f, rmax = 0.f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float2 mo = __fmul2_rn(e4m3x2_to_f32(x.mw >> (16 * h) & 0xFFFFu), both(x.ms));
    const float2 ro = __fmul2_rn(e4m3x2_to_f32(x.vw >> (16 * h) & 0xFFFFu), both(x.vs));
    const Elem2 e = adam_elem2<kSmall>(a, decay, __fmul2_rn(make_float2(g[2 * h], g[2 * h + 1]), both(gs)),
                               make_float2(x.p[2 * h], x.p[2 * h + 1]), mo, __fmul2_rn(ro, ro));
    const bool in0 = kWhole || 2 * h < have, in1 = kWhole || 2 * h + 1 < have;
    m[2 * h] = in0 ? e.m.x : 0.f;
    m[2 * h + 1] = in1 ? e.m.y : 0.f;
    r[2 * h] = in0 ? e.r.x : 0.f;
    r[2 * h + 1] = in1 ? e.r.y : 0.f;
    x.p[2 * h] = e.p.x;
    x.p[2 * h + 1] = e.p.y;
    mmax = fmaxf(mmax, fmaxf(fabsf(m[2 * h]), fabsf(m[2 * h + 1])));
    rmax = fmaxf(rmax, fmaxf(r[2 * h], r[2 * h + 1]));
  }
  // (nonnegative floats order as their patterns do; fmaxf leaves a NaN out of the
  // group's largest, so that it stays in its element)
  mmax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mmax)));
  rmax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(rmax)));
  float mns = __fmul_rn(mmax, 1.f / 448.f), vns = __fmul_rn(rmax, 1.f / 448.f);
  float mq[4], y[4];
  bool zeros = false;
  // (8e-14: a v below 1e-37, whose root root2 misses, then gets the smallest code
  // either way; a tensor of nothing but smaller roots takes 1397 us instead of 715)
  if ((mmax > 1e-25f || mmax == 0.f) && rmax > (kSmall ? 1e-25f : 8e-14f) && fmaxf(mmax, rmax) <= FLT_MAX) {
    // (m is zero, its root not, where an expert has had no rows for long: 0 / 0 is 0 here)
    const float mi = mmax > 0.f ? __frcp_rn(mns) : 0.f, vi = __frcp_rn(vns);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float2 q = quotient2(make_float2(m[2 * h], m[2 * h + 1]), mns, mi);
      const float2 z = quotient2(make_float2(r[2 * h], r[2 * h + 1]), vns, vi);
      mq[2 * h] = q.x;
      mq[2 * h + 1] = q.y;
      y[2 * h] = z.x;
      y[2 * h + 1] = z.y;
    }
  } else if (__all_sync(0xffffffffu, m[0] == 0.f && m[1] == 0.f && m[2] == 0.f && m[3] == 0.f && r[0] == 0.f &&
                                         r[1] == 0.f && r[2] == 0.f && r[3] == 0.f)) {
    zeros = true;
#pragma unroll
    for (int j = 0; j < 4; ++j) mq[j] = y[j] = 0.f;
  } else {
    const Scaled8 o = scale_unusual(a, make_float4(m[0], m[1], m[2], m[3]), make_float4(r[0], r[1], r[2], r[3]), x.vw,
                                    x.vs, make_float4(g[0], g[1], g[2], g[3]), gs);
    mq[0] = o.m.x; mq[1] = o.m.y; mq[2] = o.m.z; mq[3] = o.m.w;
    y[0] = o.r.x; y[1] = o.r.y; y[2] = o.r.z; y[3] = o.r.w;
    mns = o.m_scale;
    vns = o.r_scale;
  }
  if (lane == 0) {
    t.m_scale[group] = mns;
    t.v_scale[group] = vns;
  }
  const uint32_t key = random_key(a.seed, tensor, i);
  uint32_t vo = 0;
  if (__all_sync(0xffffffffu, min_nan(min_nan(y[0], y[1]), min_nan(y[2], y[3])) >= 0x1p-6f)) {
    // (roots within a factor of 28672 of the group's largest, no NaN: the usual case)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      vo |= encode_random_high(y[j], random20(key, static_cast<uint32_t>(i) + j)) << (8 * j);
  } else if (!zeros) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t code = encode_random(y[j], random20(key, static_cast<uint32_t>(i) + j));
      vo |= (isnan(r[j]) ? kCodeNan : r[j] > 0.f && vns > 0.f ? code : 0u) << (8 * j);
    }
  }
  const uint32_t mo = cvt_e4m3x2(mq[0], mq[1]) | (static_cast<uint32_t>(cvt_e4m3x2(mq[2], mq[3])) << 16);
  if (kWhole) {
    __stcs(reinterpret_cast<float4*>(t.param + i), make_float4(x.p[0], x.p[1], x.p[2], x.p[3]));
    __stcs(reinterpret_cast<uint32_t*>(mc + i), mo);
    __stcs(reinterpret_cast<uint32_t*>(vc + i), vo);
    if (t.model) *reinterpret_cast<uint2*>(t.model + i) = model4(t, x.p);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j >= have) continue;
      t.param[i + j] = x.p[j];
      mc[i + j] = static_cast<uint8_t>(mo >> (8 * j));
      vc[i + j] = static_cast<uint8_t>(vo >> (8 * j));
      const float one[4] = {x.p[j], 0.f, 0.f, 0.f};
      if (t.model) t.model[i + j] = static_cast<uint16_t>(model4(t, one).x & 0xFFFFu);
    }
  }
}

template <int kGrad>
__device__ __forceinline__ void load_group8(const AdamEntry& t, int64_t group, Group8& x) {
  const int64_t i = group * 128 + 4 * (threadIdx.x % 32);
  const bool ok = (group + 1) * 128 <= t.n && MOE_IN_BOUNDS(group >= 0);
  x.graw = load_grad4<kGrad>(t, i, ok);
  float4 p4 = {};
  if (ok) p4 = __ldcs(reinterpret_cast<const float4*>(t.param + i));
  x.p[0] = p4.x; x.p[1] = p4.y; x.p[2] = p4.z; x.p[3] = p4.w;
  if (ok) x.mw = __ldcs(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(t.m) + i));
  if (ok) x.vw = __ldcs(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(t.v) + i));
  if (ok) x.ms = t.m_scale[group];
  if (ok) x.vs = t.v_scale[group];
}

// (apart, so that its registers are not the loop's)
template <bool kSmall>
__device__ __noinline__ void adamw8_last(const AdamParams& a, float decay, float gs, uint32_t tensor) {
  const AdamEntry t = a.table[tensor];
  const int lane = threadIdx.x % 32;
  const int64_t group = t.n / 128, i = group * 128 + 4 * lane;
  if (!MOE_IN_BOUNDS(tensor < static_cast<uint32_t>(a.count) && t.n % 128)) return;   // (a scale for the group)
  const int have = t.n - i >= 4 ? 4 : t.n > i ? static_cast<int>(t.n - i) : 0;
  Group8 x = {};
  float g[4] = {};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (j >= have) continue;
    g[j] = load_grad1(t, i + j);
    x.p[j] = t.param[i + j];
    x.mw |= static_cast<uint32_t>(static_cast<const uint8_t*>(t.m)[i + j]) << (8 * j);
    x.vw |= static_cast<uint32_t>(static_cast<const uint8_t*>(t.v)[i + j]) << (8 * j);
  }
  x.ms = t.m_scale[group];
  x.vs = t.v_scale[group];
  __syncwarp();   // (lane 0 rewrites the scales that every lane has read)
  adamw8_group<false, kSmall>(a, t, decay, gs, tensor, group, x, g, have);
}

// While a CTA computes a chunk, its next chunk's loads are in flight (where
// that is of the same tensor): with loads and arithmetic in turn the warps
// mostly waited.  The CTAs walk the chunks side by side, not each a stretch of
// its own: a thousand separate streams cost the translation of as many pages.
template <int kGrad, bool kSmall>
__global__ void __launch_bounds__(kThreads, 3) adamw8_kernel(const __grid_constant__ AdamParams a) {
  pdl_wait();
  if (a.skip && *a.skip) return;
  const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
  const int warp = threadIdx.x / 32;
  constexpr int kWarps = kThreads / 32;
  int64_t c = blockIdx.x;
  while (c < a.chunks) {
    const int index = find_entry(a, c);
    const AdamEntry t = a.table[index];
    const int64_t past = t.first_chunk + (t.n + kChunk - 1) / kChunk;   // the tensor's chunks end here
    if (c >= past) return;   // (more chunks than the table has)
    const float decay = fmaf(-a.lr, t.weight_decay, 1.0f);
    const uint32_t id = static_cast<uint32_t>(index);
    Group8 next[kSteps];
    int64_t group = (c - t.first_chunk) * (kChunk / 128) + warp;
    if (t.kind == kGrad + kEightBits) {
#pragma unroll
      for (int u = 0; u < kSteps; ++u) load_group8<kGrad>(t, group + u * kWarps, next[u]);
    }
    for (; c < past; c += gridDim.x) {
      if (t.kind != kGrad + kEightBits) continue;
      Group8 x[kSteps];
#pragma unroll
      for (int u = 0; u < kSteps; ++u) x[u] = next[u];
      const int64_t ahead = group + static_cast<int64_t>(gridDim.x) * (kChunk / 128);
      if (c + gridDim.x < past) {
#pragma unroll
        for (int u = 0; u < kSteps; ++u) load_group8<kGrad>(t, ahead + u * kWarps, next[u]);
      }
#pragma unroll
      for (int u = 0; u < kSteps; ++u) {
        if ((group + u * kWarps + 1) * 128 > t.n || !MOE_IN_BOUNDS(index >= 0 && index < a.count && group >= 0)) continue;
        float g[4];
        grad4<kGrad>(x[u].graw, g);
        adamw8_group<true, kSmall>(a, t, decay, gs, id, group + u * kWarps, x[u], g, 4);
      }
      // a partly filled last group
      if (c + 1 == past && t.n % 128 && warp == 0) adamw8_last<kSmall>(a, decay, gs, id);
      group = ahead;
    }
  }
}

using AdamKernel = void (*)(AdamParams);
template <bool kSmall>
AdamKernel adamw_kernel_of(int type, int state_bits) {
  if (state_bits == 32)
    return type == MOE_TYPE_BF16   ? adamw32_kernel<MOE_TYPE_BF16, kSmall>
           : type == MOE_TYPE_FP16 ? adamw32_kernel<MOE_TYPE_FP16, kSmall>
                                   : adamw32_kernel<MOE_TYPE_FP32, kSmall>;
  return type == MOE_TYPE_BF16   ? adamw8_kernel<MOE_TYPE_BF16, kSmall>
         : type == MOE_TYPE_FP16 ? adamw8_kernel<MOE_TYPE_FP16, kSmall>
                                 : adamw8_kernel<MOE_TYPE_FP32, kSmall>;
}
AdamKernel adamw_kernel(int type, int state_bits, bool small) {
  return small ? adamw_kernel_of<true>(type, state_bits) : adamw_kernel_of<false>(type, state_bits);
}

}  // namespace
}  // namespace moe

extern "C" {

size_t moe_adamw_table_bytes(int count) {
  if (count < 1 || count > 65536) return 0;
  return static_cast<size_t>(count) * sizeof(moe::AdamEntry);
}

moe_status moe_adamw_table_init(const moe_adamw_tensor* tensors, int count, int state_bits, void* table,
                                size_t table_bytes, int64_t* chunks, int32_t* grad_types, moe_stream_t stream) {
  using namespace moe;
  if (state_bits != 32 && state_bits != 8) return MOE_ERR_DTYPE;
  if (count < 1 || count > 65536) return MOE_ERR_SHAPE;
  if (!tensors || !table || !chunks || !grad_types) return MOE_ERR_NULL;
  if (!aligned16(table)) return MOE_ERR_ALIGN;
  if (table_bytes < moe_adamw_table_bytes(count)) return MOE_ERR_CAPACITY;
  int64_t total = 0;
  int32_t types = 0;
  std::vector<AdamEntry> host;
  try {
    host.resize(static_cast<size_t>(count));
  } catch (const std::bad_alloc&) {
    return MOE_ERR_CAPACITY;
  }
  for (int i = 0; i < count; ++i) {
    const moe_adamw_tensor& t = tensors[i];
    if (t.n < 0 || t.n >= (int64_t(1) << 46) || !std::isfinite(t.weight_decay)) return MOE_ERR_SHAPE;
    if (!is_type(t.grad_dtype) || (t.model && !is_half_type(t.model_dtype))) return MOE_ERR_DTYPE;
    if (t.n > 0) {
      if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq) return MOE_ERR_NULL;
      if (state_bits == 8 && (!t.exp_avg_scale || !t.exp_avg_sq_scale)) return MOE_ERR_NULL;
      if (!aligned16(t.param) || !aligned16(t.model) || !aligned16(t.grad) || !aligned16(t.exp_avg) ||
          !aligned16(t.exp_avg_sq) || !aligned4(t.exp_avg_scale, t.exp_avg_sq_scale))
        return MOE_ERR_ALIGN;
    }
    AdamEntry& e = host[static_cast<size_t>(i)];
    e.param = t.param;
    e.model = t.model;
    e.grad = t.grad;
    e.m = t.exp_avg;
    e.v = t.exp_avg_sq;
    e.m_scale = t.exp_avg_scale;
    e.v_scale = t.exp_avg_sq_scale;
    e.n = t.n;
    e.first_chunk = total;
    e.weight_decay = static_cast<float>(t.weight_decay);
    e.kind = t.grad_dtype + (state_bits == 8 ? kEightBits : 0);
    e.model_dtype = t.model ? t.model_dtype : MOE_TYPE_BF16;
    total += ceil_div(t.n, kChunk);
    if (t.n > 0) types |= 1 << t.grad_dtype;
  }
  DeviceInfo dev;
  if (current_device(&dev) != MOE_OK) return MOE_ERR_CUDA;
  if (!on_device(table, dev.device)) return MOE_ERR_DEVICE;
  for (int i = 0; i < count; ++i) {
    const AdamEntry& e = host[static_cast<size_t>(i)];
    if (e.n == 0) continue;
    const void* ptrs[] = {e.param, e.model, e.grad, e.m, e.v, state_bits == 8 ? e.m_scale : nullptr,
                          state_bits == 8 ? e.v_scale : nullptr};
    for (const void* p : ptrs)
      if (p && !on_device(p, dev.device)) return MOE_ERR_DEVICE;
  }
  // from pageable memory: staged before the call returns
  MOE_CUDA_TRY(cudaMemcpyAsync(table, host.data(), host.size() * sizeof(AdamEntry), cudaMemcpyHostToDevice, stream));
  MOE_CUDA_TRY(cudaStreamSynchronize(stream));
  *chunks = total;
  *grad_types = types;
  return MOE_OK;
}

moe_status moe_adamw_step(const moe_adamw_args* g, moe_stream_t stream) {
  using namespace moe;
  if (!g) return MOE_ERR_NULL;
  if (g->state_bits != 32 && g->state_bits != 8) return MOE_ERR_DTYPE;
  if (g->count < 1 || g->count > 65536 || g->chunks < 0 || g->grad_types < 0 || g->grad_types > 7 || g->step < 1 || !(g->lr >= 0) || !std::isfinite(g->lr) ||
      !(g->eps >= 0) || !std::isfinite(g->eps) || !(g->beta1 >= 0 && g->beta1 < 1) ||
      !(g->beta2 >= 0 && g->beta2 < 1))
    return MOE_ERR_SHAPE;
  if (!g->table) return MOE_ERR_NULL;
  if (!aligned16(g->table) || !aligned4(g->grad_scale, g->skip)) return MOE_ERR_ALIGN;
  if (g->chunks == 0) return MOE_OK;
  DeviceInfo dev;
  if (current_device(&dev) != MOE_OK) return MOE_ERR_CUDA;
  if (!on_device(g->table, dev.device) || (g->grad_scale && !on_device(g->grad_scale, dev.device)) ||
      (g->skip && !on_device(g->skip, dev.device)))
    return MOE_ERR_DEVICE;
  AdamParams p;
  p.table = static_cast<const AdamEntry*>(g->table);
  p.grad_scale = g->grad_scale;
  p.skip = g->skip;
  p.chunks = g->chunks;
  p.lr = static_cast<float>(g->lr);
  p.beta1 = static_cast<float>(g->beta1);
  p.one_minus_beta1 = static_cast<float>(1.0 - g->beta1);
  p.beta2 = static_cast<float>(g->beta2);
  p.one_minus_beta2 = static_cast<float>(1.0 - g->beta2);
  const double n = static_cast<double>(g->step);
  p.step_size = static_cast<float>(g->lr / (1.0 - std::pow(g->beta1, n)));
  p.root_scale = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(g->beta2, n)));
  p.eps = static_cast<float>(g->eps);
  p.seed = g->seed;
  p.count = g->count;
  // 8-bit states: as many CTAs as are resident at once.  32-bit states: about three
  // times the five or six that are (80-92 registers a thread); measured side by side
  // at 268 million elements, 16 CTAs an SM took 1153 us, five 1195, six 1314, ten 1196.
  const int64_t most = static_cast<int64_t>(dev.sms) * (g->state_bits == 32 ? 16 : 3);
  const unsigned grid = static_cast<unsigned>(g->chunks < most ? g->chunks : most);
  // The update's denominator is sqrt(v) root_scale + eps.  Roots that root2 misses
  // without kSmall are below 3.2e-19 (their v below 1e-37), so from this eps on they
  // change no more than its last bit.
  const bool small = p.eps < 6e-12f * p.root_scale;
  // a kernel for each type of gradient that the table holds
  for (int type = 0; type < 3; ++type) {
    if (!(g->grad_types >> type & 1)) continue;
    const auto kernel = adamw_kernel(type, g->state_bits, small);
    MOE_CUDA_TRY(launch_pdl(kernel, dim3(grid), dim3(kThreads), 0, stream, 1, p));
  }
  return MOE_OK;
}

}  // extern "C"

MOE_BOUNDS_TU()
