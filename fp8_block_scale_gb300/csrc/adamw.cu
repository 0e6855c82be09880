// One AdamW step over many tensors in one launch (moe_adamw_step).
//
// A device table lists the tensors; each is cut into chunks of 4096 elements
// and the CTAs walk the chunks of all tensors, so that a list of small
// tensors costs one launch.  Per element the step reads the gradient, the
// parameter and both states once and writes the parameter, its 16-bit copy
// and the states once: HBM bounds it.
//
// The arithmetic is FP32.
#include <cmath>
#include <mutex>
#include <new>
#include <vector>

#include "train.cuh"

namespace moe {
namespace {

constexpr int kChunk = 4096;   // elements per chunk
constexpr int kThreads = 256;
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
  double weight_decay;
  int32_t grad_dtype;
  int32_t model_dtype;
};

struct AdamParams {
  const AdamEntry* table;
  const float* grad_scale;
  const int32_t* skip;
  int64_t chunks;
  double lr;
  float beta1, one_minus_beta1, beta2, one_minus_beta2;
  float step_size;   // lr / (1 - beta1^step)
  float root_scale;  // 1 / sqrt(1 - beta2^step)
  float eps;
  uint32_t seed;
  int count;
};

// The new m, v, root of v and parameter of one element.  m and v are rounded
// once per written operation; the root and the quotient of the update come
// from the hardware's approximations (within 2 units of the last place of the
// update, which is far below the parameter's own rounding).
struct Elem {
  float m, v, r, p;
};
__device__ __forceinline__ float sqrt_fast(float v) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp_fast(float v) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ Elem adam_elem(const AdamParams& a, float decay, float g, float p, float m, float v) {
  Elem e;
  e.m = __fadd_rn(__fmul_rn(m, a.beta1), __fmul_rn(g, a.one_minus_beta1));
  e.v = __fadd_rn(__fmul_rn(v, a.beta2), __fmul_rn(__fmul_rn(g, g), a.one_minus_beta2));
  e.r = sqrt_fast(e.v);
  const float den = fmaf(e.r, a.root_scale, a.eps);
  e.p = __fsub_rn(__fmul_rn(p, decay), __fmul_rn(__fmul_rn(e.m, a.step_size), rcp_fast(den)));
  return e;
}

// Four gradients; kGrad = -1: of a type known at run time.
template <int kGrad>
__device__ __forceinline__ void load_grad4(const AdamEntry& t, int64_t i, float (&g)[4]) {
  const int type = kGrad >= 0 ? kGrad : t.grad_dtype;
  if (type == MOE_TYPE_FP32) {
    const float4 v = __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(t.grad) + i));
    g[0] = v.x; g[1] = v.y; g[2] = v.z; g[3] = v.w;
    return;
  }
  const uint2 v = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(t.grad) + i));
  float2 a, b;
  if (type == MOE_TYPE_BF16) {
    a = Pack2<__nv_bfloat16>::load(v.x);
    b = Pack2<__nv_bfloat16>::load(v.y);
  } else {
    a = Pack2<__half>::load(v.x);
    b = Pack2<__half>::load(v.y);
  }
  g[0] = a.x; g[1] = a.y; g[2] = b.x; g[3] = b.y;
}
__device__ __forceinline__ float load_grad1(const AdamEntry& t, int64_t i) {
  if (t.grad_dtype == MOE_TYPE_FP32) return static_cast<const float*>(t.grad)[i];
  const uint32_t v = static_cast<const uint16_t*>(t.grad)[i];
  return t.grad_dtype == MOE_TYPE_BF16 ? Pack2<__nv_bfloat16>::load(v).x : Pack2<__half>::load(v).x;
}
__device__ __forceinline__ uint2 model4(const AdamEntry& t, const float (&p)[4]) {
  if (t.model_dtype == MOE_TYPE_BF16)
    return make_uint2(Pack2<__nv_bfloat16>::store(p[0], p[1]), Pack2<__nv_bfloat16>::store(p[2], p[3]));
  return make_uint2(Pack2<__half>::store(p[0], p[1]), Pack2<__half>::store(p[2], p[3]));
}

// The table entry that holds chunk c (whole warps): 32 entries are compared at
// a time, so a list of 1024 tensors takes two dependent loads.
__device__ __forceinline__ int find_entry(const AdamParams& a, int64_t c) {
  int lo = 0, n = a.count;   // table[lo].first_chunk <= c; the entry is in [lo, lo + n)
  while (n > 1) {
    const int stride = (n + 31) / 32, i = lo + static_cast<int>(threadIdx.x % 32) * stride;
    const unsigned le = __ballot_sync(0xffffffffu, i < lo + n && a.table[min(i, a.count - 1)].first_chunk <= c);
    const int k = 31 - __clz(le | 1u);
    const int end = min(lo + n, lo + (k + 1) * stride);
    lo += k * stride;
    n = end - lo;
  }
  return lo;
}

// ---------------------------------------------------------------- 32-bit states

template <int kGrad>
__device__ __forceinline__ void adamw32_chunk(const AdamParams& a, const AdamEntry& t, float decay, float gs,
                                              int64_t i0) {
  // every load of the chunk goes out before the first result is needed
  float g[kSteps][4];
  float4 p4[kSteps], m4[kSteps], v4[kSteps];
  float* m = static_cast<float*>(t.m);
  float* v = static_cast<float*>(t.v);
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const int64_t i = i0 + 4 * (threadIdx.x + u * kThreads);
    load_grad4<kGrad>(t, i, g[u]);
    p4[u] = __ldcs(reinterpret_cast<const float4*>(t.param + i));
    m4[u] = __ldcs(reinterpret_cast<const float4*>(m + i));
    v4[u] = __ldcs(reinterpret_cast<const float4*>(v + i));
  }
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const int64_t i = i0 + 4 * (threadIdx.x + u * kThreads);
    float p[4];
    const float po[4] = {p4[u].x, p4[u].y, p4[u].z, p4[u].w};
    float* mp = &m4[u].x;
    float* vp = &v4[u].x;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const Elem e = adam_elem(a, decay, __fmul_rn(g[u][j], gs), po[j], mp[j], vp[j]);
      p[j] = e.p;
      mp[j] = e.m;
      vp[j] = e.v;
    }
    __stcs(reinterpret_cast<float4*>(t.param + i), make_float4(p[0], p[1], p[2], p[3]));
    __stcs(reinterpret_cast<float4*>(m + i), m4[u]);
    __stcs(reinterpret_cast<float4*>(v + i), v4[u]);
    if (t.model) *reinterpret_cast<uint2*>(t.model + i) = model4(t, p);
  }
}

__global__ void __launch_bounds__(kThreads) adamw32_kernel(const AdamParams a) {
  pdl_wait();
  if (a.skip && *a.skip) return;
  const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
  for (int64_t c = blockIdx.x; c < a.chunks; c += gridDim.x) {
    const AdamEntry t = a.table[find_entry(a, c)];
    const float decay = static_cast<float>(1.0 - a.lr * t.weight_decay);
    const int64_t i0 = (c - t.first_chunk) * kChunk;
    if (i0 + kChunk <= t.n) {
      if (t.grad_dtype == MOE_TYPE_FP32) adamw32_chunk<MOE_TYPE_FP32>(a, t, decay, gs, i0);
      else if (t.grad_dtype == MOE_TYPE_BF16) adamw32_chunk<MOE_TYPE_BF16>(a, t, decay, gs, i0);
      else adamw32_chunk<MOE_TYPE_FP16>(a, t, decay, gs, i0);
      continue;
    }
    // a tensor's last chunk, one element a thread and step
    float* m = static_cast<float*>(t.m);
    float* v = static_cast<float*>(t.v);
    for (int64_t k = i0 + threadIdx.x; k < t.n; k += kThreads) {
      const Elem e = adam_elem(a, decay, __fmul_rn(load_grad1(t, k), gs), t.param[k], m[k], v[k]);
      t.param[k] = e.p;
      m[k] = e.m;
      v[k] = e.v;
      const float p[4] = {e.p, 0.f, 0.f, 0.f};
      if (t.model) t.model[k] = static_cast<uint16_t>(model4(t, p).x & 0xFFFFu);
    }
  }
}

// ---------------------------------------------------------------- 8-bit states

// Twenty bits for one element: an integer hash (two multiply-xorshift rounds)
// of seed, tensor and element; `key` is what the elements of 2^32 share.
__device__ __forceinline__ uint32_t random_key(uint32_t seed, uint32_t tensor, int64_t i) {
  return static_cast<uint32_t>(i >> 32) * 0x85EBCA77u + seed + 0x9E3779B9u * (tensor + 1u);
}
__device__ __forceinline__ uint32_t random20(uint32_t key, uint32_t i) {
  uint32_t x = i * 0x9E3779B1u + key;
  x = (x ^ (x >> 16)) * 0x7FEB352Du;
  x = (x ^ (x >> 15)) * 0x846CA68Bu;
  return (x ^ (x >> 16)) >> 12;
}

// E4M3 code of y in [0, 448.x], rounded up with probability (part cut off) /
// (code spacing).  From 2^-6 on the spacing is 2^20 units of the FP32 pattern
// (three mantissa bits stay), so the random bits are added below it and cut
// off; the exponent's bias goes from 127 to 7.  Below, codes are multiples of
// 2^-9.  A positive y stays at least at the smallest code.
__device__ __forceinline__ uint32_t encode_random(float y, uint32_t u20) {
  const uint32_t high = min(((__float_as_uint(y) + u20) >> 20) - ((127u - 7u) << 3), 0x7Eu);
  const uint32_t low = static_cast<uint32_t>(
      __fadd_rn(__fmul_rn(fmaxf(y, 0x1p-9f), 512.f), __fmul_rn(static_cast<float>(u20), 0x1p-20f)));
  return y >= 0x1p-6f ? high : low;
}

// A warp's groups of 128 elements (four a lane), kGroups at once.
struct Group8 {
  float g[4], p[4];
  uint32_t mw, vw;
  float ms, vs;
};
template <bool kWhole>
__device__ __forceinline__ void adamw8_group(const AdamParams& a, const AdamEntry& t, float decay, float gs,
                                             uint32_t tensor, int64_t group, Group8& x, int have) {
  const int lane = threadIdx.x % 32;
  const int64_t i = group * 128 + 4 * lane;
  uint8_t* mc = static_cast<uint8_t*>(t.m);
  uint8_t* vc = static_cast<uint8_t*>(t.v);
  float m[4], r[4];
  const float2 ma = e4m3x2_to_f32(x.mw & 0xFFFFu), mb = e4m3x2_to_f32(x.mw >> 16);
  const float2 va = e4m3x2_to_f32(x.vw & 0xFFFFu), vb = e4m3x2_to_f32(x.vw >> 16);
  m[0] = ma.x; m[1] = ma.y; m[2] = mb.x; m[3] = mb.y;
  r[0] = va.x; r[1] = va.y; r[2] = vb.x; r[3] = vb.y;
  float mmax = 0.f, rmax = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float ro = __fmul_rn(r[j], x.vs);
    const Elem e = adam_elem(a, decay, __fmul_rn(x.g[j], gs), x.p[j], __fmul_rn(m[j], x.ms), __fmul_rn(ro, ro));
    const bool in = kWhole || j < have;
    m[j] = in ? e.m : 0.f;
    r[j] = in ? e.r : 0.f;
    x.p[j] = e.p;
    mmax = fmaxf(mmax, fabsf(m[j]));
    rmax = fmaxf(rmax, r[j]);
  }
  // (nonnegative floats order as their patterns do)
  mmax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mmax)));
  rmax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(rmax)));
  const float mns = __fdiv_rn(mmax, 448.f), vns = __fdiv_rn(rmax, 448.f);
  if (lane == 0) {
    t.m_scale[group] = mns;
    t.v_scale[group] = vns;
  }
  float mq[4], y[4];
  if (fminf(mmax, rmax) > 1e-30f) {
    // one reciprocal per group: the quotients are within two units of the last place
    const float mi = __fdiv_rn(448.f, mmax), vi = __fdiv_rn(448.f, rmax);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      mq[j] = __fmul_rn(m[j], mi);
      y[j] = __fmul_rn(r[j], vi);
    }
  } else {   // zeros, or values whose reciprocal could overflow
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      mq[j] = mns > 0.f ? __fdiv_rn(m[j], mns) : 0.f;
      y[j] = vns > 0.f ? __fdiv_rn(r[j], vns) : 0.f;
    }
  }
  const uint32_t key = random_key(a.seed, tensor, i);
  uint32_t vo = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t code = encode_random(y[j], random20(key, static_cast<uint32_t>(i) + j));
    vo |= (r[j] > 0.f && vns > 0.f ? code : 0u) << (8 * j);
  }
  const uint32_t mo = cvt_e4m3x2(mq[0], mq[1]) | (static_cast<uint32_t>(cvt_e4m3x2(mq[2], mq[3])) << 16);
  if (kWhole) {
    __stcs(reinterpret_cast<float4*>(t.param + i), make_float4(x.p[0], x.p[1], x.p[2], x.p[3]));
    __stcs(reinterpret_cast<uint32_t*>(mc + i), mo);
    __stcs(reinterpret_cast<uint32_t*>(vc + i), vo);
    if (t.model) *reinterpret_cast<uint2*>(t.model + i) = model4(t, x.p);
  } else {
    for (int j = 0; j < have; ++j) {
      t.param[i + j] = x.p[j];
      mc[i + j] = static_cast<uint8_t>(mo >> (8 * j));
      vc[i + j] = static_cast<uint8_t>(vo >> (8 * j));
      const float one[4] = {x.p[j], 0.f, 0.f, 0.f};
      if (t.model) t.model[i + j] = static_cast<uint16_t>(model4(t, one).x & 0xFFFFu);
    }
  }
}

template <int kGrad>
__device__ __forceinline__ void adamw8_chunk(const AdamParams& a, const AdamEntry& t, float decay, float gs,
                                             uint32_t tensor, int64_t group0) {
  const int lane = threadIdx.x % 32;
  Group8 x[kSteps];
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const int64_t group = group0 + u * (kThreads / 32), i = group * 128 + 4 * lane;
    load_grad4<kGrad>(t, i, x[u].g);
    const float4 p4 = __ldcs(reinterpret_cast<const float4*>(t.param + i));
    x[u].p[0] = p4.x; x[u].p[1] = p4.y; x[u].p[2] = p4.z; x[u].p[3] = p4.w;
    x[u].mw = __ldcs(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(t.m) + i));
    x[u].vw = __ldcs(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(t.v) + i));
    x[u].ms = t.m_scale[group];
    x[u].vs = t.v_scale[group];
  }
#pragma unroll
  for (int u = 0; u < kSteps; ++u)
    adamw8_group<true>(a, t, decay, gs, tensor, group0 + u * (kThreads / 32), x[u], 4);
}

__global__ void __launch_bounds__(kThreads) adamw8_kernel(const AdamParams a) {
  pdl_wait();
  if (a.skip && *a.skip) return;
  const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  for (int64_t c = blockIdx.x; c < a.chunks; c += gridDim.x) {
    const int index = find_entry(a, c);
    const AdamEntry t = a.table[index];
    const float decay = static_cast<float>(1.0 - a.lr * t.weight_decay);
    const int64_t group0 = (c - t.first_chunk) * (kChunk / 128) + warp;
    if ((c - t.first_chunk + 1) * kChunk <= t.n) {
      if (t.grad_dtype == MOE_TYPE_FP32) adamw8_chunk<MOE_TYPE_FP32>(a, t, decay, gs, index, group0);
      else if (t.grad_dtype == MOE_TYPE_BF16) adamw8_chunk<MOE_TYPE_BF16>(a, t, decay, gs, index, group0);
      else adamw8_chunk<MOE_TYPE_FP16>(a, t, decay, gs, index, group0);
      continue;
    }
    // a tensor's last chunk: a group at a time, the last one partly filled
    for (int64_t group = group0; group * 128 < t.n && group < (c - t.first_chunk + 1) * (kChunk / 128);
         group += kThreads / 32) {
      const int64_t i = group * 128 + 4 * lane;
      const int have = t.n - i >= 4 ? 4 : t.n > i ? static_cast<int>(t.n - i) : 0;
      Group8 x = {};
      for (int j = 0; j < have; ++j) {
        x.g[j] = load_grad1(t, i + j);
        x.p[j] = t.param[i + j];
        x.mw |= static_cast<uint32_t>(static_cast<const uint8_t*>(t.m)[i + j]) << (8 * j);
        x.vw |= static_cast<uint32_t>(static_cast<const uint8_t*>(t.v)[i + j]) << (8 * j);
      }
      x.ms = t.m_scale[group];
      x.vs = t.v_scale[group];
      __syncwarp();   // (lane 0 rewrites the scales that every lane has read)
      adamw8_group<false>(a, t, decay, gs, static_cast<uint32_t>(index), group, x, have);
    }
  }
}

}  // namespace
}  // namespace moe

extern "C" {

size_t moe_adamw_table_bytes(int count) {
  if (count < 1 || count > 65536) return 0;
  return static_cast<size_t>(count) * sizeof(moe::AdamEntry);
}

moe_status moe_adamw_table_init(const moe_adamw_tensor* tensors, int count, int state_bits, void* table,
                                size_t table_bytes, int64_t* chunks, moe_stream_t stream) {
  using namespace moe;
  if (state_bits != 32 && state_bits != 8) return MOE_ERR_DTYPE;
  if (count < 1 || count > 65536) return MOE_ERR_SHAPE;
  if (!tensors || !table || !chunks) return MOE_ERR_NULL;
  if (!aligned16(table)) return MOE_ERR_ALIGN;
  if (table_bytes < moe_adamw_table_bytes(count)) return MOE_ERR_CAPACITY;
  int64_t total = 0;
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
          !aligned16(t.exp_avg_sq) || (reinterpret_cast<uintptr_t>(t.exp_avg_scale) & 3u) ||
          (reinterpret_cast<uintptr_t>(t.exp_avg_sq_scale) & 3u))
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
    e.weight_decay = t.weight_decay;
    e.grad_dtype = t.grad_dtype;
    e.model_dtype = t.model ? t.model_dtype : MOE_TYPE_BF16;
    total += ceil_div(t.n, kChunk);
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
  return MOE_OK;
}

moe_status moe_adamw_step(const moe_adamw_args* g, moe_stream_t stream) {
  using namespace moe;
  if (!g) return MOE_ERR_NULL;
  if (g->state_bits != 32 && g->state_bits != 8) return MOE_ERR_DTYPE;
  if (g->count < 1 || g->count > 65536 || g->chunks < 0 || g->step < 1 || !(g->lr >= 0) || !std::isfinite(g->lr) ||
      !(g->eps >= 0) || !std::isfinite(g->eps) || !(g->beta1 >= 0 && g->beta1 < 1) ||
      !(g->beta2 >= 0 && g->beta2 < 1))
    return MOE_ERR_SHAPE;
  if (!g->table) return MOE_ERR_NULL;
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
  p.lr = g->lr;
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
  const int64_t most = static_cast<int64_t>(dev.sms) * 8;
  const unsigned grid = static_cast<unsigned>(g->chunks < most ? g->chunks : most);
  MOE_CUDA_TRY(launch_pdl(g->state_bits == 32 ? adamw32_kernel : adamw8_kernel, dim3(grid), dim3(kThreads), 0, stream,
                          1, p));
  return MOE_OK;
}

}  // extern "C"

MOE_BOUNDS_TU()
