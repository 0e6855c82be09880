// Rows on their way to the experts and back (moe_plan_groups,
// moe_gather_rows, moe_sum_routes) and the SwiGLU gradient by rows.
//
// All of them move each byte once and compute little: HBM bounds them, so
// every access is 16 bytes wide and a row is one warp's (or CTA's) contiguous
// stretch.  (Small calls are one launch, some 3 us on the GPU.)
#include "train.cuh"

namespace moe {
namespace {

// ---------------------------------------------------------------- plan groups
//
// A plan's blocks ascend by expert, so each expert's range comes from two
// binary searches, and its count from a third over the pads of its last block;
// no counting pass and no atomics.

__global__ void __launch_bounds__(256)
    plan_groups_kernel(const int32_t* __restrict__ sorted, const int32_t* __restrict__ experts,
                       const int32_t* __restrict__ padded, int64_t blocks_cap, int block_m, int64_t R, int E,
                       int32_t* __restrict__ start, int32_t* __restrict__ rows, int32_t* __restrict__ route_slot) {
  pdl_wait();
  int64_t nb = max(*padded, 0) / block_m;
  if (nb > blocks_cap) nb = blocks_cap;
  const int64_t tid = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (tid < E) {
    // the plan's blocks ascend by expert: [first, last) are this expert's
    const int e = static_cast<int>(tid);
    int64_t lo[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      int64_t a = 0, b = nb;
      while (a < b) {
        const int64_t m = (a + b) / 2;
        if (MOE_IN_BOUNDS(m >= 0 && m < blocks_cap) && experts[m] < e + i) a = m + 1; else b = m;
      }
      lo[i] = a;
    }
    int64_t n = 0;
    if (lo[1] > lo[0]) {
      // pads fill the end of the last block
      const int32_t* ids = sorted + (lo[1] - 1) * block_m;
      int a = 0, b = block_m;
      while (a < b) {
        const int m = (a + b) / 2;
        if (MOE_IN_BOUNDS((lo[1] - 1) * block_m + m < blocks_cap * block_m) && ids[m] >= 0 && ids[m] < R)
          a = m + 1;
        else
          b = m;
      }
      n = (lo[1] - 1 - lo[0]) * block_m + a;
    }
    start[e] = n > 0 ? static_cast<int32_t>(lo[0] * block_m) : 0;
    rows[e] = static_cast<int32_t>(n);
  }
  if (route_slot) {
    const int64_t slots = nb * block_m, stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t s = tid; s < slots; s += stride) {
      const int32_t r = sorted[s];
      if (r >= 0 && r < R && MOE_IN_BOUNDS(s < blocks_cap * block_m)) route_slot[r] = static_cast<int32_t>(s);
    }
  }
}

// ---------------------------------------------------------------- gather

// One warp per slot, its lanes along the row in 16-byte vectors.  A token is
// read once per route, from L2 where the rows that stream out have not displaced
// it (8192 tokens of 8 routes: 250 of the 537 MB come from DRAM), so the stores are
// marked as streaming; that many warps are resident matters more than loads in
// flight per lane.  65536 rows of 8 KB from 8192 tokens: 116 us, 5.2 TB/s (125
// with plain stores and four loads in flight; bulk copies through shared memory
// 139); 9000 rows of 14 KB: 22 us against 29.
__global__ void __launch_bounds__(256)
    gather_rows_kernel(const uint4* __restrict__ x, int64_t M, int vecs, int64_t ldx, uint4* __restrict__ xs,
                       int64_t rows, int64_t ldxs, const int32_t* __restrict__ route_ids, int top_k,
                       const int32_t* __restrict__ num_rows) {
  pdl_wait();
  const int64_t n = num_rows ? min(static_cast<int64_t>(max(*num_rows, 0)), rows) : rows;
  const int lane = threadIdx.x % 32;
  for (int64_t s = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32; s < n;
       s += static_cast<int64_t>(gridDim.x) * 8) {
    const int32_t r = route_ids[s];
    const int64_t t = r >= 0 ? r / top_k : M;
    const bool live = t < M && MOE_IN_BOUNDS(t >= 0 && s < rows);
    const uint4* src = live ? x + t * ldx : x;
    uint4* dst = xs + s * ldxs;
    for (int v = lane; v < vecs; v += 32) __stcs(dst + v, live ? src[v] : make_uint4(0, 0, 0, 0));
  }
}

// ---------------------------------------------------------------- sum

template <typename T>
__device__ __forceinline__ void add_vec(const uint4& v, float (&acc)[8]) {
  float f[8];
  unpack8<T>(v, f);
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] += f[i];
}
template <>
__device__ __forceinline__ void add_vec<float>(const uint4& v, float (&acc)[8]) {
  acc[0] += __uint_as_float(v.x);
  acc[1] += __uint_as_float(v.y);
  acc[2] += __uint_as_float(v.z);
  acc[3] += __uint_as_float(v.w);
}
template <typename T>
__device__ __forceinline__ uint4 to_vec(const float (&acc)[8]) {
  return pack8<T>(acc);
}
template <>
__device__ __forceinline__ uint4 to_vec<float>(const float (&acc)[8]) {
  return make_uint4(__float_as_uint(acc[0]), __float_as_uint(acc[1]), __float_as_uint(acc[2]),
                    __float_as_uint(acc[3]));
}

// One thread per 16-byte vector of the output, kBatch routes' rows in flight at
// a time, added in order.  Rounds without idle places count: every load and
// addition is predicated, and few registers keep many threads resident.  1000
// tokens of 9 routes, rows of 14 KB: 19.3 us in rounds of 5, 24.2 in rounds of 8;
// 4096 of 4, 8 KB: 23.0 against 30.2; 8192 of 8, 8 KB: 89.1 in rounds of 4 (6.8
// TB/s, a little of it from L2), 90.3 in one of 8.
template <typename T, int kBatch>
__global__ void __launch_bounds__(256)
    sum_routes_kernel(const uint4* __restrict__ y, int64_t rows, int vecs, int64_t ldy, uint4* __restrict__ out,
                      int64_t M, int64_t ldout, const int32_t* __restrict__ route_slot, int top_k, int accumulate) {
  pdl_wait();
  const int64_t total = M * vecs;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t t = i / vecs;
    const int v = static_cast<int>(i - t * vecs);
    if (!MOE_IN_BOUNDS(t >= 0 && t < M && v >= 0 && v < vecs)) continue;
    float acc[8] = {};
    if (accumulate) add_vec<T>(out[t * ldout + v], acc);
    for (int j0 = 0; j0 < top_k; j0 += kBatch) {
      int32_t slot[kBatch];
      uint4 row[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) slot[j] = j0 + j < top_k ? __ldg(route_slot + t * top_k + j0 + j) : -1;
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        row[j] = make_uint4(0, 0, 0, 0);
        if (slot[j] >= 0 && slot[j] < rows && MOE_IN_BOUNDS(ldy >= vecs)) row[j] = __ldcs(y + slot[j] * ldy + v);
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (slot[j] >= 0 && slot[j] < rows) add_vec<T>(row[j], acc);
    }
    __stcs(out + t * ldout + v, to_vec<T>(acc));
  }
}

template <typename T>
auto sum_routes_of(int batch) {
  return batch == 1   ? sum_routes_kernel<T, 1>
         : batch == 2 ? sum_routes_kernel<T, 2>
         : batch == 3 ? sum_routes_kernel<T, 3>
         : batch == 4 ? sum_routes_kernel<T, 4>
                      : sum_routes_kernel<T, 5>;
}

// ---------------------------------------------------------------- SwiGLU gradient

struct SwigluParams {
  const uint16_t* dh;
  const uint16_t* pre;
  uint16_t* dpre;
  uint16_t* h;
  const int32_t* route_ids;
  const int32_t* num_rows;
  const float* weights;
  float* dweights;
  int64_t rows, lddh, ldpre, lddpre, ldh, R;
  int I;
};

// One warp per row, eight elements a lane and step; the row's sum for dweights
// in FP32 by shuffles.  (dpre may be pre and h may be dh: a thread reads its
// elements before it writes them.)  65536 rows of I = 1024: 123 us, 6.5 TB/s.
template <typename T>
__global__ void __launch_bounds__(256) swiglu_backward_kernel(const SwigluParams p) {
  pdl_wait();
  const int64_t n = p.num_rows ? min(static_cast<int64_t>(max(*p.num_rows, 0)), p.rows) : p.rows;
  const int lane = threadIdx.x % 32;
  for (int64_t s = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32; s < n;
       s += static_cast<int64_t>(gridDim.x) * 8) {
    int64_t r = s;
    if (p.route_ids) {
      r = p.route_ids[s];
      if (r < 0 || r >= p.R) continue;
    }
    if (!MOE_IN_BOUNDS(s >= 0 && s < p.rows && r >= 0 && (p.route_ids ? r < p.R : r < p.rows))) continue;
    const float wt = p.weights ? p.weights[r] : 1.0f;
    float dot = 0.f;
    for (int i = 8 * lane; i < p.I; i += 256) {
      float d[8], g[8], u[8], dg[8], du[8], h[8];
      unpack8<T>(*reinterpret_cast<const uint4*>(p.dh + s * p.lddh + i), d);
      unpack8<T>(*reinterpret_cast<const uint4*>(p.pre + s * p.ldpre + i), g);
      unpack8<T>(*reinterpret_cast<const uint4*>(p.pre + s * p.ldpre + p.I + i), u);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float sig = sigmoid_f32(g[j]);
        const float silu = g[j] * sig;
        const float hu = silu * u[j];
        dot += d[j] * hu;
        const float dw = d[j] * wt;
        dg[j] = dw * u[j] * sig * (1.0f + g[j] * (1.0f - sig));
        du[j] = dw * silu;
        h[j] = hu * wt;
      }
      *reinterpret_cast<uint4*>(p.dpre + s * p.lddpre + i) = pack8<T>(dg);
      *reinterpret_cast<uint4*>(p.dpre + s * p.lddpre + p.I + i) = pack8<T>(du);
      if (p.h) *reinterpret_cast<uint4*>(p.h + s * p.ldh + i) = pack8<T>(h);
    }
    if (p.dweights) {
#pragma unroll
      for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      if (lane == 0) p.dweights[r] = dot;
    }
  }
}

// Blocks of `per` units, at most eight resident rounds of 256-thread CTAs.
unsigned grid_of(int64_t units, int64_t per, int sms) {
  const int64_t want = ceil_div(units, per), most = static_cast<int64_t>(sms) * 64;
  return static_cast<unsigned>(want < 1 ? 1 : want > most ? most : want);
}

}  // namespace
}  // namespace moe

extern "C" {

moe_status moe_plan_groups(const int32_t* sorted_token_ids, int64_t sorted_cap, const int32_t* expert_ids,
                           int64_t blocks_cap, const int32_t* num_tokens_post_padded, int block_m, int64_t R, int E,
                           int32_t* group_start, int32_t* group_rows, int32_t* route_slot, moe_stream_t stream) {
  using namespace moe;
  if (E < 1 || E > 2048 || block_m < 8 || block_m > 1024 || block_m % 8 || R < 0 || R >= (int64_t(1) << 31) ||
      blocks_cap < 0)
    return MOE_ERR_SHAPE;
  if (blocks_cap > (int64_t(1) << 31) / block_m || sorted_cap < blocks_cap * block_m) return MOE_ERR_CAPACITY;
  if (!num_tokens_post_padded || !group_start || !group_rows || (blocks_cap > 0 && (!sorted_token_ids || !expert_ids)))
    return MOE_ERR_NULL;
  if (!aligned4(sorted_token_ids, expert_ids, num_tokens_post_padded, group_start, group_rows, route_slot))
    return MOE_ERR_ALIGN;
  DeviceInfo dev;
  if (current_device(&dev) != MOE_OK) return MOE_ERR_CUDA;
  const void* ptrs[] = {sorted_token_ids, expert_ids, num_tokens_post_padded, group_start, group_rows, route_slot};
  for (const void* p : ptrs)
    if (p && !on_device(p, dev.device)) return MOE_ERR_DEVICE;
  if (R == 0) route_slot = nullptr;
  if (route_slot) MOE_CUDA_TRY(cudaMemsetAsync(route_slot, 0xFF, static_cast<size_t>(R) * 4, stream));
  const int64_t units = route_slot && blocks_cap * block_m > E ? blocks_cap * block_m : E;
  int64_t grid = ceil_div(units, 1024);
  if (grid < ceil_div(E, 256)) grid = ceil_div(E, 256);
  MOE_CUDA_TRY(launch_pdl(plan_groups_kernel, dim3(static_cast<unsigned>(grid)), dim3(256), 0, stream, 1,
                          sorted_token_ids, expert_ids, num_tokens_post_padded, blocks_cap, block_m, R, E, group_start,
                          group_rows, route_slot));
  return MOE_OK;
}

moe_status moe_gather_rows(const void* x, int64_t M, int width, int64_t ldx, void* xs, int64_t rows, int64_t ldxs,
                           const int32_t* route_ids, int top_k, const int32_t* num_rows, int dtype,
                           moe_stream_t stream) {
  using namespace moe;
  if (!is_type(dtype)) return MOE_ERR_DTYPE;
  const int eb = type_bytes(dtype), vec = 16 / eb;
  if (!ok_routes(M, top_k) || rows < 0 || rows >= (int64_t(1) << 31) || width < vec || width % vec || ldx % vec ||
      ldxs % vec || ldx < width || ldxs < width || ldx > kMostElements || ldxs > kMostElements)
    return MOE_ERR_SHAPE;
  if (rows == 0) return MOE_OK;
  if ((M > 0 && !x) || !xs || !route_ids) return MOE_ERR_NULL;   // (without tokens every row becomes zero)
  if (!aligned16(x) || !aligned16(xs) || !aligned4(route_ids, num_rows)) return MOE_ERR_ALIGN;
  if (overlap(Rows{x, M, ldx, width}, Rows{xs, rows, ldxs, width}, eb)) return MOE_ERR_SHAPE;
  DeviceInfo dev;
  if (current_device(&dev) != MOE_OK) return MOE_ERR_CUDA;
  const void* ptrs[] = {x, xs, route_ids, num_rows};
  for (const void* p : ptrs)
    if (p && !on_device(p, dev.device)) return MOE_ERR_DEVICE;
  MOE_CUDA_TRY(launch_pdl(gather_rows_kernel, dim3(grid_of(rows, 8, dev.sms)), dim3(256), 0, stream, 1,
                          static_cast<const uint4*>(x), M, width / vec, ldx / vec, static_cast<uint4*>(xs), rows,
                          ldxs / vec, route_ids, top_k, num_rows));
  return MOE_OK;
}

moe_status moe_sum_routes(const void* y, int64_t rows, int width, int64_t ldy, void* out, int64_t M, int64_t ldout,
                          const int32_t* route_slot, int top_k, int accumulate, int dtype, moe_stream_t stream) {
  using namespace moe;
  if (!is_type(dtype)) return MOE_ERR_DTYPE;
  const int eb = type_bytes(dtype), vec = 16 / eb;
  if (!ok_routes(M, top_k) || rows < 0 || rows >= (int64_t(1) << 31) || width < vec || width % vec || ldy % vec ||
      ldout % vec || ldy < width || ldout < width || ldy > kMostElements || ldout > kMostElements)
    return MOE_ERR_SHAPE;
  if (M == 0) return MOE_OK;
  if ((rows > 0 && !y) || !out || !route_slot) return MOE_ERR_NULL;   // (without rows every sum is empty)
  if (!aligned16(y) || !aligned16(out) || !aligned4(route_slot)) return MOE_ERR_ALIGN;
  if (overlap(Rows{y, rows, ldy, width}, Rows{out, M, ldout, width}, eb)) return MOE_ERR_SHAPE;
  DeviceInfo dev;
  if (current_device(&dev) != MOE_OK) return MOE_ERR_CUDA;
  const void* ptrs[] = {y, out, route_slot};
  for (const void* p : ptrs)
    if (p && !on_device(p, dev.device)) return MOE_ERR_DEVICE;
  // rounds of at most five routes, as equal as they can be (rounds of 10, 12 and
  // 16 were slower for every top_k)
  const int batch = static_cast<int>(ceil_div(top_k, ceil_div(top_k, 5)));
  auto kernel = dtype == MOE_TYPE_BF16   ? sum_routes_of<__nv_bfloat16>(batch)
                : dtype == MOE_TYPE_FP16 ? sum_routes_of<__half>(batch)
                                         : sum_routes_of<float>(batch);
  MOE_CUDA_TRY(launch_pdl(kernel, dim3(grid_of(M * (width / vec), 256, dev.sms)), dim3(256), 0, stream, 1,
                          static_cast<const uint4*>(y), rows, width / vec, ldy / vec, static_cast<uint4*>(out), M,
                          ldout / vec, route_slot, top_k, accumulate));
  return MOE_OK;
}

moe_status moe_swiglu_backward(const moe_swiglu_backward_args* a, moe_stream_t stream) {
  using namespace moe;
  if (!a) return MOE_ERR_NULL;
  if (!is_half_type(a->dtype)) return MOE_ERR_DTYPE;
  const int64_t I = a->I;
  if (a->rows < 0 || a->rows >= (int64_t(1) << 31) || a->R < 0 || I < 8 || I % 8 || a->lddh % 8 || a->ldpre % 8 ||
      a->lddpre % 8 || a->lddh < I || a->ldpre < 2 * I || a->lddpre < 2 * I || a->lddh > kMostElements ||
      a->ldpre > kMostElements || a->lddpre > kMostElements ||
      (a->h && (a->ldh % 8 || a->ldh < I || a->ldh > kMostElements)))
    return MOE_ERR_SHAPE;
  if (a->rows == 0) return MOE_OK;
  if (!a->dh || !a->pre || !a->dpre) return MOE_ERR_NULL;
  if (!aligned16(a->dh) || !aligned16(a->pre) || !aligned16(a->dpre) || !aligned16(a->h) ||
      !aligned4(a->route_ids, a->num_rows, a->route_weights, a->dweights))
    return MOE_ERR_ALIGN;
  // in place only element by element: the same rows at the same stride
  const Rows dh{a->dh, a->rows, a->lddh, I}, pre{a->pre, a->rows, a->ldpre, 2 * I};
  const Rows dpre{a->dpre, a->rows, a->lddpre, 2 * I}, h{a->h, a->h ? a->rows : 0, a->ldh, I};
  const bool pre_in_place = a->dpre == a->pre && a->lddpre == a->ldpre, h_in_place = a->h == a->dh && a->ldh == a->lddh;
  if ((!pre_in_place && overlap(dpre, pre, 2)) || overlap(dpre, dh, 2) || overlap(h, dpre, 2) || overlap(h, pre, 2) ||
      (!h_in_place && overlap(h, dh, 2)))
    return MOE_ERR_SHAPE;
  DeviceInfo dev;
  if (current_device(&dev) != MOE_OK) return MOE_ERR_CUDA;
  const void* ptrs[] = {a->dh, a->pre, a->dpre, a->h, a->route_ids, a->num_rows, a->route_weights, a->dweights};
  for (const void* p : ptrs)
    if (p && !on_device(p, dev.device)) return MOE_ERR_DEVICE;
  SwigluParams p;
  p.dh = a->dh;
  p.pre = a->pre;
  p.dpre = a->dpre;
  p.h = a->h;
  p.route_ids = a->route_ids;
  p.num_rows = a->num_rows;
  p.weights = a->route_weights;
  p.dweights = a->dweights;
  p.rows = a->rows;
  p.lddh = a->lddh;
  p.ldpre = a->ldpre;
  p.lddpre = a->lddpre;
  p.ldh = a->ldh;
  p.R = a->R;
  p.I = a->I;
  auto kernel = a->dtype == MOE_TYPE_BF16 ? swiglu_backward_kernel<__nv_bfloat16> : swiglu_backward_kernel<__half>;
  MOE_CUDA_TRY(launch_pdl(kernel, dim3(grid_of(a->rows, 8, dev.sms)), dim3(256), 0, stream, 1, p));
  return MOE_OK;
}

}  // extern "C"

MOE_BOUNDS_TU()
