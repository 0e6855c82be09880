// Products grouped by expert (moe_grouped_gemm, moe_grouped_wgrad): the
// simple form, FP32 products of 64x64 tiles on the CUDA cores.
#include "train.cuh"

namespace moe {
namespace {

__device__ __forceinline__ float to_f32(uint16_t v, int dtype) {
  return dtype == MOE_TYPE_BF16 ? Pack2<__nv_bfloat16>::load(v).x : Pack2<__half>::load(v).x;
}
__device__ __forceinline__ uint16_t from_f32(float v, int dtype) {
  return static_cast<uint16_t>((dtype == MOE_TYPE_BF16 ? Pack2<__nv_bfloat16>::store(v, 0.f)
                                                       : Pack2<__half>::store(v, 0.f)) & 0xFFFFu);
}

// c[i, j] = sum_z a[i * ais + z * azs] b[j * bis + z * bzs], i < mi, j < mj, z < mz, for one 64x64 tile.
struct Operand {
  const uint16_t* p;
  int64_t is, zs;
};
__device__ __forceinline__ void tile_product(const Operand a, const Operand b, int i0, int j0, int mi, int mj, int mz,
                                             int dtype, float (&acc)[4][4], float (*sa)[65], float (*sb)[65]) {
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
  for (int z0 = 0; z0 < mz; z0 += 16) {
    for (int u = threadIdx.x; u < 1024; u += 256) {
      const int z = u % 16, i = u / 16;
      sa[z][i] = i0 + i < mi && z0 + z < mz ? to_f32(a.p[(i0 + i) * a.is + (z0 + z) * a.zs], dtype) : 0.f;
      sb[z][i] = j0 + i < mj && z0 + z < mz ? to_f32(b.p[(j0 + i) * b.is + (z0 + z) * b.zs], dtype) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int z = 0; z < 16; ++z)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] += sa[z][ty + 16 * i] * sb[z][tx + 16 * j];
    __syncthreads();
  }
}

__device__ __forceinline__ bool group_of(const int32_t* start, const int32_t* rows, int e, int64_t cap, int64_t& s0,
                                         int& n, int32_t* status, bool report) {
  s0 = start[e];
  n = rows[e];
  if (n == 0) return true;
  if (s0 < 0 || n < 0 || s0 + n > cap) {
    if (report && status) atomicOr(status, MOE_DEV_BAD_GROUP);
    n = 0;
    return false;
  }
  return true;
}

__global__ void __launch_bounds__(256) grouped_simple_kernel(const moe_grouped_args a) {
  __shared__ float sa[16][65], sb[16][65];
  __shared__ float sg[64][65];
  pdl_wait();
  const int e = blockIdx.z;
  int64_t s0;
  int n;
  group_of(a.group_start, a.group_rows, e, a.rows, s0, n, a.device_status, threadIdx.x == 0);
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const bool fwd = a.direction == MOE_GROUPED_FORWARD, glu = a.epilogue == MOE_GROUPED_SWIGLU;
  const int cols = fwd ? (glu ? a.N / 2 : a.N) : a.K, depth = fwd ? a.K : a.N;
  const int j0 = blockIdx.x * 64;
  const uint16_t* we = a.w + static_cast<int64_t>(e) * a.N * a.K;
  for (int i0 = blockIdx.y * 64; i0 < n; i0 += 64 * gridDim.y) {
    float acc[4][4];
    const Operand x = {a.x + s0 * a.ldx, a.ldx, 1};
    const Operand w = {we, fwd ? a.K : 1, fwd ? 1 : a.K};
    tile_product(x, w, i0, j0, n, cols, depth, a.dtype, acc, sa, sb);
    if (glu) {
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) sg[ty + 16 * i][tx + 16 * j] = acc[i][j];
      __syncthreads();
      const Operand up = {we + static_cast<int64_t>(cols) * a.K, a.K, 1};
      tile_product(x, up, i0, j0, n, cols, depth, a.dtype, acc, sa, sb);
    }
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 4; ++j) {
        const int ri = i0 + ty + 16 * i, c = j0 + tx + 16 * j;
        if (ri >= n || c >= cols) continue;
        const int64_t s = s0 + ri;
        if (!glu) {
          a.y[s * a.ldy + c] = from_f32(acc[i][j], a.dtype);
          continue;
        }
        const float g = sg[ty + 16 * i][tx + 16 * j], u = acc[i][j];
        float wt = 1.f;
        if (a.route_weights) {
          int64_t r = s;
          if (a.route_ids) r = a.route_ids[s];
          wt = a.route_ids && (r < 0 || r >= a.R) ? 0.f : a.route_weights[r];
        }
        a.y[s * a.ldy + c] = from_f32(silu_f32(g) * u * wt, a.dtype);
        if (a.pre) {
          a.pre[s * a.ldpre + c] = from_f32(g, a.dtype);
          a.pre[s * a.ldpre + cols + c] = from_f32(u, a.dtype);
        }
      }
    __syncthreads();
  }
}

__global__ void __launch_bounds__(256) wgrad_simple_kernel(const moe_grouped_wgrad_args a) {
  __shared__ float sa[16][65], sb[16][65];
  pdl_wait();
  const int e = blockIdx.z;
  int64_t s0;
  int n;
  group_of(a.group_start, a.group_rows, e, a.rows, s0, n, a.device_status, threadIdx.x == 0);
  if (n == 0 && a.accumulate) return;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int i0 = blockIdx.y * 64, j0 = blockIdx.x * 64;
  float acc[4][4];
  tile_product({a.dy + s0 * a.lddy, 1, a.lddy}, {a.x + s0 * a.ldx, 1, a.ldx}, i0, j0, a.N, a.K, n, a.dtype, acc, sa, sb);
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int r = i0 + ty + 16 * i, c = j0 + tx + 16 * j;
      if (r >= a.N || c >= a.K) continue;
      const int64_t o = (static_cast<int64_t>(e) * a.N + r) * a.K + c;
      if (a.dw_dtype == MOE_TYPE_FP32) {
        float* d = static_cast<float*>(a.dw) + o;
        *d = a.accumulate ? *d + acc[i][j] : acc[i][j];
      } else {
        static_cast<uint16_t*>(a.dw)[o] = from_f32(acc[i][j], a.dtype);
      }
    }
}

bool ok_sizes(int64_t rows, int E, int N, int K) {
  return rows >= 0 && rows < (int64_t(1) << 31) && E >= 1 && E <= 2048 && N >= 8 && N % 8 == 0 && K >= 8 && K % 8 == 0;
}

}  // namespace
}  // namespace moe

extern "C" {

moe_status moe_grouped_gemm(const moe_grouped_args* a, moe_stream_t stream) {
  using namespace moe;
  if (!a) return MOE_ERR_NULL;
  if (!is_half_type(a->dtype)) return MOE_ERR_DTYPE;
  const bool fwd = a->direction == MOE_GROUPED_FORWARD, glu = a->epilogue == MOE_GROUPED_SWIGLU;
  if ((!fwd && a->direction != MOE_GROUPED_INPUT_GRADIENT) || (!glu && a->epilogue != MOE_GROUPED_PLAIN) ||
      (glu && (!fwd || a->N % 16)) || !ok_sizes(a->rows, a->E, a->N, a->K) || a->R < 0)
    return MOE_ERR_SHAPE;
  const int64_t in = fwd ? a->K : a->N, out = fwd ? (glu ? a->N / 2 : a->N) : a->K;
  const bool pre = glu && a->pre;
  if (a->ldx % 8 || a->ldx < in || a->ldy % 8 || a->ldy < out || (pre && (a->ldpre % 8 || a->ldpre < a->N)))
    return MOE_ERR_SHAPE;
  if (a->rows == 0) return MOE_OK;
  if (!a->x || !a->w || !a->y || !a->group_start || !a->group_rows) return MOE_ERR_NULL;
  if (!aligned16(a->x) || !aligned16(a->w) || !aligned16(a->y) || (pre && !aligned16(a->pre))) return MOE_ERR_ALIGN;
  const int64_t bx = extent_bytes(a->rows, a->ldx, in, 2), by = extent_bytes(a->rows, a->ldy, out, 2);
  const int64_t bw = 2ll * a->E * a->N * a->K, bp = pre ? extent_bytes(a->rows, a->ldpre, a->N, 2) : 0;
  if (overlap(a->y, by, a->x, bx) || overlap(a->y, by, a->w, bw) || overlap(a->pre, bp, a->x, bx) ||
      overlap(a->pre, bp, a->w, bw) || overlap(a->pre, bp, a->y, by))
    return MOE_ERR_SHAPE;
  DeviceInfo dev;
  if (current_device(&dev) != MOE_OK) return MOE_ERR_CUDA;
  if (dev.major != 10 || dev.minor != 3) return MOE_ERR_DEVICE;
  const void* ptrs[] = {a->x, a->w, a->y, pre ? a->pre : nullptr, a->group_start, a->group_rows,
                        glu ? a->route_ids : nullptr, glu ? a->route_weights : nullptr, a->device_status};
  for (const void* p : ptrs)
    if (p && !on_device(p, dev.device)) return MOE_ERR_DEVICE;
  moe_grouped_args k = *a;
  if (!glu) k.route_ids = nullptr, k.route_weights = nullptr, k.pre = nullptr;
  const unsigned gy = static_cast<unsigned>(a->rows < 64 * 16 ? ceil_div(a->rows, 64) : 16);
  MOE_CUDA_TRY(launch_pdl(grouped_simple_kernel, dim3(static_cast<unsigned>(ceil_div(out, 64)), gy, a->E), dim3(256), 0,
                          stream, 1, k));
  return MOE_OK;
}

moe_status moe_grouped_wgrad(const moe_grouped_wgrad_args* a, moe_stream_t stream) {
  using namespace moe;
  if (!a) return MOE_ERR_NULL;
  if (!is_half_type(a->dtype) || (a->dw_dtype != a->dtype && a->dw_dtype != MOE_TYPE_FP32)) return MOE_ERR_DTYPE;
  if (a->accumulate && a->dw_dtype != MOE_TYPE_FP32) return MOE_ERR_DTYPE;
  if (!ok_sizes(a->rows, a->E, a->N, a->K) || a->lddy % 8 || a->ldx % 8 || a->lddy < a->N || a->ldx < a->K)
    return MOE_ERR_SHAPE;
  if (!a->dw || !a->group_start || !a->group_rows || (a->rows > 0 && (!a->dy || !a->x))) return MOE_ERR_NULL;
  if (!aligned16(a->dy) || !aligned16(a->x) || !aligned16(a->dw)) return MOE_ERR_ALIGN;
  const int64_t bd = static_cast<int64_t>(type_bytes(a->dw_dtype)) * a->E * a->N * a->K;
  if (overlap(a->dw, bd, a->dy, extent_bytes(a->rows, a->lddy, a->N, 2)) ||
      overlap(a->dw, bd, a->x, extent_bytes(a->rows, a->ldx, a->K, 2)))
    return MOE_ERR_SHAPE;
  DeviceInfo dev;
  if (current_device(&dev) != MOE_OK) return MOE_ERR_CUDA;
  if (dev.major != 10 || dev.minor != 3) return MOE_ERR_DEVICE;
  const void* ptrs[] = {a->dy, a->x, a->dw, a->group_start, a->group_rows, a->device_status};
  for (const void* p : ptrs)
    if (p && !on_device(p, dev.device)) return MOE_ERR_DEVICE;
  MOE_CUDA_TRY(launch_pdl(wgrad_simple_kernel,
                          dim3(static_cast<unsigned>(ceil_div(a->K, 64)), static_cast<unsigned>(ceil_div(a->N, 64)),
                               static_cast<unsigned>(a->E)),
                          dim3(256), 0, stream, 1, *a));
  return MOE_OK;
}

}  // extern "C"

MOE_BOUNDS_TU()
