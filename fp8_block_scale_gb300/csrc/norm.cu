// A block's exit and the next one's entry in one pass (moe_norm_residual): norm
// of the branch, gate, residual scale, norm of the stream, and the experts'
// input in FP8.
//
// Each byte is read and written once, a row at a time: its elements stay in
// registers between the two norms, which need a sum over the row each.  HBM bounds
// it; what there is to hide is the chain load, sum, sum, store of a row, so
// several rows are in flight on an SM.
#include "norm.cuh"

namespace moe {
namespace {

struct NormParams {
  const void* y;
  const void* r;
  const void* gate;
  const void* w_post;
  const void* w_pre;
  void* h;
  void* z;
  uint8_t* q;
  float* q_scale;
  const int32_t* num_rows;
  int64_t M, ldy, ldr, ldh, ldz, ldgate;
  int H, wide, gate_mode, post_norm, pow2;
  float residual_scale, weight_offset, eps;
};

// Smallest power of two >= s (as the quantisers round: a scale above 2^127 is kept).
__device__ __forceinline__ float scale_to_pow2(float s) {
  const uint32_t b = __float_as_uint(s), ex = b >> 23;
  if ((b & 0x7FFFFFu) == 0 || ex >= 254) return s;
  if (ex != 0) return __uint_as_float((ex + 1) << 23);
  const int top = 31 - __clz(b);
  if ((b & (b - 1)) == 0) return s;
  return top + 1 >= 23 ? __uint_as_float(1u << 23) : __uint_as_float(1u << (top + 1));
}

// kVec vectors of eight elements a thread; kWarpRow: a warp per row, else a CTA.
template <typename Tb, typename Ts, int kVec, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? 256 : 1024) norm_kernel(const __grid_constant__ NormParams p) {
  __shared__ float part[2][1][32];
  pdl_wait();
  pdl_launch_dependents();
  int turn = 0;
  const int team = kWarpRow ? 32 : blockDim.x, tid = kWarpRow ? threadIdx.x % 32 : threadIdx.x;
  const int64_t live = p.num_rows ? min(static_cast<int64_t>(max(*p.num_rows, 0)), p.M) : p.M;
  const int64_t row0 = kWarpRow ? static_cast<int64_t>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32 : blockIdx.x;
  const int64_t step = kWarpRow ? static_cast<int64_t>(gridDim.x) * (blockDim.x / 32) : gridDim.x;
  const float inv_h = 1.f / static_cast<float>(p.H);
  for (int64_t row = row0; row < live; row += step) {
    Vec8<Tb> yr[kVec], gr[kVec];
    Vec8<Ts> rr[kVec];
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const int c = 8 * (tid + v * team);
      if (c < p.H) {
        yr[v] = load_vec<Tb>(static_cast<const Tb*>(p.y) + row * p.ldy + c);
        if (p.r) rr[v] = load_vec<Ts>(static_cast<const Ts*>(p.r) + row * p.ldr + c);
        if (p.gate_mode == MOE_GATE_FULL) gr[v] = load_vec<Tb>(static_cast<const Tb*>(p.gate) + row * p.ldgate + c);
      }
    }
    float h[kVec][8];
    float root = 1.f;
    if (p.post_norm) {
      float sum[1] = {0.f};
#pragma unroll
      for (int v = 0; v < kVec; ++v)
        if (8 * (tid + v * team) < p.H) {
          widen<Tb>(yr[v], h[v]);
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[0] = fmaf(h[v][i], h[v][i], sum[0]);
        }
      row_sums<1, kWarpRow>(sum, part, turn);
      root = rsqrtf(fmaf(sum[0], inv_h, p.eps));
    }
    const float token = p.gate_mode == MOE_GATE_TOKEN ? __ldg(static_cast<const float*>(p.gate) + row) : 1.f;
    float sum[1] = {0.f};
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const int c = 8 * (tid + v * team);
      if (c < p.H) {
        widen<Tb>(yr[v], h[v]);
        if (p.post_norm) {
          float w[8];
          load_weights<Tb>(p.w_post, p.wide, c, p.weight_offset, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) h[v][i] = h[v][i] * root * w[i];
        }
        if (p.gate_mode == MOE_GATE_TOKEN) {
#pragma unroll
          for (int i = 0; i < 8; ++i) h[v][i] *= token;
        } else if (p.gate_mode != MOE_GATE_NONE) {
          float g[8];
          if (p.gate_mode == MOE_GATE_FULL)
            widen<Tb>(gr[v], g);
          else
            load_weights<Tb>(p.gate, p.wide, c, 0.f, g);
#pragma unroll
          for (int i = 0; i < 8; ++i) h[v][i] *= g[i];
        }
        if (p.r) {
          float r[8];
          widen<Ts>(rr[v], r);
#pragma unroll
          for (int i = 0; i < 8; ++i) h[v][i] = fmaf(p.residual_scale, r[i], h[v][i]);
        }
        if (p.h) store_vec<Ts>(static_cast<Ts*>(p.h) + row * p.ldh + c, h[v]);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[0] = fmaf(h[v][i], h[v][i], sum[0]);
      }
    }
    if (!p.z && !p.q) continue;
    row_sums<1, kWarpRow>(sum, part, turn);
    root = rsqrtf(fmaf(sum[0], inv_h, p.eps));
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const int c = 8 * (tid + v * team);
      // (a group of 128 columns is 16 neighbouring lanes of one warp: all of them or none have columns)
      if (c < p.H) {
        float w[8];
        load_weights<Tb>(p.w_pre, p.wide, c, p.weight_offset, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[v][i] = h[v][i] * root * w[i];
        if (p.z) store_vec<Tb>(static_cast<Tb*>(p.z) + row * p.ldz + c, h[v]);
      }
      if (p.q) {
        float amax = 0.f;
        if (c < p.H) {
#pragma unroll
          for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(h[v][i]));
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        float s = __fdiv_rn(amax, 448.f);
        if (p.pow2 && s > 0.f) s = scale_to_pow2(s);
        if (c < p.H) {
          uint32_t code[2] = {0, 0};
          if (s > 0.f) {
#pragma unroll
            for (int i = 0; i < 8; i += 2)
              code[i / 4] |= static_cast<uint32_t>(cvt_e4m3x2(__fdiv_rn(h[v][i], s), __fdiv_rn(h[v][i + 1], s))) << (8 * (i % 4));
          }
          if (MOE_IN_BOUNDS(row >= 0 && row < p.M)) {
            *reinterpret_cast<uint2*>(p.q + row * p.H + c) = make_uint2(code[0], code[1]);
            if (tid % 16 == 0) p.q_scale[row * (p.H / 128) + c / 128] = s;
          }
        }
      }
    }
  }
}

template <typename Tb, typename Ts>
cudaError_t launch_norm(const NormParams& p, int sms, cudaStream_t stream) {
  const int vecs = p.H / 8;
  if (vecs <= 64) {
    const int64_t ctas = ceil_div(p.M, 8), most = static_cast<int64_t>(sms) * 64;
    const dim3 grid(static_cast<unsigned>(ctas < most ? ctas : most));
    return vecs <= 32 ? launch_pdl(norm_kernel<Tb, Ts, 1, true>, grid, dim3(256), 0, stream, 1, p)
                      : launch_pdl(norm_kernel<Tb, Ts, 2, true>, grid, dim3(256), 0, stream, 1, p);
  }
  const int64_t most = static_cast<int64_t>(sms) * 64;
  const dim3 grid(static_cast<unsigned>(p.M < most ? p.M : most));
  if (vecs <= 1024 && p.M <= sms)
    return launch_pdl(norm_kernel<Tb, Ts, 1, false>, grid, dim3(team_threads(vecs, 1)), 0, stream, 1, p);
  return launch_pdl(norm_kernel<Tb, Ts, 2, false>, grid, dim3(team_threads(vecs, 2)), 0, stream, 1, p);
}

}  // namespace
}  // namespace moe

extern "C" {

moe_status moe_norm_residual(const moe_norm_args* a, moe_stream_t stream) {
  using namespace moe;
  if (!a) return MOE_ERR_NULL;
  const moe_status bad = check_norm(a->M, a->H, a->dtype, a->stream_dtype, a->weight_dtype, a->gate_mode, a->gate,
                                    a->ldgate, a->residual_scale, a->weight_offset, a->eps);
  if (bad != MOE_OK) return bad;
  const int64_t M = a->M;
  const int H = a->H, eb = type_bytes(a->dtype), es = type_bytes(a->stream_dtype), ew = type_bytes(a->weight_dtype);
  if (!ok_stride(a->y, a->ldy, H) || !ok_stride(a->r, a->ldr, H) || !ok_stride(a->h, a->ldh, H) ||
      !ok_stride(a->z, a->ldz, H) || (a->q && H % 128) ||
      (a->q && a->scale_mode != MOE_SCALES_FP32 && a->scale_mode != MOE_SCALES_UE8M0))
    return MOE_ERR_SHAPE;
  if (M == 0) return MOE_OK;
  if (!a->y || (!a->h && !a->z && !a->q) || !a->q != !a->q_scale || (a->gate_mode != MOE_GATE_NONE && !a->gate)) return MOE_ERR_NULL;
  const void* gate = a->gate_mode == MOE_GATE_NONE ? nullptr : a->gate;
  const void* w_post = a->post_norm ? a->w_post : nullptr;
  const void* w_pre = a->z || a->q ? a->w_pre : nullptr;
  for (const void* p : {a->y, a->r, w_post, w_pre, static_cast<const void*>(a->h), static_cast<const void*>(a->z),
                        static_cast<const void*>(a->q), a->gate_mode == MOE_GATE_TOKEN ? nullptr : gate})
    if (!aligned16(p)) return MOE_ERR_ALIGN;
  if (!aligned4(gate, a->q_scale, a->num_rows)) return MOE_ERR_ALIGN;
  const Span y = span(a->y, M, a->ldy, H, eb), r = span(a->r, M, a->ldr, H, es), h = span(a->h, M, a->ldh, H, es),
             z = span(a->z, M, a->ldz, H, eb);
  const Span ins[] = {y, r, gate_span(a->gate_mode, gate, M, H, a->ldgate, a->gate_mode == MOE_GATE_CHANNEL ? ew : eb),
                      span(w_post, 1, H, H, ew), span(w_pre, 1, H, H, ew), span(a->num_rows, 1, 1, 1, 4)};
  const Span outs[] = {h, z, span(a->q, M, H, H, 1), span(a->q_scale, M, H / 128, H / 128, 4)};
  for (int o = 0; o < 4; ++o) {
    for (int i = 0; i < 6; ++i) {
      const bool in_place = (o == 0 && i == 1 && same_rows(h, r)) || (o == 1 && i == 0 && same_rows(z, y));
      if (!in_place && overlap(outs[o], ins[i])) return MOE_ERR_SHAPE;
    }
    for (int i = 0; i < o; ++i)
      if (overlap(outs[o], outs[i])) return MOE_ERR_SHAPE;
  }
  DeviceInfo dev;
  if (current_device(&dev) != MOE_OK) return MOE_ERR_CUDA;
  for (const void* p : {a->y, a->r, gate, w_post, w_pre, static_cast<const void*>(a->h), static_cast<const void*>(a->z),
                        static_cast<const void*>(a->q), static_cast<const void*>(a->q_scale), static_cast<const void*>(a->num_rows)})
    if (p && !on_device(p, dev.device)) return MOE_ERR_DEVICE;
  NormParams p;
  p.y = a->y;
  p.r = a->r;
  p.gate = gate;
  p.w_post = w_post;
  p.w_pre = w_pre;
  p.h = a->h;
  p.z = a->z;
  p.q = a->q;
  p.q_scale = a->q_scale;
  p.num_rows = a->num_rows;
  p.M = M;
  p.ldy = a->ldy;
  p.ldr = a->ldr;
  p.ldh = a->ldh;
  p.ldz = a->ldz;
  p.ldgate = a->ldgate;
  p.H = H;
  p.wide = a->weight_dtype == MOE_TYPE_FP32;
  p.gate_mode = a->gate_mode;
  p.post_norm = a->post_norm;
  p.pow2 = a->scale_mode == MOE_SCALES_UE8M0;
  p.residual_scale = a->residual_scale;
  p.weight_offset = a->weight_offset;
  p.eps = a->eps;
  const bool wide = a->stream_dtype == MOE_TYPE_FP32;
  const cudaError_t err = a->dtype == MOE_TYPE_FP32 ? launch_norm<float, float>(p, dev.sms, stream)
                          : a->dtype == MOE_TYPE_BF16
                              ? (wide ? launch_norm<__nv_bfloat16, float>(p, dev.sms, stream)
                                      : launch_norm<__nv_bfloat16, __nv_bfloat16>(p, dev.sms, stream))
                              : (wide ? launch_norm<__half, float>(p, dev.sms, stream)
                                      : launch_norm<__half, __half>(p, dev.sms, stream));
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"

MOE_BOUNDS_TU()
