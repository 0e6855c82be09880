// The gradient of the norms around a block (moe_norm_residual_backward).
//
// Row by row as the forward pass, with two rounds of sums over a row (the second
// needs the first's result).  The gradients that are sums over rows (both weights',
// a channel gate's) gather in registers, each thread's columns over all of its
// rows; every CTA leaves its sums in the workspace, and a second launch adds
// them in a fixed order.
#include "norm.cuh"

namespace moe {
namespace {

constexpr int kMaxParts = 320;      // CTAs whose sums over rows the workspace holds
constexpr int kSums = 3;            // dw_pre, dw_post, a channel gate's

struct NormGradParams {
  const void* y;
  const void* h;
  const void* gate;
  const void* w_post;
  const void* w_pre;
  const void* dh;
  const void* dz;
  void* dy;
  void* dr;
  void* dgate;
  float* parts;                     // [kSums, CTAs, H]
  const int32_t* num_rows;
  int64_t M, ldy, ldh, ldgate, lddh, lddz, lddy, lddr, lddgate;
  int H, wide, gate_mode, post_norm;
  int sums;                         // bit n: sum n is asked for
  float residual_scale, weight_offset, eps;
};

template <typename Tb, typename Ts, int kVec, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? 256 : 1024) norm_backward_kernel(const __grid_constant__ NormGradParams p) {
  __shared__ float part[2][3][32];
  extern __shared__ float gathered[];
  pdl_wait();
  pdl_launch_dependents();
  int turn = 0;
  const int team = kWarpRow ? 32 : blockDim.x, tid = kWarpRow ? threadIdx.x % 32 : threadIdx.x;
  const int64_t live = p.num_rows ? min(static_cast<int64_t>(max(*p.num_rows, 0)), p.M) : p.M;
  const int64_t row0 = kWarpRow ? static_cast<int64_t>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32 : blockIdx.x;
  const int64_t step = kWarpRow ? static_cast<int64_t>(gridDim.x) * (blockDim.x / 32) : gridDim.x;
  const float inv_h = 1.f / static_cast<float>(p.H);
  float acc[kSums][kVec][8];
#pragma unroll
  for (int n = 0; n < kSums; ++n)
#pragma unroll
    for (int v = 0; v < kVec; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[n][v][i] = 0.f;

  for (int64_t row = row0; row < live; row += step) {
    Vec8<Tb> yr[kVec], zr[kVec], gr[kVec];
    Vec8<Ts> hr[kVec], dr[kVec];
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const int c = 8 * (tid + v * team);
      if (c < p.H) {
        yr[v] = load_vec<Tb>(static_cast<const Tb*>(p.y) + row * p.ldy + c);
        if (p.dz) {
          zr[v] = load_vec<Tb>(static_cast<const Tb*>(p.dz) + row * p.lddz + c);
          if (p.h) hr[v] = load_vec<Ts>(static_cast<const Ts*>(p.h) + row * p.ldh + c);
        }
        if (p.dh) dr[v] = load_vec<Ts>(static_cast<const Ts*>(p.dh) + row * p.lddh + c);
        if (p.gate_mode == MOE_GATE_FULL) gr[v] = load_vec<Tb>(static_cast<const Tb*>(p.gate) + row * p.ldgate + c);
      }
    }
    // first round: squares of h and y, and dz w h
    float sum[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const int c = 8 * (tid + v * team);
      if (c < p.H) {
        float x[8];
        if (p.dz) {
          float z[8], w[8];
          if (p.h) widen<Ts>(hr[v], x); else widen<Tb>(yr[v], x);
          widen<Tb>(zr[v], z);
          load_weights<Tb>(p.w_pre, p.wide, c, p.weight_offset, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            sum[0] = fmaf(x[i], x[i], sum[0]);
            sum[1] = fmaf(z[i] * w[i], x[i], sum[1]);
          }
        }
        if (p.post_norm) {
          widen<Tb>(yr[v], x);
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[2] = fmaf(x[i], x[i], sum[2]);
        }
      }
    }
    row_sums<3, kWarpRow>(sum, part, turn);
    const float root_h = rsqrtf(fmaf(sum[0], inv_h, p.eps)), root_y = p.post_norm ? rsqrtf(fmaf(sum[2], inv_h, p.eps)) : 1.f;
    const float back_h = root_h * root_h * root_h * (sum[1] * inv_h);
    const float token = p.gate_mode == MOE_GATE_TOKEN ? __ldg(static_cast<const float*>(p.gate) + row) : 1.f;

    // second round: dH, and with it du w y (a token gate's share of it once for the row)
    float d[kVec][8];
    float dot[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const int c = 8 * (tid + v * team);
      if (c < p.H) {
        if (p.dh) {
          widen<Ts>(dr[v], d[v]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) d[v][i] = 0.f;
        }
        float y[8];
        widen<Tb>(yr[v], y);
        if (p.dz) {
          float x[8], z[8], w[8];
          if (p.h) widen<Ts>(hr[v], x); else widen<Tb>(yr[v], x);
          widen<Tb>(zr[v], z);
          load_weights<Tb>(p.w_pre, p.wide, c, p.weight_offset, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            acc[0][v][i] = fmaf(z[i] * x[i], root_h, acc[0][v][i]);
            d[v][i] = fmaf(z[i] * w[i], root_h, fmaf(-x[i], back_h, d[v][i]));
          }
        }
        if (p.dr) {
          float o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = p.residual_scale * d[v][i];
          store_vec<Ts>(static_cast<Ts*>(p.dr) + row * p.lddr + c, o);
        }
        float u[8];                       // y R(y) (w + offset), or y
        float w[8];
        if (p.post_norm) {
          load_weights<Tb>(p.w_post, p.wide, c, p.weight_offset, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) u[i] = y[i] * root_y * w[i];
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) u[i] = y[i];
        }
        if (p.gate_mode == MOE_GATE_TOKEN) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dot[1] = fmaf(d[v][i], u[i], dot[1]);
            d[v][i] *= token;
          }
        } else if (p.gate_mode == MOE_GATE_CHANNEL) {
          float g[8];
          load_weights<Tb>(p.gate, p.wide, c, 0.f, g);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            acc[2][v][i] = fmaf(d[v][i], u[i], acc[2][v][i]);
            d[v][i] *= g[i];
          }
        } else if (p.gate_mode == MOE_GATE_FULL) {
          float g[8], o[8];
          widen<Tb>(gr[v], g);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            o[i] = d[v][i] * u[i];
            d[v][i] *= g[i];
          }
          if (p.dgate) store_vec<Tb>(static_cast<Tb*>(p.dgate) + row * p.lddgate + c, o);
        }
        if (p.post_norm) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            acc[1][v][i] = fmaf(d[v][i] * y[i], root_y, acc[1][v][i]);
            dot[0] = fmaf(d[v][i] * w[i], y[i], dot[0]);
          }
        }
      }
    }
    float back_y = 0.f;
    if (p.post_norm || (p.gate_mode == MOE_GATE_TOKEN && p.dgate)) {
      row_sums<3, kWarpRow>(dot, part, turn);
      back_y = root_y * root_y * root_y * (dot[0] * inv_h);
      if (p.gate_mode == MOE_GATE_TOKEN && p.dgate && tid == 0) static_cast<float*>(p.dgate)[row] = dot[1];
    }
    if (p.dy) {
#pragma unroll
      for (int v = 0; v < kVec; ++v) {
        const int c = 8 * (tid + v * team);
        if (c < p.H) {
          if (p.post_norm) {
            float w[8], y[8];
            load_weights<Tb>(p.w_post, p.wide, c, p.weight_offset, w);
            widen<Tb>(yr[v], y);
#pragma unroll
            for (int i = 0; i < 8; ++i) d[v][i] = fmaf(d[v][i] * w[i], root_y, -(y[i] * back_y));
          }
          store_vec<Tb>(static_cast<Tb*>(p.dy) + row * p.lddy + c, d[v]);
        }
      }
    }
  }

  if (!p.sums) return;
  if (kWarpRow) {
    // the CTA's warps one after another into shared memory, then out
    const int warp = threadIdx.x / 32, warps = blockDim.x / 32;
    for (int w = 0; w < warps; ++w) {
      if (w == warp) {
#pragma unroll
        for (int n = 0; n < kSums; ++n)
#pragma unroll
          for (int v = 0; v < kVec; ++v) {
            const int c = 8 * (tid + v * team);
            if (c < p.H)
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                float* at = gathered + n * p.H + c + i;
                *at = w == 0 ? acc[n][v][i] : *at + acc[n][v][i];
              }
          }
      }
      __syncthreads();
    }
    for (int n = 0; n < kSums; ++n)
      if ((p.sums >> n) & 1)
        for (int c = threadIdx.x; c < p.H; c += blockDim.x)
          p.parts[(static_cast<int64_t>(n) * gridDim.x + blockIdx.x) * p.H + c] = gathered[n * p.H + c];
  } else {
#pragma unroll
    for (int n = 0; n < kSums; ++n)
      if ((p.sums >> n) & 1)
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
          const int c = 8 * (tid + v * team);
          if (c < p.H) store_vec<float>(p.parts + (static_cast<int64_t>(n) * gridDim.x + blockIdx.x) * p.H + c, acc[n][v]);
        }
  }
}

// out[n][c] (+)= sum over the CTAs' parts, in their order: eight warps take every eighth
// one, their sums are added by the first.
struct JoinParams {
  const float* parts;
  float* out[kSums];
  int count, H, accumulate;
};
__global__ void __launch_bounds__(256) join_parts_kernel(const __grid_constant__ JoinParams p) {
  __shared__ float s[8][32];
  pdl_wait();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, c = blockIdx.x * 32 + lane, n = blockIdx.y;
  float* out = n == 0 ? p.out[0] : n == 1 ? p.out[1] : p.out[2];
  if (!out) return;                                         // (the whole CTA)
  float v = 0.f;
  if (c < p.H)
    for (int i = warp; i < p.count; i += 8) v += p.parts[(static_cast<int64_t>(n) * p.count + i) * p.H + c];
  s[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < p.H) {
#pragma unroll
    for (int w = 1; w < 8; ++w) v += s[w][lane];
    out[c] = p.accumulate ? out[c] + v : v;
  }
}

template <typename Tb, typename Ts>
cudaError_t launch_backward(NormGradParams& p, int sms, int* ctas, cudaStream_t stream) {
  const int vecs = p.H / 8;
  const int64_t most = 2 * sms < kMaxParts ? 2 * sms : kMaxParts;
  if (vecs <= 64) {
    const int64_t want = ceil_div(p.M, 8);
    *ctas = static_cast<int>(want < 1 ? 1 : want < most ? want : most);
    const size_t smem = static_cast<size_t>(kSums) * p.H * 4;
    return vecs <= 32 ? launch_pdl(norm_backward_kernel<Tb, Ts, 1, true>, dim3(*ctas), dim3(256), smem, stream, 1, p)
                      : launch_pdl(norm_backward_kernel<Tb, Ts, 2, true>, dim3(*ctas), dim3(256), smem, stream, 1, p);
  }
  *ctas = static_cast<int>(p.M < 1 ? 1 : p.M < most ? p.M : most);
  if (vecs <= 512)
    return launch_pdl(norm_backward_kernel<Tb, Ts, 1, false>, dim3(*ctas), dim3(team_threads(vecs, 1)), 0, stream, 1, p);
  return launch_pdl(norm_backward_kernel<Tb, Ts, 2, false>, dim3(*ctas), dim3(team_threads(vecs, 2)), 0, stream, 1, p);
}

}  // namespace
}  // namespace moe

extern "C" {

size_t moe_norm_residual_workspace_size(int64_t M, int H) {
  using namespace moe;
  if (M < 0 || M >= (int64_t(1) << 31) || H < 8 || H % 8 || H > kNormMaxH) return 0;
  return static_cast<size_t>(M < 1 ? 1 : M < kMaxParts ? M : kMaxParts) * kSums * static_cast<size_t>(H) * 4;
}

moe_status moe_norm_residual_backward(const moe_norm_backward_args* a, moe_stream_t stream) {
  using namespace moe;
  if (!a) return MOE_ERR_NULL;
  const moe_status bad = check_norm(a->M, a->H, a->dtype, a->stream_dtype, a->weight_dtype, a->gate_mode, a->gate,
                                    a->ldgate, a->residual_scale, a->weight_offset, a->eps);
  if (bad != MOE_OK) return bad;
  const int64_t M = a->M;
  const int H = a->H, eb = type_bytes(a->dtype), es = type_bytes(a->stream_dtype), ew = type_bytes(a->weight_dtype);
  const bool full = a->gate_mode == MOE_GATE_FULL, channel = a->gate_mode == MOE_GATE_CHANNEL;
  if (!ok_stride(a->y, a->ldy, H) || !ok_stride(a->h, a->ldh, H) || !ok_stride(a->dh, a->lddh, H) ||
      !ok_stride(a->dz, a->lddz, H) || !ok_stride(a->dy, a->lddy, H) || !ok_stride(a->dr, a->lddr, H) ||
      (full && !ok_stride(a->dgate, a->lddgate, H)) || (a->dgate && a->gate_mode == MOE_GATE_NONE) ||
      (a->dw_post && !a->post_norm) || (!a->h && a->dz && M > 0 && (a->post_norm || a->gate_mode != MOE_GATE_NONE)))
    return MOE_ERR_SHAPE;
  float* sums[kSums] = {a->dw_pre, a->dw_post, channel ? static_cast<float*>(a->dgate) : nullptr};
  int asked = 0;
  for (int n = 0; n < kSums; ++n) asked |= sums[n] ? 1 << n : 0;
  if (M == 0 && !asked) return MOE_OK;
  // (an empty batch's row buffers have no address; its sums are zero)
  if (M > 0 && (!a->y || (!a->dh && !a->dz) || (a->dw_pre && !a->dz) || (a->gate_mode != MOE_GATE_NONE && !a->gate)))
    return MOE_ERR_NULL;
  if (asked && !a->workspace) return MOE_ERR_NULL;
  if (asked && a->workspace_bytes < moe_norm_residual_workspace_size(M, H)) return MOE_ERR_CAPACITY;
  const void* workspace = asked ? a->workspace : nullptr;
  const void* gate = a->gate_mode == MOE_GATE_NONE ? nullptr : a->gate;
  const void* w_post = a->post_norm ? a->w_post : nullptr;
  const void* w_pre = a->dz ? a->w_pre : nullptr;
  const void* h = a->dz ? a->h : nullptr;
  const void* wide16[] = {a->y, h, full || channel ? gate : nullptr, w_post, w_pre, a->dh, a->dz, a->dy, a->dr,
                          full || channel ? a->dgate : nullptr, a->dw_post, a->dw_pre, workspace};
  for (const void* p : wide16)
    if (!aligned16(p)) return MOE_ERR_ALIGN;
  if (!aligned4(gate, a->dgate, a->num_rows)) return MOE_ERR_ALIGN;
  const Span y = span(a->y, M, a->ldy, H, eb), hs = span(h, M, a->ldh, H, es), dh = span(a->dh, M, a->lddh, H, es),
             dz = span(a->dz, M, a->lddz, H, eb), dy = span(a->dy, M, a->lddy, H, eb), dr = span(a->dr, M, a->lddr, H, es);
  const Span ins[] = {y, hs, dh, dz, gate_span(a->gate_mode, gate, M, H, a->ldgate, channel ? ew : eb),
                      span(w_post, 1, H, H, ew), span(w_pre, 1, H, H, ew), span(a->num_rows, 1, 1, 1, 4)};
  const Span outs[] = {dy, dr, gate_span(a->gate_mode, a->dgate, M, H, a->lddgate, channel ? 4 : eb),
                       span(a->dw_post, 1, H, H, 4), span(a->dw_pre, 1, H, H, 4),
                       span(workspace, 1, static_cast<int64_t>(a->workspace_bytes), static_cast<int64_t>(a->workspace_bytes), 1)};
  for (int o = 0; o < 6; ++o) {
    for (int i = 0; i < 8; ++i) {
      const bool in_place = (o == 0 && (i == 0 || i == 3) && same_rows(dy, ins[i])) ||
                            (o == 1 && (i == 1 || i == 2) && same_rows(dr, ins[i]));
      if (!in_place && overlap(outs[o], ins[i])) return MOE_ERR_SHAPE;
    }
    for (int i = 0; i < o; ++i)
      if (overlap(outs[o], outs[i])) return MOE_ERR_SHAPE;
  }
  DeviceInfo dev;
  if (current_device(&dev) != MOE_OK) return MOE_ERR_CUDA;
  const void* ptrs[] = {a->y, h, gate, w_post, w_pre, a->dh, a->dz, a->dy, a->dr, a->dgate, a->dw_post, a->dw_pre, workspace, a->num_rows};
  for (const void* p : ptrs)
    if (p && !on_device(p, dev.device)) return MOE_ERR_DEVICE;
  NormGradParams p;
  p.y = a->y;
  p.h = h;
  p.gate = gate;
  p.w_post = w_post;
  p.w_pre = w_pre;
  p.dh = a->dh;
  p.dz = a->dz;
  p.dy = a->dy;
  p.dr = a->dr;
  p.dgate = a->dgate;
  p.parts = static_cast<float*>(a->workspace);
  p.num_rows = a->num_rows;
  p.M = M;
  p.ldy = a->ldy;
  p.ldh = a->ldh;
  p.ldgate = a->ldgate;
  p.lddh = a->lddh;
  p.lddz = a->lddz;
  p.lddy = a->lddy;
  p.lddr = a->lddr;
  p.lddgate = a->lddgate;
  p.H = H;
  p.wide = a->weight_dtype == MOE_TYPE_FP32;
  p.gate_mode = a->gate_mode;
  p.post_norm = a->post_norm;
  p.sums = asked;
  p.residual_scale = a->residual_scale;
  p.weight_offset = a->weight_offset;
  p.eps = a->eps;
  const bool wide = a->stream_dtype == MOE_TYPE_FP32;
  int ctas = 0;
  MOE_CUDA_TRY(a->dtype == MOE_TYPE_FP32 ? (launch_backward<float, float>(p, dev.sms, &ctas, stream))
               : a->dtype == MOE_TYPE_BF16
                   ? (wide ? launch_backward<__nv_bfloat16, float>(p, dev.sms, &ctas, stream)
                           : launch_backward<__nv_bfloat16, __nv_bfloat16>(p, dev.sms, &ctas, stream))
                   : (wide ? launch_backward<__half, float>(p, dev.sms, &ctas, stream)
                           : launch_backward<__half, __half>(p, dev.sms, &ctas, stream)));
  if (asked) {
    JoinParams j;
    j.parts = p.parts;
    for (int n = 0; n < kSums; ++n) j.out[n] = sums[n];
    j.count = ctas;
    j.H = H;
    j.accumulate = a->accumulate;
    MOE_CUDA_TRY(launch_pdl(join_parts_kernel, dim3(static_cast<unsigned>(ceil_div(H, 32)), kSums), dim3(256), 0, stream, 1, j));
  }
  return MOE_OK;
}

}  // extern "C"

MOE_BOUNDS_TU()
