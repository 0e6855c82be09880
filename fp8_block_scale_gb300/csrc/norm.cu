// A block's exit and the next one's entry in one pass (moe_norm_residual): norm
// of the branch, gate, residual scale, norm of the stream, and the experts'
// input in FP8.
//
// Each byte is read and written once, a row at a time: its elements stay in
// registers between the two norms, which need a sum over the row each.  (h's
// could be formed from sums known before it, but not where r and the branch cancel.)
// HBM bounds it; what there is to hide is a row's chain of sums (8192 x 4096 with an FP32 stream
// 66 us, 6.1 TB/s; 16384 x 7168 with codes 160 us, 6.6 TB/s; one row of 7168 4.0 us).
#include <atomic>
#include <type_traits>

#include "norm.cuh"

namespace moe {
namespace {

struct NormParams {
  RowsOf y, r, gate, h, z;
  const void* w_post;
  const void* w_pre;
  uint8_t* q;
  float* q_scale;
  const int32_t* num_rows;
  int64_t M;
  int H, wide, gate_mode, post_norm, pow2;
  int team;                         // threads of a row
  int stages;                       // rows of a team in shared memory
  float residual_scale, weight_offset, eps;
};

// Eight values over one scale as E4M3 codes, each from the correctly rounded quotient: the product
// with the reciprocal, corrected twice by its residual (Markstein), which is exact where no
// value that rounds to a code is near FP32's smallest; one of them by a divide otherwise.
__device__ __forceinline__ uint2 codes_of(const float2 (&f)[4], float s) {
  uint32_t code[2] = {0, 0};
  if (s >= 0x1p-80f && s <= 0x1p100f) {
    const float2 inv = both(__frcp_rn(s)), minus = both(-s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 q = mul2(f[i], inv);
      q = fma2(fma2(minus, q, f[i]), inv, q);
      q = fma2(fma2(minus, q, f[i]), inv, q);
      code[i / 2] |= static_cast<uint32_t>(cvt_e4m3x2(q.x, q.y)) << (16 * (i % 2));
    }
  } else if (s > 0.f) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      code[i / 2] |= static_cast<uint32_t>(cvt_e4m3x2(__fdiv_rn(f[i].x, s), __fdiv_rn(f[i].y, s))) << (16 * (i % 2));
  }
  return make_uint2(code[0], code[1]);
}

// What a fixed variant keeps in shared memory, as the gradient does: for each warp of a team the
// weights (post, or the channel gate, or their product; pre) in FP32, which its teams
// share, then for each warp p.stages times the pieces of a row's inputs (y, r, gate).
template <typename Tb, typename Ts, int kVec, int kPost, int kGate>
struct Layout {
  static constexpr int kB = kPieces<Tb>, kS = kPieces<Ts>;
  static constexpr int kAtR = kVec * kB, kAtG = kAtR + kVec * kS, kUnits = kAtG + (kGate == MOE_GATE_FULL ? kVec * kB : 0);
  static constexpr int kAtPost = 2 * kVec, kWeights = kAtPost + (kPost || kGate == MOE_GATE_CHANNEL ? 2 * kVec : 0);
  static __host__ __device__ constexpr int bytes(int team, int teams, int stages) {
    return (kWeights + teams * stages * kUnits) * (kPiece / 32) * team;
  }
};

// The sum over a team of one value: every thread gets the same bits.
__device__ __forceinline__ float team_sum(float v, float (*part)[32], int& turn, int warps, int index) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (warps == 1) return v;
  const int lane = threadIdx.x % 32;
  if (lane == 0) part[turn][threadIdx.x / 32] = v;
  named_barrier(1 + index, 32 * warps);
  v = lane < warps ? part[turn][index * warps + lane] : 0.f;
  turn ^= 1;                                // (the next sum's parts: a thread behind still reads these)
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A row's team is `team` threads with kVec vectors of eight columns each; a CTA holds several
// teams, each with its own rows and barrier, and keeps their next rows' inputs on the way into
// shared memory.  kPost, kGate (a token's as none: it is a number): a variant fixed at compile time;
// kGate = -1: any variant, from memory itself.
template <typename Tb, typename Ts, int kVec, int kPost, int kGate>
__global__ void __launch_bounds__(1024, 1) norm_kernel(const __grid_constant__ NormParams p) {
  constexpr bool kFixed = kGate >= 0;
  constexpr bool kShared = kFixed && sizeof(Ts) == 4;
  using At = Layout<Tb, Ts, kVec, kPost == 1, kGate>;
  __shared__ float part[2][32];
  extern __shared__ __align__(16) uint8_t memory[];
  pdl_wait();
  pdl_launch_dependents();
  const int team = p.team, mine = threadIdx.x / team, tid = threadIdx.x - mine * team, teams = blockDim.x / team;
  const int lane = threadIdx.x % 32, warps = team / 32;
  const int gate = kFixed ? kGate : p.gate_mode == MOE_GATE_TOKEN ? MOE_GATE_NONE : p.gate_mode;
  const bool post = kFixed ? kPost != 0 : p.post_norm != 0, has_r = p.r.p != nullptr, second = p.z.p || p.q;
  const bool token_gate = gate == MOE_GATE_NONE && p.gate_mode == MOE_GATE_TOKEN;
  const uint32_t M = static_cast<uint32_t>(p.M), live = p.num_rows ? min(static_cast<uint32_t>(max(*p.num_rows, 0)), M) : M;
  const uint32_t step = gridDim.x * teams;
  const float inv_h = 1.f / static_cast<float>(p.H);
  const Places in = places(lane);
  const uint32_t w_at = smem_u32(memory) + (tid / 32) * (At::kWeights * kPiece) + 16u * lane;
  auto column = [&](int v) { return 8 * (tid + v * team); };
  Tb* const of_branch = nullptr;
  Ts* const of_stream = nullptr;

  auto get = [&](auto* type, const RowsOf& rows, int piece, uint32_t at, uint32_t row, int c, float2 (&f)[4]) {
    using T = std::remove_pointer_t<decltype(type)>;
    if constexpr (kFixed)
      widen2<T>(from_pieces<T>(in, at, piece), f);
    else
      widen2<T>(load_vec<T>(reinterpret_cast<const T*>(rows.at<false>(row, c * sizeof(T)))), f);
  };
  auto put = [&](auto* type, const RowsOf& rows, int piece, uint32_t at, uint32_t row, int c, const float2 (&f)[4]) {
    using T = std::remove_pointer_t<decltype(type)>;
    if constexpr (kFixed && sizeof(T) == 4)
      put_pieces(in, at, piece, f);
    else
      store2<T>(reinterpret_cast<T*>(rows.at<kFixed>(row, c * sizeof(T))), f);
  };
  auto weights = [&](int piece, float2 (&f)[4]) {
    widen2<float>(Vec8<float>{shared16(w_at + piece * kPiece), shared16(w_at + (piece + 1) * kPiece)}, f);
  };
  // the columns' factor of the branch: its norm's weights, a channel gate, or their product
  auto factor = [&](int c, float2 (&f)[4]) {
    if (post) weights2<Tb>(p.w_post, p.wide, c, p.weight_offset, f);
    if (gate == MOE_GATE_CHANNEL) {
      float2 g[4];
      weights2<Tb>(p.gate.p, p.wide, c, 0.f, g);
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = post ? mul2(f[i], g[i]) : g[i];
    }
  };
  auto fetch_row = [&](uint32_t at, uint32_t row) {
    if constexpr (kFixed) {
      if (row < live) {
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
          const int c = column(v);
          to_pieces(in, at, v * At::kB, At::kB, p.y, row, c, p.H);
          if (has_r) to_pieces(in, at, At::kAtR + v * At::kS, At::kS, p.r, row, c, p.H);
          if (gate == MOE_GATE_FULL) to_pieces(in, at, At::kAtG + v * At::kB, At::kB, p.gate, row, c, p.H);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  };

  uint32_t row = blockIdx.x * teams + mine;
  const uint32_t first = smem_u32(memory) + (team / 32) * (At::kWeights * kPiece) +
                         (threadIdx.x / 32) * (p.stages * (At::kUnits * kPiece));
  const uint32_t end = first + p.stages * (At::kUnits * kPiece);
  uint32_t at = first, free = first;
  int turn = 0;
  if constexpr (kFixed) {
    for (int i = 0; i < p.stages - 1; ++i, free += At::kUnits * kPiece) fetch_row(free, row + i * step);
    if (mine == 0) {
#pragma unroll
      for (int v = 0; v < kVec; ++v) {
        const int c = column(v);
        if (c < p.H) {
          float2 f[4];
          weights2<Tb>(p.w_pre, p.wide, c, p.weight_offset, f);
          put16(w_at + 2 * v * kPiece, f[0], f[1]);
          put16(w_at + (2 * v + 1) * kPiece, f[2], f[3]);
          if (post || gate == MOE_GATE_CHANNEL) {
            factor(c, f);
            put16(w_at + (At::kAtPost + 2 * v) * kPiece, f[0], f[1]);
            put16(w_at + (At::kAtPost + 2 * v + 1) * kPiece, f[2], f[3]);
          }
        }
      }
    }
    if (teams > 1) __syncthreads();
  }

  for (; row < live; row += step) {
    if constexpr (kShared) __syncwarp();    // (every lane is done with the row that was there)
    fetch_row(free, row + (p.stages - 1) * step);
    if constexpr (kFixed) {
      if (p.stages == 3)
        asm volatile("cp.async.wait_group 2;" ::: "memory");
      else
        asm volatile("cp.async.wait_group 1;" ::: "memory");
      if constexpr (kShared) __syncwarp();  // (the other lanes' copies)
    }
    float2 h[kVec][4];
    float root = 1.f;
#pragma unroll
    for (int v = 0; v < kVec; ++v)
      if (column(v) < p.H) get(of_branch, p.y, v * At::kB, at, row, column(v), h[v]);
    if (post) {
      float2 sum = {};
#pragma unroll
      for (int v = 0; v < kVec; ++v)
        if (column(v) < p.H) {
#pragma unroll
          for (int i = 0; i < 4; ++i) sum = fma2(h[v][i], h[v][i], sum);
        }
      root = rsqrtf(fmaf(team_sum(sum.x + sum.y, part, turn, warps, mine), inv_h, p.eps));
    }
    if (token_gate) root *= __ldg(static_cast<const float*>(p.gate.p) + row);
    float2 sum = {};
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const int c = column(v);
      if (c < p.H) {
        if (post || token_gate) {
#pragma unroll
          for (int i = 0; i < 4; ++i) h[v][i] = mul2(h[v][i], both(root));
        }
        if (post || gate == MOE_GATE_CHANNEL) {
          float2 w[4];
          if constexpr (kFixed) weights(At::kAtPost + 2 * v, w); else factor(c, w);
#pragma unroll
          for (int i = 0; i < 4; ++i) h[v][i] = mul2(h[v][i], w[i]);
        }
        if (gate == MOE_GATE_FULL) {
          float2 g[4];
          get(of_branch, p.gate, At::kAtG + v * At::kB, at, row, c, g);
#pragma unroll
          for (int i = 0; i < 4; ++i) h[v][i] = mul2(h[v][i], g[i]);
        }
        if (has_r) {
          float2 r[4];
          get(of_stream, p.r, At::kAtR + v * At::kS, at, row, c, r);
#pragma unroll
          for (int i = 0; i < 4; ++i) h[v][i] = fma2(both(p.residual_scale), r[i], h[v][i]);
        }
        if (p.h.p) put(of_stream, p.h, At::kAtR + v * At::kS, at, row, c, h[v]);
#pragma unroll
        for (int i = 0; i < 4; ++i) sum = fma2(h[v][i], h[v][i], sum);
      }
    }
    if constexpr (kShared) {
      __syncwarp();
      if (p.h.p) {
#pragma unroll
        for (int v = 0; v < kVec; ++v) flush_pieces(in, at, At::kAtR + v * At::kS, p.h, row, column(v), p.H);
      }
    }
    if (second) {
      root = rsqrtf(fmaf(team_sum(sum.x + sum.y, part, turn, warps, mine), inv_h, p.eps));
#pragma unroll
      for (int v = 0; v < kVec; ++v) {
        const int c = column(v);
        const bool live_column = c < p.H;
        if (live_column) {
          float2 w[4];
          if constexpr (kFixed) weights(2 * v, w); else weights2<Tb>(p.w_pre, p.wide, c, p.weight_offset, w);
#pragma unroll
          for (int i = 0; i < 4; ++i) h[v][i] = mul2(mul2(h[v][i], both(root)), w[i]);
          if (p.z.p) put(of_branch, p.z, v * At::kB, at, row, c, h[v]);
        }
        if (p.q) {
          // (a group of 128 columns is 16 neighbouring lanes: all of them or none have columns)
          // (a NaN reaches the scale: the codes alone could lose it)
          float amax = 0.f;
          if (live_column) {
#pragma unroll
            for (int i = 0; i < 4; ++i) amax = max_nan(amax, max_nan(fabsf(h[v][i].x), fabsf(h[v][i].y)));
          }
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          float s = __fdiv_rn(amax, 448.f);
          if (p.pow2 && s > 0.f) s = pow2_round_up(s);
          if (live_column && MOE_IN_BOUNDS(row < M)) {
            *reinterpret_cast<uint2*>(p.q + static_cast<int64_t>(row) * p.H + c) = codes_of(h[v], s);
            if (lane % 16 == 0) p.q_scale[static_cast<int64_t>(row) * (p.H / 128) + c / 128] = s;
          }
        }
      }
      if constexpr (kFixed && sizeof(Tb) == 4) {
        __syncwarp();
        if (p.z.p) {
#pragma unroll
          for (int v = 0; v < kVec; ++v) flush_pieces(in, at, v * At::kB, p.z, row, column(v), p.H);
        }
      }
    }
    free = at;
    at = at + At::kUnits * kPiece == end ? first : at + At::kUnits * kPiece;
  }
}

// (FP32 streams: beyond, one team and three stages are faster than two of two)
constexpr int kMostShared = 224 * 1024, kMostWideRing = 112 * 1024;

template <typename Tb, typename Ts, int kVec, int kPost, int kGate>
cudaError_t launch_teams(NormParams& p, int sms, cudaStream_t stream) {
  constexpr bool kFixed = kGate >= 0;
  using At = Layout<Tb, Ts, kVec, kPost == 1, kGate>;
  p.team = team_threads(p.H / 8, kVec);
  int teams = 1024 / p.team;
  if (p.team > 32 && teams > 15) teams = 15;     // (a named barrier each)
  auto fits = [&](int n) {
    const int all = At::bytes(p.team, n, 2);
    return all <= kMostShared && (sizeof(Ts) == 2 || all - At::bytes(p.team, 0, 2) <= kMostWideRing);
  };
  while (kFixed && teams > 1 && !fits(teams)) --teams;
  if (ceil_div(p.M, sms) < teams) teams = static_cast<int>(ceil_div(p.M, sms));
  // Several teams hide one another's sums, and two stages each are enough (8192 x 4096 with one norm:
  // 43 us, 47 with three); one team needs a row more on the way (FP32 rows of 4096 columns, which
  // fill the ring alone: 84 us, 90 with two; 87 as two teams of three stages).
  p.stages = teams == 1 && At::bytes(p.team, 1, 3) <= kMostShared ? 3 : 2;
  const int64_t want = ceil_div(p.M, teams), most = kFixed ? sms : 8 * sms;
  auto kernel = norm_kernel<Tb, Ts, kVec, kPost, kGate>;
  static std::atomic<bool> sized[64];            // per device: the attribute outlasts the call
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (kFixed && err == cudaSuccess && (dev >= 64 || !sized[dev].load())) {
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostShared);
    if (err == cudaSuccess && dev < 64) sized[dev].store(true);
  }
  if (err != cudaSuccess) return err;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(want < most ? want : most)), dim3(p.team * teams),
                    kFixed ? static_cast<size_t>(At::bytes(p.team, teams, p.stages)) : 0, stream, 1, p);
}

// The fixed variant where a row of it fits, else the one for any.
template <typename Tb, typename Ts, int kPost, int kGate>
cudaError_t launch_fixed(NormParams& p, int sms, cudaStream_t stream) {
  // One vector a thread while two teams fit a CTA, for a few rows (latency), and up to 896 where
  // a row has enough to move for the time of its sums: one norm (16384 x 7168 with FP8 output: 160
  // us, 178 as two teams with two vectors a thread) or an FP32 stream (8192 x 7168: 105, 124);
  // not for two norms in 16 bits (8192 x 7168: 107, 91).
  const int vecs = p.H / 8, one = team_threads(vecs, 1), two = team_threads(vecs, 2);
  if (vecs <= 512 || (vecs <= 896 && (!kPost || sizeof(Ts) == 4)) || (p.M <= sms && vecs <= 1024)) {
    if (Layout<Tb, Ts, 1, kPost, kGate>::bytes(one, 1, 2) <= kMostShared) return launch_teams<Tb, Ts, 1, kPost, kGate>(p, sms, stream);
  } else if (Layout<Tb, Ts, 2, kPost, kGate>::bytes(two, 1, 2) <= kMostShared) {
    return launch_teams<Tb, Ts, 2, kPost, kGate>(p, sms, stream);
  }
  return vecs <= 1024 ? launch_teams<Tb, Ts, 1, -1, -1>(p, sms, stream) : launch_teams<Tb, Ts, 2, -1, -1>(p, sms, stream);
}
template <typename Tb, typename Ts, int kPost>
cudaError_t launch_gate(NormParams& p, int sms, cudaStream_t stream) {
  return p.gate_mode == MOE_GATE_FULL      ? launch_fixed<Tb, Ts, kPost, MOE_GATE_FULL>(p, sms, stream)
         : p.gate_mode == MOE_GATE_CHANNEL ? launch_fixed<Tb, Ts, kPost, MOE_GATE_CHANNEL>(p, sms, stream)
                                           : launch_fixed<Tb, Ts, kPost, MOE_GATE_NONE>(p, sms, stream);
}
template <typename Tb, typename Ts>
cudaError_t launch_norm(NormParams& p, int sms, cudaStream_t stream) {
  bool near = true;                              // row strides below 4 GB
  for (const RowsOf* r : {&p.y, &p.r, &p.gate, &p.h, &p.z}) near = near && r->ld < (int64_t(1) << 32);
  if (!near) return launch_teams<Tb, Ts, 2, -1, -1>(p, sms, stream);
  return p.post_norm ? launch_gate<Tb, Ts, 1>(p, sms, stream) : launch_gate<Tb, Ts, 0>(p, sms, stream);
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
  p.y = {a->y, a->ldy * eb};
  p.r = {a->r, a->ldr * es};
  p.gate = {gate, a->gate_mode == MOE_GATE_FULL ? a->ldgate * eb : 0};
  p.h = {a->h, a->ldh * es};
  p.z = {a->z, a->ldz * eb};
  p.w_post = w_post;
  p.w_pre = w_pre;
  p.q = a->q;
  p.q_scale = a->q_scale;
  p.num_rows = a->num_rows;
  p.M = M;
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
