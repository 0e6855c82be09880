// The gradient of the norms around a block (moe_norm_residual_backward).
//
// Row by row as the forward pass, with one round of sums over a row: what the branch's
// norm needs is linear in what the stream's norm adds, so that all six sums are formed from
// the inputs at once.  The gradients that are sums over rows (both weights', a channel gate's)
// gather in registers, each thread's columns over all of its rows; every CTA leaves its sums
// in the workspace, and a second launch adds them in a fixed order.
//
// HBM bounds it: 8192 x 4096 with an FP32 stream and a channel gate 95 us (6.4 TB/s), 16384 x
// 7168 with a full gate 293 us (6.4 TB/s).  Few rows: two launches and the parts (64 x 4096: 6.0 us).
#include <atomic>
#include <type_traits>

#include "norm.cuh"

namespace moe {
namespace {

constexpr int kMaxParts = 320;      // CTAs whose sums over rows the workspace holds
constexpr int kSums = 3;            // dw_pre, dw_post, a channel gate's
constexpr int kHeld = 2;            // ... of which the last two are one sum times the other's factor

struct NormGradParams {
  RowsOf y, h, gate, dh, dz, dy, dr, dgate;
  const void* w_post;
  const void* w_pre;
  float* parts;                     // [kSums, CTAs, H]
  const int32_t* num_rows;
  int64_t M;
  int H, wide, gate_mode, post_norm;
  int sums;                         // bit n: sum n is asked for
  int team;                         // threads of a row
  int stages;                       // rows of a team in shared memory
  float residual_scale, weight_offset, eps;
};

// The row sums that everything else follows from, with k = gate y (w_post + offset) and
// t = dz (w_pre + offset): one round of them, because the sum that the branch's norm needs is
// linear in dH:  sum k dH = sum k dh + R_h (sum k t - (R_h mean(t h)) (R_h sum k h)).
// A root's cube leaves FP32's range long before the root does (rows beyond 1e13, or of zeros with
// an eps below 1e-26), so each of its factors meets a sum or an element first.  Nothing hides the
// chain of scalars between a row's sums and its outputs, so it is kept short: with one more
// multiplication after another 16384 x 7168 with a full gate takes 297 to 301 us instead of 293.
enum { kHH, kTH, kYY, kKD, kKT, kKH, kRowSums = 8 };

// Sums of eight values over a warp: lane l ends with the total of value (l / 4) % 8.
__device__ __forceinline__ float warp_sums8(float (&v)[8], int lane) {
#pragma unroll
  for (int half = 4; half > 0; half /= 2) {
    const int o = 4 * half;
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float give = up ? v[i] : v[i + half], keep = up ? v[i + half] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
  return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}
// The totals over a team's warps' parts [warps][8]: lane l adds value l % 8 of every fourth warp.
__device__ __forceinline__ void join_sums8(const float* parts, int warps, int lane, float (&v)[8]) {
  float sum = 0.f;
  const float* mine = parts + lane;
  const int more = warps - lane / 8;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (4 * i < more) sum += mine[32 * i];
  sum += __shfl_xor_sync(0xffffffffu, sum, 8);
  sum += __shfl_xor_sync(0xffffffffu, sum, 16);
#pragma unroll
  for (int i = 0; i <= kKH; ++i) v[i] = __shfl_sync(0xffffffffu, sum, i);
}

// What a fixed variant keeps in shared memory: for each warp of a team the weights (pre; post, or
// the channel gate, or their product) in FP32, which its teams share, then for each warp
// p.stages times the pieces of a row's inputs (y, dz, h, dh, gate).
template <typename Tb, typename Ts, int kPre, int kPost, int kGate>
struct Layout {
  static constexpr int kB = kPieces<Tb>, kS = kPieces<Ts>;
  static constexpr int kAtZ = kB, kAtH = kAtZ + (kPre ? kB : 0), kAtD = kAtH + (kPre ? kS : 0), kAtG = kAtD + kS,
                       kUnits = kAtG + (kGate == MOE_GATE_FULL ? kB : 0);
  static constexpr int kAtPost = kPre ? 2 : 0, kWeights = kAtPost + (kPost || kGate == MOE_GATE_CHANNEL ? 2 : 0);
  // bytes of `teams` teams of `team` threads
  static __host__ __device__ constexpr int bytes(int team, int teams, int stages) {
    return (kWeights + teams * stages * kUnits) * (kPiece / 32) * team;
  }
};
constexpr int kMostStages = 3;      // (a fourth takes L1 and gives nothing; two: 8192 x 4096 75 us against 69 without post_norm)
// Threads of a fixed variant's CTA, by registers.  Up to 512 a thread keeps a row's vectors from
// the sums to the outputs (65536 rows of 256 columns: 39 us, 52 with 1024 threads that read
// shared memory twice); 7168 columns take 896, whose 72 registers just hold a thread's share: with
// the 64 of 1024 threads a few bytes spill, and beside a full shared memory the L1 has no room
// for them (16384 x 7168 with a full gate: 419 us against 305, which two stages made 294).
constexpr int kKeepThreads = 512, kFixedThreads = 896, kAnyThreads = 1024;

// A row's team is `team` threads with kVec vectors each; a CTA holds as many teams as fit, and
// each takes its own rows.  All sums of a row are formed in one round, so that its one barrier
// and the shuffles around it are what is not hidden; meanwhile the next rows'
// inputs are on their way into shared memory, every thread's vectors to its own place (the
// copies need no barrier), and with them HBM stays busy.
//
// kPre (dz and h given), kPost, kGate (a token's as none: it is a number): a variant fixed
// at compile time, its rows and weights in shared memory, kVec 1.  Branches on run-time flags cost
// 40% more instructions and, because loads do not move across them, half of the speed;
// weights from memory cost another 20%: they fall out of the L1 beside a full shared
// memory.  kPre = -1: any variant, from memory itself.
template <typename Tb, typename Ts, int kVec, int kPre, int kPost, int kGate, int kThreads>
__global__ void __launch_bounds__(kThreads, 1) norm_backward_kernel(const __grid_constant__ NormGradParams p) {
  constexpr bool kFixed = kPre >= 0;
  using At = Layout<Tb, Ts, kPre == 1, kPost == 1, kGate>;
  static_assert(!kFixed || kVec == 1, "one vector a thread");
  constexpr bool kShared = kFixed && sizeof(Ts) == 4;      // a warp's FP32 pieces are its lanes' together
  constexpr bool kKeep = kFixed && kThreads <= kKeepThreads;
  __shared__ float s_parts[2][kThreads / 32][kRowSums];
  extern __shared__ __align__(16) uint8_t memory[];
  pdl_wait();
  pdl_launch_dependents();
  const int team = p.team, mine = threadIdx.x / team, tid = threadIdx.x - mine * team, teams = blockDim.x / team;
  const int lane = threadIdx.x % 32, warps = team / 32;
  const int gate = kFixed ? kGate : p.gate_mode == MOE_GATE_TOKEN ? MOE_GATE_NONE : p.gate_mode;
  const bool post = kFixed ? kPost != 0 : p.post_norm != 0, pre = kFixed ? kPre != 0 : p.dz.p != nullptr;
  const bool own_h = kFixed ? kPre != 0 : p.h.p != nullptr, has_dh = p.dh.p != nullptr;
  const bool token_gate = gate == MOE_GATE_NONE && p.gate_mode == MOE_GATE_TOKEN;
  const bool dots = post || (token_gate && p.dgate.p);
  const uint32_t M = static_cast<uint32_t>(p.M), live = p.num_rows ? min(static_cast<uint32_t>(max(*p.num_rows, 0)), M) : M;
  const uint32_t step = gridDim.x * teams;
  const float inv_h = 1.f / static_cast<float>(p.H);
  const Places in = places(lane);
  const uint32_t of_weights = (tid / 32) * (At::kWeights * kPiece) + 16u * lane, w_at = smem_u32(memory) + of_weights;
  auto column = [&](int v) { return 8 * (tid + v * team); };

  // one vector of an input of row `row`, which is at `at` in shared memory
  auto get = [&](auto* type, const RowsOf& rows, int piece, uint32_t at, uint32_t row, int c, float2 (&f)[4]) {
    using T = std::remove_pointer_t<decltype(type)>;
    Vec8<T> r;
    if constexpr (kFixed) {
      r = from_pieces<T>(in, at, piece);
    } else {
      r = load_vec<T>(reinterpret_cast<const T*>(rows.at<false>(row, c * sizeof(T))));
    }
    widen2<T>(r, f);
  };
  Tb* const of_branch = nullptr;
  Ts* const of_stream = nullptr;
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
        const int c = column(0);
        auto bring = [&](int piece, int pieces, const RowsOf& rows) { to_pieces(in, at, piece, pieces, rows, row, c, p.H); };
        bring(0, At::kB, p.y);
        if (pre) bring(At::kAtZ, At::kB, p.dz), bring(At::kAtH, At::kS, p.h);
        if (has_dh) bring(At::kAtD, At::kS, p.dh);
        if (gate == MOE_GATE_FULL) bring(At::kAtG, At::kB, p.gate);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  };
  // one vector of an output: to memory, or (FP32, fixed variants) to the place of an input that
  // has been used, from where flush_row takes it
  auto put = [&](auto* type, const RowsOf& rows, int piece, uint32_t at, uint32_t row, int c, const float2 (&f)[4]) {
    using T = std::remove_pointer_t<decltype(type)>;
    if constexpr (kFixed && sizeof(T) == 4) {
      put_pieces(in, at, piece, f);
    } else {
      store2<T>(reinterpret_cast<T*>(rows.at<kFixed>(row, c * sizeof(T))), f);
    }
  };
  auto flush = [&](const RowsOf& rows, int piece, uint32_t at, uint32_t row) { flush_pieces(in, at, piece, rows, row, column(0), p.H); };

  if constexpr (kFixed) {
    const int c = column(0);
    if (mine == 0 && c < p.H) {
      auto keep = [&](const float2 (&f)[4], int piece) {
        put16(w_at + piece * kPiece, f[0], f[1]);
        put16(w_at + (piece + 1) * kPiece, f[2], f[3]);
      };
      float2 f[4];
      if (pre) {
        weights2<Tb>(p.w_pre, p.wide, c, p.weight_offset, f);
        keep(f, 0);
      }
      if (post || gate == MOE_GATE_CHANNEL) {
        factor(c, f);
        keep(f, At::kAtPost);
      }
    }
    if (teams > 1) __syncthreads();
  }

  float2 acc[kHeld][kVec][4];
#pragma unroll
  for (int n = 0; n < kHeld; ++n)
#pragma unroll
    for (int v = 0; v < kVec; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][v][i] = make_float2(0.f, 0.f);

  uint32_t row = blockIdx.x * teams + mine;
  // the stages in turn: `at` holds this row, `free` is for the row stages - 1 further on
  const uint32_t first = smem_u32(memory) + (team / 32) * (At::kWeights * kPiece) +
                         (threadIdx.x / 32) * ((kKeep ? p.stages : 2) * (At::kUnits * kPiece));
  const uint32_t end = first + (kKeep ? p.stages : 2) * (At::kUnits * kPiece);
  uint32_t at = first, free = first;
  int turn = 0;
  const int stages = kKeep ? p.stages : 2;
  if constexpr (kFixed) {
    for (int i = 0; i < stages - (kKeep ? 1 : 0); ++i, free += At::kUnits * kPiece) fetch_row(free, row + i * step);
  }
  for (; row < live; row += step) {
    if constexpr (kShared) __syncwarp();    // (every lane is done with the row that was there)
    if constexpr (kKeep) fetch_row(free, row + (stages - 1) * step);
    if constexpr (kFixed) {
      if (stages == 3)
        asm volatile("cp.async.wait_group 2;" ::: "memory");
      else
        asm volatile("cp.async.wait_group 1;" ::: "memory");
      if constexpr (kShared) __syncwarp();  // (the other lanes' copies)
    }
    // the row's inputs and the weights as they are needed; kKeep: once for both uses
    float2 y[4], x[4] = {}, z[4] = {}, d[4] = {}, g[4], w_pre[4], w[4];
    float2 sum[6] = {};
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const int c = column(v);
      if (c < p.H) {
        float2 k[4];
        get(of_branch, p.y, 0, at, row, c, y);
        if (pre) {
          if constexpr (kFixed) weights(0, w_pre); else weights2<Tb>(p.w_pre, p.wide, c, p.weight_offset, w_pre);
          if (own_h) get(of_stream, p.h, At::kAtH, at, row, c, x); else copy4(y, x);
          get(of_branch, p.dz, At::kAtZ, at, row, c, z);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            sum[kHH] = fma2(x[i], x[i], sum[kHH]);
            sum[kTH] = fma2(mul2(z[i], w_pre[i]), x[i], sum[kTH]);
          }
        }
        if (kKeep || dots) {
          copy4(y, k);
          if (post || gate == MOE_GATE_CHANNEL) {
            if constexpr (kFixed) weights(At::kAtPost, w); else factor(c, w);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (post) sum[kYY] = fma2(y[i], y[i], sum[kYY]);
              k[i] = mul2(y[i], w[i]);
            }
          }
          if (gate == MOE_GATE_FULL) {
            get(of_branch, p.gate, At::kAtG, at, row, c, g);
#pragma unroll
            for (int i = 0; i < 4; ++i) k[i] = mul2(k[i], g[i]);
          }
          if (has_dh) {
            get(of_stream, p.dh, At::kAtD, at, row, c, d);
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[kKD] = fma2(k[i], d[i], sum[kKD]);
          }
          if (pre) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              sum[kKT] = fma2(k[i], mul2(z[i], w_pre[i]), sum[kKT]);
              sum[kKH] = fma2(k[i], x[i], sum[kKH]);
            }
          }
        }
      }
    }
    float s[8] = {};
#pragma unroll
    for (int i = 0; i < 6; ++i) s[i] = sum[i].x + sum[i].y;
    const float total = warp_sums8(s, lane);
    if (lane % 4 == 0) s_parts[turn][threadIdx.x / 32][lane / 4] = total;
    if (warps == 1)
      __syncwarp();
    else
      named_barrier(1 + mine, team);
    join_sums8(&s_parts[turn][mine * warps][0], warps, lane, s);
    turn ^= 1;                              // (the next row's parts: a thread behind still reads these)
    const float root_h = pre ? rsqrtf(fmaf(s[kHH], inv_h, p.eps)) : 0.f, root_y = post ? rsqrtf(fmaf(s[kYY], inv_h, p.eps)) : 1.f;
    const float token = token_gate ? __ldg(static_cast<const float*>(p.gate.p) + row) : 1.f;
    const float mean_h = root_h * (s[kTH] * inv_h);                                             // of t h R
    const float dot = fmaf(root_h, fmaf(-mean_h, root_h * s[kKH], s[kKT]), s[kKD]);             // sum k dH (without a token's gate)
    const float mean_y = root_y * inv_h * dot;
    if (token_gate && p.dgate.p && tid == 0) static_cast<float*>(const_cast<void*>(p.dgate.p))[row] = root_y * dot;
    // the factors of h R and of y R (with a token's gate)
    const float2 rh2 = both(root_h), bh2 = both(-mean_h * root_h), by2 = both(-mean_y * root_y), ry2 = both(root_y * token);
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const int c = column(v);
      if (c < p.H) {
        if (!kKeep) {
          get(of_branch, p.y, 0, at, row, c, y);
          if (has_dh) {
            get(of_stream, p.dh, At::kAtD, at, row, c, d);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) d[i] = make_float2(0.f, 0.f);
          }
        }
        if (pre) {
          if (!kKeep) {
            if constexpr (kFixed) weights(0, w_pre); else weights2<Tb>(p.w_pre, p.wide, c, p.weight_offset, w_pre);
            if (own_h) get(of_stream, p.h, At::kAtH, at, row, c, x); else copy4(y, x);
            get(of_branch, p.dz, At::kAtZ, at, row, c, z);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] = mul2(x[i], rh2);
            acc[0][v][i] = fma2(z[i], x[i], acc[0][v][i]);
            d[i] = fma2(mul2(z[i], rh2), w_pre[i], fma2(x[i], bh2, d[i]));
          }
        }
        if (p.dr.p) {
          float2 o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = mul2(d[i], both(p.residual_scale));
          put(of_stream, p.dr, At::kAtD, at, row, c, o);
        }
        if ((post || gate == MOE_GATE_CHANNEL) && !kKeep) {
          if constexpr (kFixed) weights(At::kAtPost, w); else factor(c, w);
        }
        if (post) {
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = mul2(y[i], ry2);
        }
        if (gate == MOE_GATE_FULL) {
          float2 o[4];                      // dH u, u = y R(y) (w_post + offset) or y
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = mul2(d[i], post ? mul2(y[i], w[i]) : y[i]);
          if (!kKeep) get(of_branch, p.gate, At::kAtG, at, row, c, g);
          if (p.dgate.p) put(of_branch, p.dgate, At::kAtG, at, row, c, o);
#pragma unroll
          for (int i = 0; i < 4; ++i) d[i] = mul2(d[i], g[i]);
        }
        if (post || gate == MOE_GATE_CHANNEL) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            acc[1][v][i] = fma2(d[i], y[i], acc[1][v][i]);
            d[i] = post ? fma2(mul2(d[i], ry2), w[i], mul2(y[i], by2)) : mul2(d[i], w[i]);
          }
        } else if (gate == MOE_GATE_NONE) {
#pragma unroll
          for (int i = 0; i < 4; ++i) d[i] = mul2(d[i], ry2);
        }
        if (p.dy.p) put(of_branch, p.dy, 0, at, row, c, d);
      }
    }
    if constexpr (kShared) {
      __syncwarp();
      if (p.dr.p) flush(p.dr, At::kAtD, at, row);
      if constexpr (sizeof(Tb) == 4) {
        if (gate == MOE_GATE_FULL && p.dgate.p) flush(p.dgate, At::kAtG, at, row);
        if (p.dy.p) flush(p.dy, 0, at, row);
      }
    }
    // (two stages: a row's place is asked for again as soon as it is done with)
    free = at;
    if constexpr (!kKeep) {
      if constexpr (kShared) __syncwarp();
      fetch_row(at, row + 2 * step);
    }
    at = at + At::kUnits * kPiece == end ? first : at + At::kUnits * kPiece;
  }

  if (!p.sums) return;
  // the teams' sums one after another into the first one's, then out
  if constexpr (kFixed) asm volatile("cp.async.wait_group 0;" ::: "memory");
  float2* gathered = reinterpret_cast<float2*>(memory);
  for (int m = 1; m < teams; ++m) {
    __syncthreads();                             // (the ring, then the last team's sums, are no longer read)
    if (mine == m) {
#pragma unroll
      for (int n = 0; n < kHeld; ++n)
#pragma unroll
        for (int v = 0; v < kVec; ++v)
#pragma unroll
          for (int i = 0; i < 4; ++i) gathered[((n * kVec + v) * 4 + i) * team + tid] = acc[n][v][i];
    }
    __syncthreads();
    if (mine == 0) {
#pragma unroll
      for (int n = 0; n < kHeld; ++n)
#pragma unroll
        for (int v = 0; v < kVec; ++v)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[n][v][i] = add2(acc[n][v][i], gathered[((n * kVec + v) * 4 + i) * team + tid]);
    }
  }
  if (mine == 0) {
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const int c = column(v);
      if (c < p.H) {
        auto leave = [&](int n, const float2 (&f)[4]) {
          if ((p.sums >> n) & 1) store2<float>(p.parts + (static_cast<int64_t>(n) * gridDim.x + blockIdx.x) * p.H + c, f);
        };
        leave(0, acc[0][v]);
        if (gate == MOE_GATE_CHANNEL) {
          // one sum, dH y R(y), times what each gradient has beside it
          float2 f[4], g[4];
          weights2<Tb>(p.gate.p, p.wide, c, 0.f, g);
          weights2<Tb>(post ? p.w_post : nullptr, p.wide, c, p.weight_offset, f);
#pragma unroll
          for (int i = 0; i < 4; ++i) g[i] = mul2(g[i], acc[1][v][i]), f[i] = mul2(f[i], acc[1][v][i]);
          leave(1, g);
          leave(2, f);
        } else {
          leave(1, acc[1][v]);
        }
      }
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

constexpr int kMostShared = 224 * 1024;

template <typename Tb, typename Ts, int kVec, int kPre, int kPost, int kGate, int kThreads>
cudaError_t launch_teams(NormGradParams& p, int sms, int* ctas, cudaStream_t stream) {
  constexpr bool kFixed = kPre >= 0;
  using At = Layout<Tb, Ts, kPre == 1, kPost == 1, kGate>;
  p.team = team_threads(p.H / 8, kVec);
  // teams: as many as threads, named barriers and shared memory allow, but first one on every SM;
  // then as many stages as fit
  int teams = kThreads / p.team;
  if (p.team > 32 && teams > 15) teams = 15;
  while (kFixed && teams > 1 && At::bytes(p.team, teams, 2) > kMostShared) --teams;
  const int64_t rows = p.M < 1 ? 1 : p.M;
  if (ceil_div(rows, sms) < teams) teams = static_cast<int>(ceil_div(rows, sms));
  const int threads = p.team * teams;
  const int64_t want = ceil_div(rows, teams);
  *ctas = static_cast<int>(want < sms ? want : sms < kMaxParts ? sms : kMaxParts);
  p.stages = 2;
  while (kFixed && kThreads <= kKeepThreads && p.stages < kMostStages && At::bytes(p.team, teams, p.stages + 1) <= kMostShared) ++p.stages;
  const int held = kFixed ? At::bytes(p.team, teams, p.stages) : 0, join = teams > 1 ? kHeld * kVec * 32 * p.team : 0;
  auto kernel = norm_backward_kernel<Tb, Ts, kVec, kPre, kPost, kGate, kThreads>;
  static std::atomic<bool> sized[64];            // per device: the attribute outlasts the call
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err == cudaSuccess && (dev >= 64 || !sized[dev].load())) {
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostShared);
    if (err == cudaSuccess && dev < 64) sized[dev].store(true);
  }
  if (err != cudaSuccess) return err;
  return launch_pdl(kernel, dim3(*ctas), dim3(threads), static_cast<size_t>(held > join ? held : join), stream, 1, p);
}

// The fixed variant where a row of it fits, else the one for any.
template <typename Tb, typename Ts, int kPre, int kPost, int kGate>
cudaError_t launch_fixed(NormGradParams& p, int sms, int* ctas, cudaStream_t stream) {
  const int team = team_threads(p.H / 8, 1);
  return Layout<Tb, Ts, kPre, kPost, kGate>::bytes(team, 1, 2) > kMostShared ? launch_teams<Tb, Ts, 1, -1, -1, -1, kAnyThreads>(p, sms, ctas, stream)
         : team <= kKeepThreads     ? launch_teams<Tb, Ts, 1, kPre, kPost, kGate, kKeepThreads>(p, sms, ctas, stream)
         : team <= kFixedThreads    ? launch_teams<Tb, Ts, 1, kPre, kPost, kGate, kFixedThreads>(p, sms, ctas, stream)
                                    : launch_teams<Tb, Ts, 1, kPre, kPost, kGate, kAnyThreads>(p, sms, ctas, stream);
}
template <typename Tb, typename Ts, int kPre, int kPost>
cudaError_t launch_gate(NormGradParams& p, int sms, int* ctas, cudaStream_t stream) {
  return p.gate_mode == MOE_GATE_FULL      ? launch_fixed<Tb, Ts, kPre, kPost, MOE_GATE_FULL>(p, sms, ctas, stream)
         : p.gate_mode == MOE_GATE_CHANNEL ? launch_fixed<Tb, Ts, kPre, kPost, MOE_GATE_CHANNEL>(p, sms, ctas, stream)
                                           : launch_fixed<Tb, Ts, kPre, kPost, MOE_GATE_NONE>(p, sms, ctas, stream);
}

template <typename Tb, typename Ts>
cudaError_t launch_backward(NormGradParams& p, int sms, int* ctas, cudaStream_t stream) {
  if (p.H > 8 * kAnyThreads) return launch_teams<Tb, Ts, 2, -1, -1, -1, kAnyThreads>(p, sms, ctas, stream);
  bool near = true;                              // row strides below 4 GB
  for (const RowsOf* r : {&p.y, &p.h, &p.gate, &p.dh, &p.dz, &p.dy, &p.dr, &p.dgate}) near = near && r->ld < (int64_t(1) << 32);
  if (!near || !p.dz.p != !p.h.p || (!p.dz.p && !p.post_norm))
    return launch_teams<Tb, Ts, 1, -1, -1, -1, kAnyThreads>(p, sms, ctas, stream);
  return !p.dz.p       ? launch_gate<Tb, Ts, 0, 1>(p, sms, ctas, stream)
         : p.post_norm ? launch_gate<Tb, Ts, 1, 1>(p, sms, ctas, stream)
                       : launch_gate<Tb, Ts, 1, 0>(p, sms, ctas, stream);
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
  p.y = {a->y, a->ldy * eb};
  p.h = {h, a->ldh * es};
  p.gate = {gate, full ? a->ldgate * eb : 0};
  p.dh = {a->dh, a->lddh * es};
  p.dz = {a->dz, a->lddz * eb};
  p.dy = {a->dy, a->lddy * eb};
  p.dr = {a->dr, a->lddr * es};
  p.dgate = {a->dgate, full ? a->lddgate * eb : 0};
  p.w_post = w_post;
  p.w_pre = w_pre;
  p.parts = static_cast<float*>(a->workspace);
  p.num_rows = a->num_rows;
  p.M = M;
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
