// Shared by the norms around a block and their gradient (include/moe_block.h):
// vectors of eight elements of any type, sums over a row, host-side checks.
#pragma once

#include "../../include/moe_block.h"
#include "train.cuh"

namespace moe {

constexpr int kNormMaxH = 16384;

// Eight consecutive elements as they lie in memory.
template <typename T> struct Vec8 { uint4 v; };
template <> struct Vec8<float> { uint4 v, w; };

template <typename T>
__device__ __forceinline__ Vec8<T> load_vec(const T* p) {
  if constexpr (sizeof(T) == 4) {
    const uint4* q = reinterpret_cast<const uint4*>(p);
    return {q[0], q[1]};
  } else {
    return {*reinterpret_cast<const uint4*>(p)};
  }
}
template <typename T>
__device__ __forceinline__ void widen(const Vec8<T>& r, float (&f)[8]) {
  if constexpr (sizeof(T) == 4) {
    const uint32_t w[8] = {r.v.x, r.v.y, r.v.z, r.v.w, r.w.x, r.w.y, r.w.z, r.w.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
  } else {
    unpack8<T>(r.v, f);
  }
}
// One rounding to the type.
template <typename T>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[8]) {
  uint4* q = reinterpret_cast<uint4*>(p);
  if constexpr (sizeof(T) == 4) {
    q[0] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    q[1] = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
  } else {
    q[0] = pack8<T>(f);
  }
}

// Eight weights from column c on: FP32 or the branch's type, plus the offset; 1 without weights.
template <typename T>
__device__ __forceinline__ void load_weights(const void* w, int wide, int c, float offset, float (&f)[8]) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 1.f;
    return;
  }
  if (wide)
    widen<float>(load_vec<float>(static_cast<const float*>(w) + c), f);
  else
    widen<T>(load_vec<T>(static_cast<const T*>(w) + c), f);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] += offset;
}

// Sums over a row by its team: a warp, or the whole CTA through shared memory, one
// barrier a call (two buffers in turn: the next call writes the other one).  Every
// thread gets the same bits.
template <int kN, bool kWarpRow>
__device__ __forceinline__ void row_sums(float (&v)[kN], float (*part)[kN][32], int& turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int n = 0; n < kN; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
  if (kWarpRow) return;
  const int lane = threadIdx.x % 32, warps = blockDim.x / 32;
  if (lane == 0)
#pragma unroll
    for (int n = 0; n < kN; ++n) part[turn][n][threadIdx.x / 32] = v[n];
  __syncthreads();
#pragma unroll
  for (int n = 0; n < kN; ++n) v[n] = lane < warps ? part[turn][n][lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int n = 0; n < kN; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
  turn ^= 1;
}

// ---- pairs of FP32 values: one instruction each for two (packed arithmetic of sm_100)

__device__ __forceinline__ uint64_t bits2(float2 a) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
  return r;
}
__device__ __forceinline__ float2 pair2(uint64_t a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
  return pair2(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
  return pair2(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
  return pair2(r);
}
__device__ __forceinline__ void copy4(const float2 (&a)[4], float2 (&b)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = a[i];
}

template <typename T>
__device__ __forceinline__ void widen2(const Vec8<T>& r, float2 (&f)[4]) {
  if constexpr (sizeof(T) == 4) {
    const uint32_t w[8] = {r.v.x, r.v.y, r.v.z, r.v.w, r.w.x, r.w.y, r.w.z, r.w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
  } else {
    const uint32_t w[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = Pack2<T>::load(w[i]);
  }
}
template <typename T>
__device__ __forceinline__ void store2(T* p, const float2 (&f)[4]) {
  uint4* q = reinterpret_cast<uint4*>(p);
  if constexpr (sizeof(T) == 4) {
    q[0] = make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x), __float_as_uint(f[1].y));
    q[1] = make_uint4(__float_as_uint(f[2].x), __float_as_uint(f[2].y), __float_as_uint(f[3].x), __float_as_uint(f[3].y));
  } else {
    q[0] = make_uint4(Pack2<T>::store(f[0].x, f[0].y), Pack2<T>::store(f[1].x, f[1].y), Pack2<T>::store(f[2].x, f[2].y),
                      Pack2<T>::store(f[3].x, f[3].y));
  }
}
template <typename T>
__device__ __forceinline__ void weights2(const void* w, int wide, int c, float offset, float2 (&f)[4]) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = both(1.f);
    return;
  }
  if (wide)
    widen2<float>(load_vec<float>(static_cast<const float*>(w) + c), f);
  else
    widen2<T>(load_vec<T>(static_cast<const T*>(w) + c), f);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = add2(f[i], both(offset));
}

// Sums over a row by its team, one of several in a CTA: whole warps, by shuffles and, for more
// than one, through shared memory with a barrier of its own (two buffers in turn: the
// next call writes the other one).  Every thread gets the same bits.
template <int kN>
__device__ __forceinline__ void team_sums(float (&v)[kN], float (*part)[3][32], int& turn, int team, int index) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int n = 0; n < kN; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
  if (team == 32) return;
  const int lane = threadIdx.x % 32, warps = team / 32, first = index * warps;
  if (lane == 0)
#pragma unroll
    for (int n = 0; n < kN; ++n) part[turn][n][threadIdx.x / 32] = v[n];
  named_barrier(1 + index, team);
#pragma unroll
  for (int n = 0; n < kN; ++n) v[n] = lane < warps ? part[turn][n][first + lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int n = 0; n < kN; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
  turn ^= 1;
}

// ---------------------------------------------------------------- host side

// A buffer an entry point was given: rows of `width` bytes, `ld` bytes apart.
struct Span {
  const void* p;
  int64_t rows, ld, width;
};
inline Span span(const void* p, int64_t rows, int64_t ld, int64_t width, int elem) {
  return {p, p ? rows : 0, ld * elem, width * elem};
}
inline bool overlap(const Span& a, const Span& b) {
  return a.rows > 0 && b.rows > 0 && overlap(Rows{a.p, a.rows, a.ld, a.width}, Rows{b.p, b.rows, b.ld, b.width}, 1);
}
// The same rows at the same stride: element by element in place.
inline bool same_rows(const Span& a, const Span& b) {
  return a.p == b.p && a.rows == b.rows && a.width == b.width && (a.ld == b.ld || a.rows == 1);
}

// A row stride: a multiple of eight elements that holds a row.
inline bool ok_stride(const void* p, int64_t ld, int H) { return !p || (ld >= H && ld % 8 == 0 && ld <= kMostElements); }

// Checks that both directions share.
inline moe_status check_norm(int64_t M, int H, int dtype, int stream_dtype, int weight_dtype, int gate_mode,
                             const void* gate, int64_t ldgate, float residual_scale, float weight_offset, float eps) {
  if (!is_type(dtype) || (stream_dtype != dtype && stream_dtype != MOE_TYPE_FP32) ||
      (weight_dtype != dtype && weight_dtype != MOE_TYPE_FP32))
    return MOE_ERR_DTYPE;
  if (M < 0 || M >= (int64_t(1) << 31) || H < 8 || H % 8 || H > kNormMaxH || gate_mode < MOE_GATE_NONE ||
      gate_mode > MOE_GATE_FULL || !(residual_scale - residual_scale == 0.f) || !(weight_offset - weight_offset == 0.f) ||
      !(eps >= 0.f) || !(eps - eps == 0.f) || (gate_mode == MOE_GATE_FULL && !ok_stride(gate, ldgate, H)))
    return MOE_ERR_SHAPE;
  return MOE_OK;
}

// Bytes of a gate (or its gradient: `elem` bytes each of a channel or full one) as a buffer.
inline Span gate_span(int mode, const void* p, int64_t M, int H, int64_t ld, int elem) {
  return mode == MOE_GATE_CHANNEL ? span(p, 1, H, H, elem)
         : mode == MOE_GATE_TOKEN ? span(p, 1, M, M, 4)
         : mode == MOE_GATE_FULL  ? span(p, M, ld, H, elem)
                                  : Span{nullptr, 0, 0, 0};
}

// Threads of a row's team: `vecs` vectors, at most `each` a thread.
inline int team_threads(int vecs, int each) { return static_cast<int>(round_up(ceil_div(vecs, each), 32)); }

}  // namespace moe
