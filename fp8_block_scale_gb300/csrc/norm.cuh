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

// Rows of an input or output: the next one `ld` bytes further on.
struct RowsOf {
  const void* p;
  int64_t ld;
  // This thread's part of row `row`, `offset` bytes into it; kNear: ld has 32 bits.
  template <bool kNear>
  __device__ __forceinline__ uint8_t* at(int64_t row, uint32_t offset) const {
    uint8_t* base = static_cast<uint8_t*>(const_cast<void*>(p)) + offset;
    if constexpr (kNear)
      return base + static_cast<uint64_t>(static_cast<uint32_t>(row)) * static_cast<uint32_t>(ld);
    else
      return base + row * ld;
  }
};


// ---- rows through shared memory
//
// Rows arrive by asynchronous 16-byte copies in pieces of 512 bytes, 16 for each lane of a warp.  A
// piece of 16-bit elements is each lane's own eight columns.  A warp's FP32 columns are two
// neighbouring pieces that its lanes fill (and empty) together in two runs of 512
// bytes: a lane's own 32 bytes in two 16-byte accesses would ask L2 for every sector twice (8192
// x 4096 with an FP32 stream, gradient: 136 us against 96).  The 16-byte units are placed so that a
// lane reads its two without bank conflicts.
constexpr int kPiece = 512;
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void put16(uint32_t at, float2 a, float2 b) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y) : "memory");
}
__device__ __forceinline__ uint4 shared16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
template <typename T> constexpr int kPieces = static_cast<int>(sizeof(T)) / 2;


// Where a lane finds its parts of a piece: its own, its place in a run, its two units of FP32.
struct Places {
  uint32_t mine16, run16, low16, high16;
};
__device__ __forceinline__ Places places(int lane) {
  const uint32_t low = 32u * lane + 16u * ((lane >> 2) & 1);
  return {16u * lane, 16u * (lane ^ ((lane >> 3) & 1)), low, low ^ 16u};
}
// Asks for this warp's columns of a row (c: the lane's first of eight), `pieces` of them.
__device__ __forceinline__ void to_pieces(const Places& in, uint32_t at, int piece, int pieces, const RowsOf& rows, uint32_t row,
                                          int c, int H) {
  if (pieces == 1) {
    if (c < H) copy16((at + in.mine16) + piece * kPiece, rows.at<true>(row, 2 * c));
  } else {
    const int c4 = c - 4 * static_cast<int>(threadIdx.x % 32);
    if (c4 < H) copy16((at + in.run16) + piece * kPiece, rows.at<true>(row, 4 * c4));
    if (c4 + 128 < H) copy16((at + in.run16) + (piece + 1) * kPiece, rows.at<true>(row, 4 * c4 + 512));
  }
}
template <typename T>
__device__ __forceinline__ Vec8<T> from_pieces(const Places& in, uint32_t at, int piece) {
  Vec8<T> r;
  if constexpr (sizeof(T) == 4) {
    r.v = shared16((at + in.low16) + piece * kPiece);
    r.w = shared16((at + in.high16) + piece * kPiece);
  } else {
    r.v = shared16((at + in.mine16) + piece * kPiece);
  }
  return r;
}
// FP32 outputs go the other way, through the place of an input that has been used: put by every
// lane, then (after a warp barrier) written to memory by runs.
__device__ __forceinline__ void put_pieces(const Places& in, uint32_t at, int piece, const float2 (&f)[4]) {
  put16((at + in.low16) + piece * kPiece, f[0], f[1]);
  put16((at + in.high16) + piece * kPiece, f[2], f[3]);
}
__device__ __forceinline__ void flush_pieces(const Places& in, uint32_t at, int piece, const RowsOf& rows, uint32_t row, int c, int H) {
  const int c4 = c - 4 * static_cast<int>(threadIdx.x % 32);
  if (c4 < H) *reinterpret_cast<uint4*>(rows.at<true>(row, 4 * c4)) = shared16((at + in.run16) + piece * kPiece);
  if (c4 + 128 < H) *reinterpret_cast<uint4*>(rows.at<true>(row, 4 * c4 + 512)) = shared16((at + in.run16) + (piece + 1) * kPiece);
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
