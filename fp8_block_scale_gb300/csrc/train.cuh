// Shared by the training-side kernels (include/moe_train.h): 16-bit element
// types and vectors of eight of them.
#pragma once

#include "../../include/moe_train.h"
#include "common.cuh"

namespace moe {

inline bool is_half_type(int dtype) { return dtype == MOE_TYPE_BF16 || dtype == MOE_TYPE_FP16; }
inline bool is_type(int dtype) { return is_half_type(dtype) || dtype == MOE_TYPE_FP32; }
inline int type_bytes(int dtype) { return dtype == MOE_TYPE_FP32 ? 4 : 2; }

// Whether pointers to 4-byte elements (tables, ids, weights, scalars) have that alignment; null has.
template <typename... P>
inline bool aligned4(P... p) {
  return ((reinterpret_cast<uintptr_t>(p) | ...) & 3u) == 0;
}

// More elements than any buffer has: products of sizes below it fit 64 bits.
constexpr int64_t kMostElements = int64_t(1) << 40;
// M * top_k route ids of 32 bits.
inline bool ok_routes(int64_t M, int top_k) {
  return M >= 0 && M < (int64_t(1) << 31) && top_k >= 1 && M * top_k < (int64_t(1) << 31);
}

// Whether the byte ranges [a, a + na) and [b, b + nb) share a byte.
inline bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const auto x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na > 0 && nb > 0 && x < y + static_cast<uint64_t>(nb) && y < x + static_cast<uint64_t>(na);
}
// Bytes from a row buffer's first element to the end of its last row.
inline int64_t extent_bytes(int64_t rows, int64_t ld, int64_t width, int elem) {
  return rows > 0 ? ((rows - 1) * ld + width) * elem : 0;
}

// A row buffer: `width` elements of each row, the next row `ld` further on.
struct Rows {
  const void* p;
  int64_t rows, ld, width;
};
// Whether two of them share a byte.  Buffers of one row stride may lie beside one
// another as columns of a wider one; of different strides they may not interleave.
inline bool overlap(const Rows& a, const Rows& b, int elem) {
  if (!overlap(a.p, extent_bytes(a.rows, a.ld, a.width, elem), b.p, extent_bytes(b.rows, b.ld, b.width, elem))) return false;
  const int64_t ld = a.rows > 1 ? a.ld : b.ld, period = ld * elem;
  if ((b.rows > 1 && b.ld != ld) || period <= 0) return true;
  int64_t at = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p)) % period;
  if (at < 0) at += period;
  return at < a.width * elem || at + b.width * elem > period;
}

template <typename T> struct Pack2;
template <> struct Pack2<__nv_bfloat16> {
  static __device__ __forceinline__ float2 load(uint32_t v) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
  }
  static __device__ __forceinline__ uint32_t store(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};
template <> struct Pack2<__half> {
  static __device__ __forceinline__ float2 load(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
  }
  static __device__ __forceinline__ uint32_t store(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};

// Eight 16-bit elements of a 16-byte vector as FP32, and back (one rounding).
template <typename T>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = Pack2<T>::load(w[i]);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(Pack2<T>::store(f[0], f[1]), Pack2<T>::store(f[2], f[3]), Pack2<T>::store(f[4], f[5]),
                    Pack2<T>::store(f[6], f[7]));
}

// 1 / (1 + exp(-g)) with the hardware exponential and divide (a few ulp; 0
// once exp(-g) passes 2^126).
__device__ __forceinline__ float sigmoid_f32(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }

}  // namespace moe
