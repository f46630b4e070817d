// Pieces of 16 bytes of rows of 1-, 2- or 4-byte elements, at any alignment.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

namespace moe {

template <typename T>
__device__ __forceinline__ float to_float(T v) { return (float)v; }
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);

template <typename T>
struct alignas(16) Piece {
  T x[kVec<T>];
};

// A load that stays where it is written: batches of these are all issued before
// the first result is used, which the compiler otherwise undoes to save
// registers (34 instead of 58 in the aligned sum, and 211 instead of 180 us for
// 8192 tokens of 7168 bf16 values, 8 rows each).
__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ void load32(const void* p, uint4& a, uint4& b) {  // 32-byte aligned
  asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
               : "l"(p));
}
// 16 bytes at any address, from the two aligned windows they lie in.
__device__ __forceinline__ uint4 load16_any(const void* p) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  const unsigned m = (unsigned)(at & 15u);
  const uint4* w = reinterpret_cast<const uint4*>(at - m);
  const uint4 a = load16(w);
  const uint4 b = load16(w + (m != 0 ? 1 : 0));
  uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  const bool two = (m & 8u) != 0, one = (m & 4u) != 0;
#pragma unroll
  for (int i = 0; i < 6; ++i) x[i] = two ? x[i + 2] : x[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) x[i] = one ? x[i + 1] : x[i];
  const unsigned s = (m & 3u) * 8u;
  return make_uint4(__funnelshift_r(x[0], x[1], s), __funnelshift_r(x[1], x[2], s), __funnelshift_r(x[2], x[3], s),
                    __funnelshift_r(x[3], x[4], s));
}
template <typename T, bool ALIGNED>
__device__ __forceinline__ Piece<T> load_piece(const T* p) {
  Piece<T> r;
  *reinterpret_cast<uint4*>(&r) = ALIGNED ? load16(p) : load16_any(p);
  return r;
}

}  // namespace moe
