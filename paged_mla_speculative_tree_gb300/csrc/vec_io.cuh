// 16-bit and 32-bit values to fp32 and back, one at a time and 16 bytes at once.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace mtv {

template <typename T> __device__ __forceinline__ float to_float(T x);
template <> __device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <> __device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
template <> __device__ __forceinline__ float to_float(float x) { return x; }
template <typename T> __device__ __forceinline__ T from_float(float x);
template <> __device__ __forceinline__ __nv_bfloat16 from_float(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_float(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ float from_float(float x) { return x; }

__device__ __forceinline__ float2 halves(uint32_t v, __nv_bfloat16) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
__device__ __forceinline__ float2 halves(uint32_t v, __half) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
__device__ __forceinline__ uint32_t join(float x, float y, __nv_bfloat16) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t join(float x, float y, __half) {
  const __half2 r = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// 16 bytes as fp32 values and back.
template <typename T> __device__ __forceinline__ void expand(const uint4& v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      x[i] = __uint_as_float(w[i]);
    } else {
      const float2 p = halves(w[i], T());
      x[2 * i] = p.x;
      x[2 * i + 1] = p.y;
    }
  }
}
template <typename T> __device__ __forceinline__ uint4 pack(const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(x[i]);
    else w[i] = join(x[2 * i], x[2 * i + 1], T());
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// N fp32 values as bf16: 8 or 16 bytes.
template <int N> __device__ __forceinline__ void store_bf16(__nv_bfloat16* to, const float* x) {
  uint32_t w[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) w[i] = join(x[2 * i], x[2 * i + 1], __nv_bfloat16());
  if constexpr (N == 8) *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
  else *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
}

}  // namespace mtv
