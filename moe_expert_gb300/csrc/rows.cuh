// Typed loads and stores of four or eight consecutive row elements, shared by
// the kernels that take FP32, BF16 or FP16 rows.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace moex {

template <int TYPE>
struct RowElem;
template <>
struct RowElem<MOEX_F32> {
  using T = float;
  static __device__ __forceinline__ float get(float v) { return v; }
};
template <>
struct RowElem<MOEX_BF16> {
  using T = __nv_bfloat16;
  static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
  }
};
template <>
struct RowElem<MOEX_F16> {
  using T = __half;
  static __device__ __forceinline__ float get(__half v) { return __half2float(v); }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t u) {
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
  }
};

// Four consecutive elements at element offset `i` (a multiple of 4).
template <int TYPE>
__device__ __forceinline__ float4 load4(const void* p, int64_t i) {
  if constexpr (TYPE == MOEX_F32) {
    return *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
    const float2 a = RowElem<TYPE>::unpack(u.x), b = RowElem<TYPE>::unpack(u.y);
    return make_float4(a.x, a.y, b.x, b.y);
  }
}

template <int TYPE>
__device__ __forceinline__ void store4(void* p, int64_t i, float4 v) {
  if constexpr (TYPE == MOEX_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = v;
  } else {
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) =
        make_uint2(RowElem<TYPE>::pack(v.x, v.y), RowElem<TYPE>::pack(v.z, v.w));
  }
}

// Eight consecutive elements at element offset `i` (a multiple of 8).
template <int TYPE>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&f)[8]) {
  if constexpr (TYPE == MOEX_F32) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 a = q[0], b = q[1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 a = RowElem<TYPE>::unpack(w[j]);
      f[2 * j] = a.x, f[2 * j + 1] = a.y;
    }
  }
}

template <int TYPE>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&f)[8]) {
  if constexpr (TYPE == MOEX_F32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(f[0], f[1], f[2], f[3]);
    q[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
        make_uint4(RowElem<TYPE>::pack(f[0], f[1]), RowElem<TYPE>::pack(f[2], f[3]), RowElem<TYPE>::pack(f[4], f[5]),
                   RowElem<TYPE>::pack(f[6], f[7]));
  }
}

}  // namespace moex
