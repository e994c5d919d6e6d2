// ep_pack.cuh -- what the epilogues of the tensor-core products share: the fast
// activation, 16-bit pairs and streaming stores.
#pragma once

#include "ep_experts.cuh"

namespace ep {

// The activation for results that are rounded to 16 bits: __expf and
// __fdividef are off by a few parts in 2^22 (times 1 + |gate|), far below the
// rounding.  Where exp(-gate) overflows the quotient is 0.
__device__ __forceinline__ float fast_sigmoid(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t u);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t u) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t u) {
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

// Outputs are stored as streaming data, first to leave L2, which the operands
// need: dgrad of 16,384 rows x 4096 -> 7168 took 634 us without, 558 us with.
template <typename T>
__device__ __forceinline__ void store2(T* p, float x, float y) { __stcs(reinterpret_cast<uint32_t*>(p), pack2<T>(x, y)); }
template <typename T>
__device__ __forceinline__ void store4(T* p, const float4& v) {
  __stcs(reinterpret_cast<uint2*>(p), make_uint2(pack2<T>(v.x, v.y), pack2<T>(v.z, v.w)));
}
template <typename T>
__device__ __forceinline__ float4 unpack4(uint2 u) {
  const float2 a = unpack2<T>(u.x), b = unpack2<T>(u.y);
  return make_float4(a.x, a.y, b.x, b.y);
}
template <typename T>
__device__ __forceinline__ float4 load4(const T* p) { return unpack4<T>(*reinterpret_cast<const uint2*>(p)); }

}  // namespace ep
