// Element types of the generation operators (FKL_TYPE_* of fkl_generate.h) on the device.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "../../include/fkl_generate.h"

namespace fkl {

inline size_t type_bytes(int32_t type) { return type == FKL_TYPE_F32 ? 4 : 2; }
inline bool type_ok(int32_t type) { return type == FKL_TYPE_F32 || type == FKL_TYPE_BF16 || type == FKL_TYPE_F16; }

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }

template <class T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }

// Two values rounded to a 16-bit T and packed, `lo` in the low half.
template <class T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 16 bytes of T as floats.
template <class T>
__device__ __forceinline__ void unpack16(const uint4& raw, float (&v)[16 / sizeof(T)]) {
  const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
  for (int i = 0; i < static_cast<int>(16 / sizeof(T)); ++i) v[i] = to_float(e[i]);
}

// Calls f with a value of the C++ type that `type` names.
template <class F>
auto with_type(int32_t type, F&& f) {
  if (type == FKL_TYPE_F32) return f(float{});
  if (type == FKL_TYPE_BF16) return f(__nv_bfloat16{});
  return f(__half{});
}

}  // namespace fkl
