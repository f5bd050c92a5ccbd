// Feature rows: element types, conversions and wave reductions shared by the
// operators on voxel rows (norm.hip, product.hip).
#pragma once

#include <hip/hip_runtime.h>

#include "device.hpp"
#include "internal.hpp"

namespace tc {

using f16 = _Float16;
using bf16 = __bf16;

// Every conversion to a 16-bit type rounds to nearest even (one instruction on gfx950).
template <typename T>
__device__ __forceinline__ float to_f32(T v) {
  return (float)v;
}
template <typename T>
__device__ __forceinline__ T from_f32(float v) {
  return (T)v;
}

__device__ __forceinline__ float wave_sum_f32(float v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, kWave);
  return v;
}
__device__ __forceinline__ double wave_max_f64(double v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v = fmax(v, __shfl_xor(v, d, kWave));
  return v;
}

// Calls f with a value of the element type that `dtype` names.
template <typename F>
inline void with_dtype(int dtype, F&& f) {
  switch (dtype) {
    case TC_F32: f(float()); return;
    case TC_F16: f(f16()); return;
    case TC_BF16: f(bf16()); return;
    default: throw Error(TC_ERR_INVALID_ARG, "unknown dtype");
  }
}
inline size_t dtype_bytes(int dtype) { return dtype == TC_F32 ? 4 : 2; }

}  // namespace tc
