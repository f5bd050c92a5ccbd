// Feature rows: element types, conversions and wave reductions shared by the
// operators on voxel rows (norm.hip, int8.hpp).
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

// v of another lane: its partner in groups of 2, 4, 8, 16 (mirrored within 8 and 16) by
// DPP, without LDS.
template <int kCtrl>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), kCtrl, 0xf, 0xf, true));
}
template <int kCtrl>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, kCtrl, 0xf, 0xf, true);
}
template <int kCtrl>
__device__ __forceinline__ double dpp(double v) {
  return __hiloint2double(__builtin_amdgcn_mov_dpp(__double2hiint(v), kCtrl, 0xf, 0xf, true),
                          __builtin_amdgcn_mov_dpp(__double2loint(v), kCtrl, 0xf, 0xf, true));
}

// f over each group of L lanes (a power of two), the same result in every lane of the group.
template <int L, typename V, typename F>
__device__ __forceinline__ V lanes_reduce(V v, F&& f) {
  if constexpr (L >= 2) v = f(v, dpp<0xb1>(v));    // lane ^ 1
  if constexpr (L >= 4) v = f(v, dpp<0x4e>(v));    // lane ^ 2
  if constexpr (L >= 8) v = f(v, dpp<0x141>(v));   // mirrored within 8
  if constexpr (L >= 16) v = f(v, dpp<0x140>(v));  // mirrored within 16
  if constexpr (L >= 32) v = f(v, __shfl_xor(v, 16, kWave));
  if constexpr (L >= 64) v = f(v, __shfl_xor(v, 32, kWave));
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

}  // namespace tc
