// 4-bit microscaled rows as the conversion and matrix instructions take them (mx4.hip, product_mx4.hip): the even
// channel of a byte in its low half, a block's exponent in the place of a float's.
#pragma once

#include "int8.hpp"

namespace tc {

typedef float v16f __attribute__((ext_vector_type(16)));

// Eight values divided by `scale` (its exponent alone counts), in 4 bits each, rounded to nearest even, at most 6.
__device__ __forceinline__ uint32_t pack_mx4(const float (&v)[8], float scale) {
  uint32_t q = 0;
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], scale, 0);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], scale, 1);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], scale, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], scale, 3);
}

// The eight values that `q` stands for under `scale`.
__device__ __forceinline__ void unpack_mx4(uint32_t q, float scale, float (&v)[8]) {
  typedef float v2f __attribute__((ext_vector_type(2)));
  auto put = [&](v2f p, int i) {
    v[i] = p[0];
    v[i + 1] = p[1];
  };
  put(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, scale, 0), 0);
  put(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, scale, 1), 2);
  put(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, scale, 2), 4);
  put(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, scale, 3), 6);
}

// One step of products: 16 rows of w by 16 rows of x over 128 input channels. A lane has 32 channels (one
// block, number lane / 16) of row lane % 16 of each, their exponents in byte kByte of ws and xs, and
// holds four rows of w (4 (lane / 16) on) of x's row lane % 16.
template <int kByte>
__device__ __forceinline__ v4f product_mx4(v4i w, v4i x, v4f sum, int ws, int xs) {
  typedef int v8i __attribute__((ext_vector_type(8)));
  const v8i a = __builtin_shufflevector(w, w, 0, 1, 2, 3, -1, -1, -1, -1);
  const v8i b = __builtin_shufflevector(x, x, 0, 1, 2, 3, -1, -1, -1, -1);
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, sum, 4, 4, kByte, ws, kByte, xs);
}

// The same for 32 rows of each over 64 input channels, which takes the matrix units half the time for the
// same products (9262 TFLOP/s for 5112 with one wave a SIMD, 6631 with two). A lane has block number lane / 32 of row
// lane % 32 of each, and holds 16 rows of w (r % 4 + 8 (r / 4) + 4 (lane / 32)) of x's row lane % 32.
template <int kByte>
__device__ __forceinline__ v16f product_mx4(v4i w, v4i x, v16f sum, int ws, int xs) {
  typedef int v8i __attribute__((ext_vector_type(8)));
  const v8i a = __builtin_shufflevector(w, w, 0, 1, 2, 3, -1, -1, -1, -1);
  const v8i b = __builtin_shufflevector(x, x, 0, 1, 2, 3, -1, -1, -1, -1);
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, sum, 4, 4, kByte, ws, kByte, xs);
}

}  // namespace tc
