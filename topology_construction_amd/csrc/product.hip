// Product of 8-bit feature rows with 8-bit weights, and the same product over
// a kernel map (a sparse convolution).
//
//   out[j][n] = ws[n] * sum_t xs[i] * (sum_c x[i][c] * w[t][n][c]) + bias[n],  i = map[j][t]
//
// The inner sum is exact (int32 accumulators of the matrix instructions); the
// sum over taps, whose rows have scales of their own, is a float sum in the
// order of the taps.
#include "rows.hpp"

namespace tc {

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kTile = 64;       // output rows and channels of a workgroup
constexpr int kStep = 64;       // input channels of one matrix instruction
constexpr int kLdsRow = kStep + 16;  // bytes between rows in LDS

// 16 bytes at row + c (c a multiple of 16), zeros from k on.
__device__ __forceinline__ v4i load_16(const int8_t* row, int c, int k) {
  union {
    int8_t b[16];
    v4i v;
  } u;
  u.v = v4i{0, 0, 0, 0};
  if (row) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (c + i < k) u.b[i] = row[c + i];
  }
  return u.v;
}

// One workgroup of four waves per 64 x 64 output tile. The weights are the
// matrix instruction's row operand and the feature rows its column operand, so
// a lane holds four consecutive output channels of one output row.
template <typename T>
__global__ void __launch_bounds__(256) k_product_any(ProductArgs a) {
  __shared__ __align__(16) int8_t s_x[kTile * kLdsRow];
  __shared__ __align__(16) int8_t s_w[kTile * kLdsRow];
  __shared__ float s_scale[kTile];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int tiles_n = (a.n + kTile - 1) / kTile;
  const i64 row0 = (i64)(blockIdx.x / tiles_n) * kTile;
  const int n0 = (blockIdx.x % tiles_n) * kTile;
  const int lr = tid >> 2, lc = (tid & 3) * 16;  // this thread's row and bytes of both LDS tiles

  v4f acc[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) acc[t] = v4f{0, 0, 0, 0};
  for (int tap = 0; tap < a.taps; ++tap) {
    i64 src = row0 + lr;
    bool have = src < a.rows;
    if (a.map) src = have ? (i64)a.map[src * a.taps + tap] : -1;
    have = have && src >= 0 && src < a.n_src;
    const int8_t* xrow = have ? a.x + src * a.x_stride : nullptr;
    const int8_t* wrow = n0 + lr < a.n ? a.w + ((i64)tap * a.n + n0 + lr) * a.w_stride : nullptr;
    if (lc == 0) s_scale[lr] = have ? a.x_scale[src] : 0.0f;
    v4i dot[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) dot[t] = v4i{0, 0, 0, 0};
    for (int c = 0; c < a.k; c += kStep) {
      const v4i xv = load_16(xrow, c + lc, a.k), wv = load_16(wrow, c + lc, a.k);
      __syncthreads();
      *reinterpret_cast<v4i*>(s_x + lr * kLdsRow + lc) = xv;
      *reinterpret_cast<v4i*>(s_w + lr * kLdsRow + lc) = wv;
      __syncthreads();
      const v4i xo = *reinterpret_cast<const v4i*>(s_x + (wave * 16 + (lane & 15)) * kLdsRow + (lane >> 4) * 16);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const v4i wo = *reinterpret_cast<const v4i*>(s_w + (t * 16 + (lane & 15)) * kLdsRow + (lane >> 4) * 16);
        dot[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wo, xo, dot[t], 0, 0, 0);
      }
    }
    if (a.k == 0) __syncthreads();
    const float xs = s_scale[wave * 16 + (lane & 15)];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[t][i] += xs * (float)dot[t][i];
    __syncthreads();  // the next tap rewrites the scales
  }
  const i64 row = row0 + wave * 16 + (lane & 15);
  if (row >= a.rows) return;
  T* out = static_cast<T*>(a.out) + row * a.out_stride;
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = n0 + t * 16 + (lane >> 4) * 4 + i;
      if (n < a.n) out[n] = from_f32<T>(acc[t][i] * a.w_scale[n] + (a.bias ? a.bias[n] : 0.0f));
    }
}

}  // namespace

void product_i8(const ProductArgs& a, hipStream_t s) {
  if (a.rows == 0 || a.n == 0) return;
  with_dtype(a.out_dtype, [&](auto t) {
    using T = decltype(t);
    launch("k_product_any", k_product_any<T>, ceil_div(a.rows, kTile) * ceil_div(a.n, kTile), 256, s, a);
  });
}

}  // namespace tc
