// Product of 4-bit microscaled rows with 4-bit microscaled weights.
//
//   out[m][n] = sum over blocks of 32 channels of 2^(xs + ws - 254) (sum_c x[m][c] * w[n][c]) + bias[n]
//
// The matrix instructions take the blocks' exponents with the values; sums are 32-bit floats.
#include "mx4.hpp"

namespace tc {

namespace {

// As load_16_tail, for a row of `k` 4-bit values: zeros from value k on.
__device__ __forceinline__ v4i load_32_tail(const uint8_t* row, int c, int k) {
  const int bytes = (k + 1) / 2;
  v4i v = load_16_tail(reinterpret_cast<const int8_t*>(row), c, bytes);
  const int last = bytes - 1 - c;  // the byte whose high half is beyond an odd k
  if (k % 2 && last >= 0 && last < 16) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i == last / 4) v[i] &= ~(0xf0 << (8 * (last % 4)));
  }
  return v;
}

// kRows * 16 rows x kCols * 16 channels per workgroup, the input channels split over its waves, operands straight
// from memory into registers. The waves' partial sums are added in LDS, in the order of the waves.
constexpr int kFewWaves = 8;
template <typename T, int kRows, int kCols>
__global__ void __launch_bounds__(kFewWaves * 64) k_product_mx4_few(ProductMx4Args a) {
  constexpr int kUnits = kRows * kCols;
  __shared__ v4f s_part[kFewWaves][kUnits][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tiles_n = (a.n + kCols * 16 - 1) / (kCols * 16);
  const i64 row0 = (i64)(blockIdx.x / tiles_n) * (kRows * 16);
  const int n0 = (blockIdx.x % tiles_n) * (kCols * 16);
  const int lr = lane & 15, lc = lane >> 4;
  const uint8_t *xrow[kRows], *wrow[kCols], *xscale[kRows], *wscale[kCols];
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const i64 row = min(row0 + j * 16 + lr, a.rows - 1);
    xrow[j] = a.x + row * a.x_stride;
    xscale[j] = a.x_scale + row * a.x_scale_stride;
  }
#pragma unroll
  for (int t = 0; t < kCols; ++t) {
    const i64 row = min(n0 + t * 16 + lr, a.n - 1);
    wrow[t] = a.w + row * a.w_stride;
    wscale[t] = a.w_scale + row * a.w_scale_stride;
  }
  v4f dot[kRows][kCols];
#pragma unroll
  for (int j = 0; j < kRows; ++j)
#pragma unroll
    for (int t = 0; t < kCols; ++t) dot[j][t] = v4f{0, 0, 0, 0};

  const int steps = (a.k + 127) / 128, each = (steps + kFewWaves - 1) / kFewWaves;
  const int s0 = wave * each, s1 = min(s0 + each, steps);
  for (int s = s0; s < s1; ++s) {
    v4i x[kRows], w[kCols];
    int xs[kRows], ws[kCols];
    const int block = s * 4 + lc;
    const bool have = block * 32 < a.k;
#pragma unroll
    for (int t = 0; t < kCols; ++t) {
      w[t] = load_32_tail(wrow[t], block * 16, a.k);
      ws[t] = have ? wscale[t][block] : 0;
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      x[j] = load_32_tail(xrow[j], block * 16, a.k);
      xs[j] = have ? xscale[j][block] : 0;
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j)
#pragma unroll
      for (int t = 0; t < kCols; ++t) dot[j][t] = product_mx4(w[t], x[j], dot[j][t], ws[t], xs[j]);
  }
#pragma unroll
  for (int j = 0; j < kRows; ++j)
#pragma unroll
    for (int t = 0; t < kCols; ++t) s_part[wave][j * kCols + t][lane] = dot[j][t];
  __syncthreads();
  for (int unit = wave; unit < kUnits; unit += kFewWaves) {
    const i64 row = row0 + (unit / kCols) * 16 + lr;
    const int n = n0 + (unit % kCols) * 16 + lc * 4;
    if (row >= a.rows) continue;
    v4f sum = s_part[0][unit][lane];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) sum += s_part[w][unit][lane];
    T* out = static_cast<T*>(a.out) + row * a.out_stride;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < a.n) out[n + i] = from_f32<T>(sum[i] + (a.bias ? a.bias[n + i] : 0.0f));
  }
}

template <typename T, int kRows, int kCols>
void launch_few(const ProductMx4Args& a, hipStream_t s) {
  const i64 blocks = ceil_div(a.rows, kRows * 16) * ceil_div(a.n, kCols * 16);
  launch("k_product_mx4_few", k_product_mx4_few<T, kRows, kCols>, blocks, kFewWaves * 64, s, a);
}

template <typename T>
void product(const ProductMx4Args& a, hipStream_t s) {
  launch_few<T, 2, 2>(a, s);
}

}  // namespace

void product_mx4(const ProductMx4Args& a, hipStream_t s) {
  if (a.rows == 0) return;
  with_dtype(a.out_dtype, [&](auto t) { product<decltype(t)>(a, s); });
}

}  // namespace tc
