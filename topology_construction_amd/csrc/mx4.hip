// Rows in microscaled 4 bits: blocks of 32 channels of e2m1 values (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
// negatives) under one power of two.
//
//   E = max(floor(log2 max|x|) - 2, -127), q = round(x 2^-E) to e2m1, scale = E + 127
//
// The largest value lies in [4, 8) 2^E, so that what is above 6 is held as 6. Divisions by a power of two are
// exact and the conversion rounds once, to nearest even: the values are the same in any implementation.
// Memory bounds both directions: four lanes a block, eight channels a lane.
#include "mx4.hpp"

namespace tc {

namespace {

constexpr int kThreads = 256;

// Items of eight channels, four to a block of 32, row after row: the place of this lane's item in a row. A workgroup
// takes kThreads items that follow each other.
struct Item {
  i64 row;
  int at;  // item of the row
  bool any;
};
__device__ __forceinline__ Item item_of(i64 rows, int per_row) {
  const i64 first = (i64)blockIdx.x * kThreads, row0 = first / per_row;
  const int at = (int)(first - row0 * per_row) + (int)threadIdx.x;
  const int r = at / per_row;
  return {row0 + r, at - r * per_row, row0 + r < rows};
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_quantise_mx4(QuantiseArgs a, int per_row) {
  const Item item = item_of(a.rows, per_row);
  const int c = item.at * 8, n = item.any ? min(8, a.channels - c) : 0;
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = 0.0f;
  const T* x = static_cast<const T*>(a.x) + item.row * a.x_stride + c;
  if (n == 8) {
    T t[8];
    __builtin_memcpy(t, x, sizeof(t));
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = to_f32(t[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) v[e] = to_f32(x[e]);
  }
  // as integers: infinities and NaN are above all numbers
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
  top = lanes_reduce<4>(top, [](uint32_t a, uint32_t b) { return max(a, b); });
  const uint32_t field = top >> 23, scale = field == 255 ? 255 : field > 2 ? field - 2 : 0;
  uint32_t q = 0;
  if (scale != 255) q = pack_mx4(v, __uint_as_float(scale << 23));
  if (!item.any) return;
  if (item.at % 4 == 0) a.scale[item.row * (per_row / 4) + item.at / 4] = (uint8_t)scale;
  const int row_bytes = (a.channels + 1) / 2;
  uint8_t* to = a.q + item.row * row_bytes + item.at * 4;
  if (n == 8) {
    __builtin_memcpy(to, &q, 4);
  } else {
    for (int i = 0; i < (n + 1) / 2; ++i) to[i] = (uint8_t)(q >> (8 * i));
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_dequantise_mx4(DequantiseArgs a, int per_row) {
  const Item item = item_of(a.rows, per_row);
  const int c = item.at * 8, n = item.any ? min(8, a.channels - c) : 0;
  if (n <= 0) return;
  const uint8_t* from = a.q + item.row * a.q_stride + item.at * 4;
  uint32_t q = 0;
  if (n == 8) {
    __builtin_memcpy(&q, from, 4);
  } else {
    for (int i = 0; i < (n + 1) / 2; ++i) q |= (uint32_t)from[i] << (8 * i);
  }
  const uint32_t scale = a.scale[item.row * a.scale_stride + item.at / 4];
  float v[8];
  unpack_mx4(q, __uint_as_float(scale << 23), v);
  T t[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) t[e] = from_f32<T>(scale == 255 ? NAN : v[e]);
  T* out = static_cast<T*>(a.out) + item.row * a.channels + c;
  if (n == 8) {
    __builtin_memcpy(out, t, sizeof(t));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) out[e] = t[e];
  }
}

int items_of(int channels) { return (int)ceil_div(channels, 32) * 4; }

}  // namespace

void quantise_mx4(const QuantiseArgs& a, hipStream_t s) {
  const int per_row = items_of(a.channels);
  with_dtype(a.dtype, [&](auto t) {
    launch("k_quantise_mx4", k_quantise_mx4<decltype(t)>, ceil_div(a.rows * per_row, kThreads), kThreads, s, a, per_row);
  });
}

void dequantise_mx4(const DequantiseArgs& a, hipStream_t s) {
  const int per_row = items_of(a.channels);
  with_dtype(a.out_dtype, [&](auto t) {
    launch("k_dequantise_mx4", k_dequantise_mx4<decltype(t)>, ceil_div(a.rows * per_row, kThreads), kThreads, s, a,
           per_row);
  });
}

}  // namespace tc
