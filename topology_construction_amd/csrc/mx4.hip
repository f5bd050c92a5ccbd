// Rows in microscaled 4 bits: blocks of 32 channels of e2m1 values (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
// negatives) under one power of two.
//
//   E = max(floor(log2 max|x|) - 2, -127), q = round(x 2^-E) to e2m1, scale = E + 127
//
// The largest value lies in [4, 8) 2^E, so that what is above 6 is held as 6. Divisions by a power of two are
// exact and the conversion rounds once, to nearest even: the values are the same in any implementation.
// Memory bounds both directions.
#include "mx4.hpp"

namespace tc {

namespace {

constexpr int kThreads = 256;

// Items of kChannels channels, row after row, every lane one of those that follow each other.
template <int kChannels>
struct Item {
  i64 row;
  int at, n;  // first channel, number of channels (0: none)
  __device__ __forceinline__ Item(i64 rows, int channels, int per_row) {
    const i64 first = (i64)blockIdx.x * kThreads, row0 = first / per_row;
    const int a = (int)(first - row0 * per_row) + (int)threadIdx.x, r = a / per_row;
    row = row0 + r;
    at = (a - r * per_row) * kChannels;
    n = row < rows ? max(0, min(kChannels, channels - at)) : 0;
  }
};

// Four lanes a block, eight channels a lane. 124800 x 256 bf16 14.6 us (5.5 TB/s; two or four items a lane: 15 to
// 17), f32 22.7, one row of 1024 1.5.
constexpr int kQuantiseChannels = 8;
template <typename T>
__global__ void __launch_bounds__(kThreads) k_quantise_mx4(QuantiseArgs a, int per_row) {
  const Item<kQuantiseChannels> item(a.rows, a.channels, per_row);
  const T* x = static_cast<const T*>(a.x) + item.row * a.x_stride + item.at;
  T t[8];
  if (item.n == 8) {
    __builtin_memcpy(t, x, sizeof(t));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = e < item.n ? x[e] : T(0);
  }
  float v[8];
  uint32_t top = 0;  // as integers: infinities and NaN are above all numbers
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    v[e] = to_f32(t[e]);
    top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
  }
  top = lanes_reduce<4>(top, [](uint32_t a, uint32_t b) { return max(a, b); });
  const uint32_t field = top >> 23, scale = field == 255 ? 255 : field > 2 ? field - 2 : 0;
  const uint32_t q = scale == 255 ? 0 : pack_mx4(v, __uint_as_float(scale << 23));
  if (item.n == 0) return;
  if (item.at % 32 == 0) a.scale[item.row * ((a.channels + 31) / 32) + item.at / 32] = (uint8_t)scale;
  uint8_t* to = a.q + item.row * ((a.channels + 1) / 2) + item.at / 2;
  if (item.n == 8) {
    __builtin_memcpy(to, &q, 4);
  } else {
    for (int b = 0; b < (item.n + 1) / 2; ++b) to[b] = (uint8_t)(q >> (8 * b));
  }
}

// 16 bytes of values a lane, so that a wave stores whole lines; rows on 16-byte boundaries (`wide`) past the caches
// (124800 x 256 bf16 12.6 for 20.5 us, f32 20.4 for 33).
template <typename T>
__global__ void __launch_bounds__(kThreads) k_dequantise_mx4(DequantiseArgs a, int per_row, bool wide) {
  constexpr int N = 16 / sizeof(T);
  const Item<N> item(a.rows, a.channels, per_row);
  if (item.n == 0) return;
  const uint8_t* from = a.q + item.row * a.q_stride + item.at / 2;
  uint32_t q = 0;
  if (item.n == N) {
    __builtin_memcpy(&q, from, N / 2);
  } else {
    for (int b = 0; b < (item.n + 1) / 2; ++b) q |= (uint32_t)from[b] << (8 * b);
  }
  const uint32_t scale = a.scale[item.row * a.scale_stride + item.at / 32];
  float v[8];
  unpack_mx4(q, __uint_as_float(scale << 23), v);
  T t[N];
#pragma unroll
  for (int e = 0; e < N; ++e) t[e] = from_f32<T>(scale == 255 ? NAN : v[e]);
  T* out = static_cast<T*>(a.out) + item.row * a.channels + item.at;
  if (item.n == N && wide) {
    __builtin_nontemporal_store(__builtin_bit_cast(v4i, t), reinterpret_cast<v4i*>(out));
  } else if (item.n == N) {
    __builtin_memcpy(out, t, sizeof(t));
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (e < item.n) out[e] = t[e];
  }
}

// Items of whole blocks of 32.
int items_of(int channels, int each) { return (int)ceil_div(channels, 32) * (32 / each); }

}  // namespace

void quantise_mx4(const QuantiseArgs& a, hipStream_t s) {
  const int per_row = items_of(a.channels, kQuantiseChannels);
  with_dtype(a.dtype, [&](auto t) {
    launch("k_quantise_mx4", k_quantise_mx4<decltype(t)>, ceil_div(a.rows * per_row, kThreads), kThreads, s, a, per_row);
  });
}

void dequantise_mx4(const DequantiseArgs& a, hipStream_t s) {
  with_dtype(a.out_dtype, [&](auto t) {
    using T = decltype(t);
    const int per_row = items_of(a.channels, 16 / sizeof(T));
    launch("k_dequantise_mx4", k_dequantise_mx4<T>, ceil_div(a.rows * per_row, kThreads), kThreads, s, a, per_row,
           aligned_16(a.out, a.channels * (i64)sizeof(T)));
  });
}

}  // namespace tc
