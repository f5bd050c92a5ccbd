// Product of 8-bit feature rows with 8-bit weights over a kernel map (a sparse
// convolution).
//
//   out[j][n] = ws[n] * sum_t xs[i] * (sum_c x[i][c] * w[t][n][c]) + bias[n],  i = map[j][t]
//
// The inner sum is exact (int32 accumulators of the matrix instructions). The
// rows a tap reads have scales of their own: each tap's integers are scaled and
// added to float sums, one conversion and one fused multiply-add a channel.
#include "int8.hpp"

namespace tc {

namespace {

constexpr int kConvWaves = 4;

// The row of an output tile's weights that row r of the matrix instruction t is, such
// that a lane's results of consecutive t are consecutive output channels (16 of them;
// with fewer than four instructions, 4 kCols).
template <int kCols>
__device__ __forceinline__ constexpr int weight_row(int t, int r) {
  if (kCols >= 4) return (t >> 2) * 64 + (r >> 2) * 16 + (t & 3) * 4 + (r & 3);
  return (r >> 2) * 4 * kCols + t * 4 + (r & 3);
}
// The LDS slot key of such a row: a function of r alone that differs between the
// rows one read takes together, two by two.
template <int kCols>
__device__ __forceinline__ constexpr int weight_key(int row) {
  if (kCols >= 4) return ((row >> 1) & 1) | ((row >> 3) & 2);
  if (kCols == 2) return ((row >> 1) & 1) | ((row >> 2) & 2);
  return (row >> 1) & 3;
}

// 16 bytes of a row of k >= 16 channels for the chunk at c: the chunk, or the
// row's last 16 bytes where it would pass the end. The weights' side of such a
// chunk holds zeros in front of c (all zeros from c >= k on), so that what x has there adds nothing.
__device__ __forceinline__ v4i load_16_end(const int8_t* row, int c, int k) {
  v4i v;
  __builtin_memcpy(&v, row + min(c, k - 16), 16);
  return v;
}
__device__ __forceinline__ v4i weight_16_end(const int8_t* row, int c, int k) {
  typedef unsigned long long u64x2 __attribute__((ext_vector_type(2)));
  u64x2 v = __builtin_bit_cast(u64x2, load_16_end(row, c, k));
  const int drop = min(c - min(c, k - 16), 16);  // bytes of the chunk before, or past the end
  if (drop > 0) {
    v[0] = drop >= 8 ? 0 : v[0] & (~0ull << (8 * drop));
    v[1] = drop >= 16 ? 0 : drop <= 8 ? v[1] : v[1] & (~0ull << (8 * (drop - 8)));
  }
  return __builtin_bit_cast(v4i, v);
}

// Scales and biases of CNT consecutive output channels, and the outputs of a row there.
template <int CNT>
struct Channels {
  int n;
  float scale[CNT], bias[CNT];
  bool wide;
  __device__ __forceinline__ Channels(const ProductArgs& a, int first) : n(first) {
#pragma unroll
    for (int i = 0; i < CNT; ++i) {
      const int c = min(n + i, a.n - 1);
      scale[i] = a.w_scale[c];
      bias[i] = a.bias ? a.bias[c] : 0.0f;
    }
    const int size = a.out_dtype == TC_F32 ? 4 : 2;
    wide = (((uintptr_t)a.out | a.out_stride * size | n * size) & 15) == 0;
  }
  __device__ __forceinline__ void store(const ProductArgs& a, i64 row, float v[CNT]) const {
#pragma unroll
    for (int i = 0; i < CNT; ++i) v[i] = v[i] * scale[i] + bias[i];
    if (a.out_dtype == TC_F32) store_run<float, CNT>(a, row, n, v, wide);
    else if (a.out_dtype == TC_F16) store_run<f16, CNT>(a, row, n, v, wide);
    else store_run<bf16, CNT>(a, row, n, v, wide);
  }
};

// One workgroup of four waves per 64 kRows output rows and 16 kCols output
// channels; a wave has kRows groups of 16 rows.
//
// Order of the rows: a tap is absent for most rows of a surface's map, and a group
// of 16 skips the taps that none of its rows has. The tile's rows are sorted by the
// Gray rank of their masks, so that rows of like masks share a group; group g goes to wave g % 4.
//
// A stage is one tap and 64 kSteps input channels (kWide: the rows have more than that, a tap
// takes several stages, and its integer sums are kept across them). Its weights are
// shared by the waves, two stages of them in LDS. Its rows are gathered by each wave into
// LDS of its own, in 16 rows x 64 bytes a load, and read from there as matrix operands
// before the next stage's are asked for. kDirect: rows and weights on 16-byte boundaries go
// straight into LDS, otherwise through registers, from any address.
template <int kRows, int kCols, int kSteps, bool kDirect, bool kWide>
__global__ void __launch_bounds__(kConvWaves * 64, kWide ? 1 : 2) k_conv_tile(ProductArgs a, int tiles_n) {
  constexpr int BM = kConvWaves * kRows * 16, BN = kCols * 16;
  constexpr int kRowLoads = kRows * kSteps;
  constexpr int kWeightLoads = (kCols * kSteps + kConvWaves - 1) / kConvWaves;  // a wave
  __shared__ __align__(16) int8_t s_x[kConvWaves * kRowLoads * 1024];
  __shared__ __align__(16) int8_t s_w[2 * BN * 64 * kSteps];
  __shared__ __align__(16) uint32_t s_key[BM];
  __shared__ int s_order[BM];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const i64 tile = xcd_block(blockIdx.x, gridDim.x);
  const i64 row0 = tile / tiles_n * BM;
  const int n0 = (int)(tile % tiles_n) * BN;
  const int taps = a.taps, k = a.k;

  // the order of the tile's rows; at most 32 taps, evenly spread, decide it
  if (tid < BM) {
    uint32_t mask = 0;
    if (row0 + tid < a.rows) {
      const int32_t* m = a.map + (row0 + tid) * taps;
      const int every = (taps + 31) / 32;
      for (int t = 0, b = 0; t < taps; t += every, ++b) mask |= (uint32_t)((uint32_t)m[t] < (uint32_t)a.n_src) << b;
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) mask ^= mask >> d;
    mask <<= taps < 32 ? 32 - taps : 0;
    s_key[tid] = (mask & ~255u) | tid;
  }
  __syncthreads();
  if (tid < BM) {
    const uint32_t mine = s_key[tid];
    int rank = 0;
    for (int i = 0; i < BM; i += 4) {
      const uint4 o = *reinterpret_cast<const uint4*>(s_key + i);
      rank += (o.x < mine) + (o.y < mine) + (o.z < mine) + (o.w < mine);
    }
    s_order[rank] = tid;
  }
  __syncthreads();

  // a lane's own row (of its group's 16): it holds the row's map entries and scale
  const int lr = lane & 15, lc = lane >> 4;
  const int my_group = lc % kRows;
  const i64 my_row = row0 + s_order[(my_group * kConvWaves + wave) * 16 + lr];
  const bool live = my_row < a.rows;
  const int32_t* my_map = a.map + (live ? my_row : 0) * taps;
  auto four_entries = [&](int first) {
    v4i v;
    if (taps >= 4) {
      __builtin_memcpy(&v, my_map + min(first, taps - 4), 16);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = my_map[min(i, taps - 1)];
    }
    return v;
  };
  v4i entries = four_entries(0), entries_ahead = four_entries(4);

  // a lane's part of the loads: row lane / 4 of 16, one chunk of its 64 bytes
  const int load_row = lane >> 2, load_chunk = ((lane & 3) ^ x_key(load_row)) * 16;
  int8_t* const my_x = s_x + wave * kRowLoads * 1024;
  const Buffer xb = buffer_at(a.x);
  v4i x_held[kDirect ? 1 : kRowLoads], w_held[kDirect ? 1 : kWeightLoads];

  int entry = -1;      // the stage's map entry of this lane's row, -1: none
  float scale = 0.0f;  // and its scale
  unsigned long long have = 0;
  auto take_entry = [&](int tap) {
    if (tap > 0 && (tap & 3) == 0) {
      entries = entries_ahead;
      entries_ahead = four_entries(tap + 4);
    }
    const int at = tap - (taps >= 4 ? min(tap & ~3, taps - 4) : 0);
    const int e = at == 0 ? entries[0] : at == 1 ? entries[1] : at == 2 ? entries[2] : entries[3];
    entry = live && (uint32_t)e < (uint32_t)a.n_src ? e : -1;
    have = __ballot(entry >= 0);
    scale = entry >= 0 ? a.x_scale[entry] : 0.0f;
  };
  auto group_has = [&](unsigned long long h, int j) { return (h >> (16 * j) & 0xffff) != 0; };
  auto ask = [&](int tap, int c0, int buffer) {
    // weights
    const int8_t* wt = a.w + ((i64)tap * a.n + n0) * k;
    const Buffer wb = buffer_at(wt);
#pragma unroll
    for (int i = 0; i < kWeightLoads; ++i) {
      const int part = i * kConvWaves + wave;
      if (part < kCols * kSteps) {
        const int r = part % kCols * 16 + load_row;
        const int c = c0 + part / kCols * 64 + ((lane & 3) ^ weight_key<kCols>(r)) * 16;
        const int wr = min(r, a.n - 1 - n0);
        if constexpr (kDirect)
          load_to_lds(wb, c < k ? (unsigned)wr * (unsigned)k + c : kOutside, 0,
                      s_w + (buffer * kCols * kSteps + part) * 1024);
        else
          w_held[i] = k >= 16 ? weight_16_end(wt + (i64)wr * k, c, k) : load_16_tail(wt + (i64)wr * k, c, k);
      }
    }
    // rows
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      if (!group_has(have, j)) continue;
      const int src = __shfl(entry, j * 16 + load_row, kWave);
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int c = c0 + s * 64 + load_chunk;
        if constexpr (kDirect) {
          load_to_lds(xb, ((src >= 0) & (c < k)) ? (unsigned)src * (unsigned)a.x_stride + c : kOutside, 0,
                      my_x + (j * kSteps + s) * 1024);
        } else if (src >= 0) {
          const int8_t* row = a.x + src * a.x_stride;
          x_held[j * kSteps + s] = k >= 16 ? load_16_end(row, c, k) : load_16_tail(row, c, k);
        }
      }
    }
  };
  auto put = [&](int buffer) {
    if constexpr (!kDirect) {
#pragma unroll
      for (int i = 0; i < kWeightLoads; ++i) {
        const int part = i * kConvWaves + wave;
        if (part < kCols * kSteps)
          *reinterpret_cast<v4i*>(s_w + (buffer * kCols * kSteps + part) * 1024 + lane * 16) = w_held[i];
      }
#pragma unroll
      for (int i = 0; i < kRowLoads; ++i) *reinterpret_cast<v4i*>(my_x + i * 1024 + lane * 16) = x_held[i];
    }
  };

  v4f acc[kRows][kCols];
  v4i dot[kWide ? kRows : 1][kWide ? kCols : 1];
#pragma unroll
  for (int j = 0; j < kRows; ++j)
#pragma unroll
    for (int t = 0; t < kCols; ++t) {
      acc[j][t] = v4f{0, 0, 0, 0};
      if constexpr (kWide) dot[j][t] = v4i{0, 0, 0, 0};
    }
  const int x_at = lr * 64 + ((lc ^ x_key(lr)) * 16);
  constexpr int kPart = kCols < 4 ? kCols : 4;  // instructions whose weights are held together

  if constexpr (!kDirect) {
#pragma unroll
    for (int i = 0; i < kRowLoads; ++i) x_held[i] = v4i{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kWeightLoads; ++i) w_held[i] = v4i{0, 0, 0, 0};
  }
  take_entry(0);
  ask(0, 0, 0);
  put(0);
  int tap = 0, c0 = 0;
  for (int stage = 0; tap < taps; ++stage) {
    wait_loads<0>();
    meet();
    // this stage's operands and scales
    const unsigned long long now = have;
    v4i x[kRows][kSteps];
    float xs[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      if (!kWide || c0 + 64 * kSteps >= k) xs[j] = __shfl(scale, j * 16 + lr, kWave);
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
        x[j][s] = *reinterpret_cast<const v4i*>(my_x + (j * kSteps + s) * 1024 + x_at);
    }
    wait_lds();  // the operands' LDS may be written again
    const bool last = !kWide || c0 + 64 * kSteps >= k;  // of the tap
    const int next_tap = last ? tap + 1 : tap, next_c0 = last ? 0 : c0 + 64 * kSteps;
    if (next_tap < taps) {
      if (last) take_entry(next_tap);
      ask(next_tap, next_c0, (stage + 1) & 1);
    }
    const int8_t* w_tile = s_w + (stage & 1) * BN * 64 * kSteps;
    if (now) {
#pragma unroll
      for (int part = 0; part < kCols / kPart; ++part) {
        v4i w[kPart][kSteps];
#pragma unroll
        for (int t = 0; t < kPart; ++t) {
          const int r = weight_row<kCols>(part * kPart + t, lr);
#pragma unroll
          for (int s = 0; s < kSteps; ++s)
            w[t][s] = *reinterpret_cast<const v4i*>(w_tile + (s * BN + r) * 64 + ((lc ^ weight_key<kCols>(r)) * 16));
        }
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
          if (!group_has(now, j)) continue;
          if constexpr (kWide) {
#pragma unroll
            for (int t = 0; t < kPart; ++t)
#pragma unroll
              for (int s = 0; s < kSteps; ++s)
                dot[j][part * kPart + t] = product_16(w[t][s], x[j][s], dot[j][part * kPart + t]);
            if (last) {
#pragma unroll
              for (int t = 0; t < kPart; ++t) {
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[j][part * kPart + t][i] += xs[j] * (float)dot[j][part * kPart + t][i];
                dot[j][part * kPart + t] = v4i{0, 0, 0, 0};
              }
            }
          } else {
            v4i d[kPart];
#pragma unroll
            for (int t = 0; t < kPart; ++t) d[t] = v4i{0, 0, 0, 0};
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
#pragma unroll
              for (int t = 0; t < kPart; ++t) d[t] = product_16(w[t][s], x[j][s], d[t]);
#pragma unroll
            for (int t = 0; t < kPart; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[j][part * kPart + t][i] += xs[j] * (float)d[t][i];
          }
        }
      }
    }
    if (next_tap < taps) put((stage + 1) & 1);
    tap = next_tap;
    c0 = next_c0;
  }

#pragma unroll
  for (int part = 0; part < kCols / kPart; ++part) {
    const Channels<kPart * 4> out(a, n0 + part * 64 + lc * 4 * kPart);
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const i64 row = row0 + s_order[(j * kConvWaves + wave) * 16 + lr];
      if (row >= a.rows) continue;
      float v[kPart * 4];
#pragma unroll
      for (int i = 0; i < kPart * 4; ++i) v[i] = acc[j][part * kPart + i / 4][i % 4];
      out.store(a, row, v);
    }
  }
}

// Few output rows: 16 of them by 16 kCols channels a workgroup, the taps split over
// its eight waves, operands straight from memory into registers, the waves'
// float sums added in LDS in the order of the waves.
constexpr int kFewWaves = 8;
template <int kCols>
__global__ void __launch_bounds__(kFewWaves * 64) k_conv_few(ProductArgs a, int tiles_n) {
  constexpr int kAhead = kCols > 2 ? 2 : 4;  // taps whose loads are in flight together
  __shared__ v4f s_part[kFewWaves][kCols][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, lc = (lane >> 4) * 16;
  const i64 row0 = (i64)(blockIdx.x / tiles_n) * 16;
  const int n0 = (int)(blockIdx.x % tiles_n) * kCols * 16;
  const bool live = row0 + lr < a.rows;
  const int32_t* my_map = a.map + (live ? row0 + lr : 0) * a.taps;
  v4f acc[kCols];
#pragma unroll
  for (int t = 0; t < kCols; ++t) acc[t] = v4f{0, 0, 0, 0};
  for (int tap0 = wave; tap0 < a.taps; tap0 += kFewWaves * kAhead) {
    int src[kAhead];
    float xs[kAhead];
    v4i dot[kAhead][kCols];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int tap = tap0 + u * kFewWaves;
      const int e = my_map[min(tap, a.taps - 1)];
      src[u] = live && tap < a.taps && (uint32_t)e < (uint32_t)a.n_src ? e : -1;
#pragma unroll
      for (int t = 0; t < kCols; ++t) dot[u][t] = v4i{0, 0, 0, 0};
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) xs[u] = src[u] >= 0 ? a.x_scale[src[u]] : 0.0f;
    for (int c = 0; c < a.k; c += 64) {
      const bool full = c + 64 <= a.k;
      v4i x[kAhead], w[kAhead][kCols];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        x[u] = v4i{0, 0, 0, 0};
        if (src[u] >= 0) {
          const int8_t* row = a.x + src[u] * a.x_stride;
          if (full) __builtin_memcpy(&x[u], row + c + lc, 16);
          else x[u] = load_16_tail(row, c + lc, a.k);
        }
        const int tap = min(tap0 + u * kFewWaves, a.taps - 1);
#pragma unroll
        for (int t = 0; t < kCols; ++t) {
          const int8_t* row = a.w + ((i64)tap * a.n + min(n0 + t * 16 + lr, a.n - 1)) * a.k;
          if (full) __builtin_memcpy(&w[u][t], row + c + lc, 16);
          else w[u][t] = load_16_tail(row, c + lc, a.k);
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
#pragma unroll
        for (int t = 0; t < kCols; ++t) dot[u][t] = product_16(w[u][t], x[u], dot[u][t]);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int t = 0; t < kCols; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][i] += xs[u] * (float)dot[u][t][i];
  }
#pragma unroll
  for (int t = 0; t < kCols; ++t) s_part[wave][t][lane] = acc[t];
  __syncthreads();
  if (wave >= kCols || !live) return;
  v4f sum = s_part[0][wave][lane];
#pragma unroll
  for (int w = 1; w < kFewWaves; ++w) sum += s_part[w][wave][lane];
  float v[4] = {sum[0], sum[1], sum[2], sum[3]};
  Channels<4>(a, n0 + wave * 16 + (lane >> 4) * 4).store(a, row0 + lr, v);
}

template <int kRows, int kCols, int kSteps, bool kDirect, bool kWide>
void launch_conv(const ProductArgs& a, hipStream_t s) {
  const int tn = (int)ceil_div(a.n, kCols * 16);
  launch("k_conv_tile", k_conv_tile<kRows, kCols, kSteps, kDirect, kWide>,
         ceil_div(a.rows, kConvWaves * kRows * 16) * tn, kConvWaves * 64, s, a, tn);
}

template <int kCols>
void launch_conv_few(const ProductArgs& a, hipStream_t s) {
  const int tn = (int)ceil_div(a.n, kCols * 16);
  launch("k_conv_few", k_conv_few<kCols>, ceil_div(a.rows, 16) * tn, kFewWaves * 64, s, a, tn);
}

// The registers of a wave hold 64 rows x 128 channels of sums, except where the rows come
// through registers as well, or integer sums are kept beside the float ones.
template <int kRows, int kCols>
void conv_tile(const ProductArgs& a, bool direct, hipStream_t s) {
  if (a.k <= 64)
    return direct ? launch_conv<kRows, kCols, 1, true, false>(a, s) : launch_conv<kRows, kCols, 1, false, false>(a, s);
  if (a.k > 128) {
    constexpr int kC = std::min(kCols, 4);
    return direct ? launch_conv<kRows, kC, 2, true, true>(a, s) : launch_conv<kRows, kC, 2, false, true>(a, s);
  }
  if (direct) return launch_conv<kRows, kCols, 2, true, false>(a, s);
  launch_conv<kCols == 8 ? std::min(kRows, 2) : kRows, kCols, 2, false, false>(a, s);
}

template <int kRows>
void conv_rows(const ProductArgs& a, bool direct, hipStream_t s) {
  if (a.n <= 16) return conv_tile<kRows, 1>(a, direct, s);
  if (a.n <= 32) return conv_tile<kRows, 2>(a, direct, s);
  if (a.n <= 64) return conv_tile<kRows, 4>(a, direct, s);
  conv_tile<kRows, 8>(a, direct, s);
}

}  // namespace

void conv_i8(const ProductArgs& a, hipStream_t s) {
  const i64 cus = device_cu_count();
  auto tiles = [&](int rows, int cols) { return ceil_div(a.rows, rows) * ceil_div(a.n, cols); };
  // the offsets of a gather straight into LDS are 31 bits
  const bool direct = (((uintptr_t)a.x | (uintptr_t)a.x_stride | (uintptr_t)a.w | (uintptr_t)a.k) & 15) == 0 &&
                      a.n_src * a.x_stride + a.k < (1ll << 31);
  if (tiles(256, 128) >= cus) return conv_rows<4>(a, direct, s);
  if (tiles(64, 128) >= cus / 2) return conv_rows<1>(a, direct, s);
  if (tiles(16, 64) >= cus) return launch_conv_few<4>(a, s);
  if (tiles(16, 32) >= cus) return launch_conv_few<2>(a, s);
  launch_conv_few<1>(a, s);
}

}  // namespace tc
