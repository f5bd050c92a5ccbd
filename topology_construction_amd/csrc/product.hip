// Product of 8-bit feature rows with 8-bit weights.
//
//   out[m][n] = xs[m] * ws[n] * (sum_c x[m][c] * w[n][c]) + bias[n]
//
// The sum is exact (int32 accumulators of the matrix instructions).
#include "int8.hpp"

namespace tc {

namespace {

// ------------------------------------------------------------------ plain product, many tiles

// Row r of the weights' matrix instruction t of a wave's 64 channels, such that a lane's
// results of two instructions are 8 consecutive channels and the four lanes of an output
// row store 64 bytes side by side; and the LDS slot key of such a row.
__device__ __forceinline__ constexpr int w_row(int t, int r) {
  return (t >> 1) * 32 + (r >> 2) * 8 + (t & 1) * 4 + (r & 3);
}
__device__ __forceinline__ int w_key(int row) { return ((row >> 1) & 1) | ((row >> 2) & 2); }

// BM x BN outputs per workgroup, (BM / WM) * (BN / 64) waves of WM x 64 each, in
// steps of 64 input channels. kDirect: rows and chunks on 16-byte boundaries go
// straight into LDS, kBufs - 1 steps ahead of the products, or (kPer = 2, four buffers)
// two steps between barriers, with the loads of the next two under way. Otherwise, from any
// address, through registers: loaded two steps ahead, written one step ahead.
//
// 16384 x 4096 -> 4096: 217 to 233 us from one card to another, 2360 to 2530 TOP/s (a library's 8-bit
// product of this size: 1990): the matrix units are busy 54% of the cycles at the 2.2 GHz the card holds
// under this load. Where this takes 233: one barrier a step 248 us; loads spread among the products instead
// of after the barrier 243; the second step's reads among the first's products no change.
// 124800 x 256 -> 768: 57 us, 224 MB at 3.9 TB/s: bound by the stores (33 us without them).
template <typename T, int BM, int BN, int WM, int kBufs, int kPer, bool kDirect>
__global__ void __launch_bounds__((BM / WM) * (BN / 64) * 64)
    k_product_tile(ProductArgs a, i64 tiles_m, int tiles_n) {
  static_assert(kDirect || kBufs == 2, "one buffer is read, one written");
  constexpr int kWaves = (BM / WM) * (BN / 64);
  constexpr int kLoads = (BM + BN) / 16 / kWaves;  // per wave and step
  constexpr int kBuf = (BM + BN) * 64;
  // One array: with several the compiler has every read of a tile wait for all loads
  // under way into any of them. Behind the tiles are the scales, read before the loop for its end.
  __shared__ __align__(16) int8_t s_tiles[kBufs * kBuf + (2 * BN + BM) * 4];
  float* const s_scale = reinterpret_cast<float*>(s_tiles + kBufs * kBuf);
  float* const s_bias = s_scale + BN;
  float* const s_rows = s_bias + BN;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  i64 tm;
  int tn;
  tile_place(xcd_block(blockIdx.x, tiles_m * tiles_n), tiles_m, tiles_n, tm, tn);
  const i64 row0 = tm * BM;
  const int n0 = tn * BN;

  // this lane's part of each load: a row of x or of w, one chunk of it
  const Buffer xb = buffer_at(a.x + row0 * a.x_stride), wb = buffer_at(a.w + (i64)n0 * a.w_stride);
  unsigned at[kLoads];         // kDirect
  const int8_t* from[kLoads];  // otherwise
  v4i held[kLoads];
  int chunk[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int part = (wave * kLoads + i) * 16, slot = lane & 3, r = part + (lane >> 2);
    chunk[i] = slot ^ (part < BM ? x_key(r) : w_key(r - BM));
    const i64 row = part < BM ? min((i64)r, a.rows - 1 - row0) : min(r - BM, a.n - 1 - n0);
    if (kDirect) at[i] = (unsigned)row * (unsigned)(part < BM ? a.x_stride : a.w_stride) + chunk[i] * 16;
    else from[i] = part < BM ? a.x + (row0 + row) * a.x_stride : a.w + (n0 + row) * a.w_stride;
  }
  const int steps = (a.k + 63) / 64;
  auto issue = [&](int step, bool last) {
    int8_t* to = s_tiles + (step % kBufs) * kBuf + wave * kLoads * 1024;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const bool have = !last || step * 64 + chunk[i] * 16 < a.k;
      load_to_lds((wave * kLoads + i) * 16 < BM ? xb : wb, have ? at[i] : kOutside, step * 64, to + i * 1024);
    }
  };
  auto load = [&](int step) {
    if ((step + 1) * 64 <= a.k) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) __builtin_memcpy(&held[i], from[i] + step * 64 + chunk[i] * 16, 16);
    } else {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) held[i] = load_16_tail(from[i], step * 64 + chunk[i] * 16, a.k);
    }
  };
  auto put = [&](int step) {
    int8_t* to = s_tiles + (step % kBufs) * kBuf + wave * kLoads * 1024 + lane * 16;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) *reinterpret_cast<v4i*>(to + i * 1024) = held[i];
  };

  const int wm = (wave / (BN / 64)) * WM, wn = (wave % (BN / 64)) * 64;
  const int lr = lane & 15, lc = lane >> 4;
  constexpr int kRows = WM / 16;
  v4i dot[kRows][4];
#pragma unroll
  for (int j = 0; j < kRows; ++j)
#pragma unroll
    for (int t = 0; t < 4; ++t) dot[j][t] = v4i{0, 0, 0, 0};
  // the keys depend on neither t nor j
  const int wr = wn + w_row(0, lr), xr = wm + lr;
  const int w_at = BM * 64 + wr * 64 + ((lc ^ w_key(wr)) * 16), x_at = xr * 64 + ((lc ^ x_key(xr)) * 16);
  auto multiply = [&](int step) {
    const int8_t* tile = s_tiles + (step % kBufs) * kBuf;
    v4i w[4], x[kRows];
#pragma unroll
    for (int t = 0; t < 4; ++t) w[t] = *reinterpret_cast<const v4i*>(tile + w_at + w_row(t, 0) * 64);
#pragma unroll
    for (int j = 0; j < kRows; ++j) x[j] = *reinterpret_cast<const v4i*>(tile + x_at + j * 1024);
#pragma unroll
    for (int j = 0; j < kRows; ++j)
#pragma unroll
      for (int t = 0; t < 4; ++t) dot[j][t] = product_16(w[t], x[j], dot[j][t]);
    // reads two row groups ahead of the products
    __builtin_amdgcn_sched_group_barrier(0x100, kRows > 2 ? 6 : 4 + kRows, 0);
#pragma unroll
    for (int j = 0; j < kRows - 2; ++j) {
      __builtin_amdgcn_sched_group_barrier(0x008, 4, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, kRows > 2 ? 8 : 4 * kRows, 0);
  };
  const int tid = threadIdx.x;
  float scale = 0.0f, bias = 0.0f, row_scale = 0.0f;
  if (tid < BN) {
    const int c = min(n0 + tid, a.n - 1);
    scale = a.w_scale[c];
    if (a.bias) bias = a.bias[c];
  }
  if (tid < BM) row_scale = a.x_scale[min(row0 + tid, a.rows - 1)];
  auto put_scales = [&]() {
    if (tid < BN) {
      s_scale[tid] = scale;
      s_bias[tid] = bias;
    }
    if (tid < BM) s_rows[tid] = row_scale;
  };
  static_assert(kWaves * 64 >= BN && kWaves * 64 >= BM, "one thread per channel and per row");

  if constexpr (kDirect && kPer == 2) {
    issue(0, true);
    if (steps > 1) issue(1, true);
    put_scales();
    int s = 0;
    for (; s + 4 < steps; s += 2) {
      wait_loads<0>();
      meet();
      issue(s + 2, false);
      issue(s + 3, false);
      multiply(s);
      multiply(s + 1);
    }
    for (; s < steps; s += 2) {
      wait_loads<0>();
      meet();
      if (s + 2 < steps) issue(s + 2, true);
      if (s + 3 < steps) issue(s + 3, true);
      multiply(s);
      if (s + 1 < steps) multiply(s + 1);
    }
  } else if constexpr (kDirect) {
#pragma unroll
    for (int s = 0; s < kBufs - 1; ++s)
      if (s < steps) issue(s, true);
    put_scales();
    int s = 0;
    for (; s + kBufs < steps; ++s) {
      wait_loads<(kBufs - 2) * kLoads>();  // the loads of the steps after s may be under way
      meet();
      issue(s + kBufs - 1, false);
      multiply(s);
    }
    for (; s < steps; ++s) {
      if (s + kBufs - 1 < steps) {
        wait_loads<(kBufs - 2) * kLoads>();
        meet();
        issue(s + kBufs - 1, true);
      } else {
        wait_loads<0>();
        meet();
      }
      multiply(s);
    }
  } else {
    load(0);
    put_scales();
    put(0);
    if (steps > 1) load(1);
    for (int s = 0; s < steps; ++s) {
      meet();
      if (s + 1 < steps) put(s + 1);
      if (s + 2 < steps) load(s + 2);
      multiply(s);
    }
  }

  const bool wide = ((((uintptr_t)a.out) | (a.out_stride * sizeof(T))) & 15) == 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c = wn + h * 32 + lc * 8;
    float ws[8], b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      ws[i] = s_scale[c + i];
      b[i] = s_bias[c + i];
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const i64 row = row0 + wm + j * 16 + lr;
      if (row >= a.rows) continue;
      const float xs = s_rows[wm + j * 16 + lr];
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = xs * (float)dot[j][h * 2 + (i >> 2)][i & 3] * ws[i] + b[i];
      store_run<T, 8>(a, row, n0 + c, v, wide);
    }
  }
}

// ------------------------------------------------------------------ plain product, few tiles

// For products whose tiles would not fill the card: kRows * 16 rows x kCols * 16
// channels per workgroup, the input channels split over its waves, operands straight
// from memory into registers. The waves' partial sums are added in LDS (int32,
// exact in any order).
constexpr int kFewWaves = 8;
template <typename T, int kRows, int kCols>
__global__ void __launch_bounds__(kFewWaves * 64) k_product_few(ProductArgs a) {
  constexpr int kUnits = kRows * kCols;
  __shared__ v4i s_part[kFewWaves][kUnits][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tiles_n = (a.n + kCols * 16 - 1) / (kCols * 16);
  const i64 row0 = (i64)(blockIdx.x / tiles_n) * (kRows * 16);
  const int n0 = (blockIdx.x % tiles_n) * (kCols * 16);
  const int lr = lane & 15, lc = (lane >> 4) * 16;
  const int8_t *xrow[kRows], *wrow[kCols];
#pragma unroll
  for (int j = 0; j < kRows; ++j) xrow[j] = a.x + min(row0 + j * 16 + lr, a.rows - 1) * a.x_stride;
#pragma unroll
  for (int t = 0; t < kCols; ++t) wrow[t] = a.w + (i64)min(n0 + t * 16 + lr, a.n - 1) * a.w_stride;
  v4i dot[kRows][kCols];
#pragma unroll
  for (int j = 0; j < kRows; ++j)
#pragma unroll
    for (int t = 0; t < kCols; ++t) dot[j][t] = v4i{0, 0, 0, 0};

  const int steps = (a.k + 63) / 64, each = (steps + kFewWaves - 1) / kFewWaves;
  const int s0 = wave * each, s1 = min(s0 + each, steps);
  auto multiply = [&](const v4i* x, const v4i* w) {
#pragma unroll
    for (int j = 0; j < kRows; ++j)
#pragma unroll
      for (int t = 0; t < kCols; ++t) dot[j][t] = product_16(w[t], x[j], dot[j][t]);
  };
  auto load = [&](const int8_t* row, int c) {
    v4i v;
    __builtin_memcpy(&v, row + c, 16);
    return v;
  };
  constexpr int kAhead = kUnits >= 8 ? 2 : 4;  // steps whose loads are in flight together
  const int full = min(s1, a.k / 64);
  int s = s0;
  for (; s + kAhead <= full; s += kAhead) {
    v4i x[kAhead][kRows], w[kAhead][kCols];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
#pragma unroll
      for (int t = 0; t < kCols; ++t) w[u][t] = load(wrow[t], (s + u) * 64 + lc);
#pragma unroll
      for (int j = 0; j < kRows; ++j) x[u][j] = load(xrow[j], (s + u) * 64 + lc);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) multiply(x[u], w[u]);
  }
  for (; s < s1; ++s) {
    v4i x[kRows], w[kCols];
    if (s < full) {
#pragma unroll
      for (int t = 0; t < kCols; ++t) w[t] = load(wrow[t], s * 64 + lc);
#pragma unroll
      for (int j = 0; j < kRows; ++j) x[j] = load(xrow[j], s * 64 + lc);
    } else {
#pragma unroll
      for (int t = 0; t < kCols; ++t) w[t] = load_16_tail(wrow[t], s * 64 + lc, a.k);
#pragma unroll
      for (int j = 0; j < kRows; ++j) x[j] = load_16_tail(xrow[j], s * 64 + lc, a.k);
    }
    multiply(x, w);
  }
#pragma unroll
  for (int j = 0; j < kRows; ++j)
#pragma unroll
    for (int t = 0; t < kCols; ++t) s_part[wave][j * kCols + t][lane] = dot[j][t];
  __syncthreads();
  for (int unit = wave; unit < kUnits; unit += kFewWaves) {
    const i64 row = row0 + (unit / kCols) * 16 + lr;
    const int n = n0 + (unit % kCols) * 16 + (lane >> 4) * 4;
    if (row >= a.rows) continue;
    v4i sum = s_part[0][unit][lane];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) sum += s_part[w][unit][lane];
    const float xs = a.x_scale[row];
    T* out = static_cast<T*>(a.out) + row * a.out_stride;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < a.n)
        out[n + i] = from_f32<T>(xs * (float)sum[i] * a.w_scale[n + i] + (a.bias ? a.bias[n + i] : 0.0f));
  }
}

template <typename T, int BM, int BN, int WM, int kBufs, int kPer, bool kDirect>
void launch_tile(const ProductArgs& a, hipStream_t s) {
  const i64 tm = ceil_div(a.rows, BM);
  const int tn = (int)ceil_div(a.n, BN);
  launch("k_product_tile", k_product_tile<T, BM, BN, WM, kBufs, kPer, kDirect>, tm * tn, (BM / WM) * (BN / 64) * 64, s, a,
         tm, tn);
}

template <typename T, int kRows, int kCols>
void launch_few(const ProductArgs& a, hipStream_t s) {
  const i64 blocks = ceil_div(a.rows, kRows * 16) * ceil_div(a.n, kCols * 16);
  launch("k_product_few", k_product_few<T, kRows, kCols>, blocks, kFewWaves * 64, s, a);
}

// The variant of a plain product. Timed at 16384 x 4096 -> 4096 (a), 124800 x 256 -> 768 (b),
// 2048 x 1024 -> 1024 (c), 100 x 4096 -> 4096 (d), 64 x 1024 -> 1024 (e), bf16 out, in us:
//   tile        256x256  256x128  64x64  few rows (best split)
//   (a)             233      284    542  1415
//   (b)              61       57     82   383
//   (c)              16       12    8.8    18
//   (d)              43       28     19    15
//   (e)              13       10    7.0   5.6
// A tile's loads and products grow as its area, its traffic as its edge: the largest tile that
// fills the card is best, but 256 x 256 runs one workgroup a CU, whose stores nothing hides
// when the input channels are few. Through registers (unaligned) the order is the same
// ((a) with 4095 input channels: 296, 390, 842). The 64x64 tile against the best of the splits
// (4x2 but for two of them), around half as many tiles as CUs (128 here):
//   tiles                            64x64   split
//   128   1024 x 4096 -> 512          19.4    15.0
//   128   1024 x 256 -> 512            5.2     5.0
//   130   640 x 1024 -> 832            7.2     9.2
//   144   1003 x 601 -> 523, f32       6.9    11.0
//   144   1024 x 4096 -> 576          19.5    25.0
//   192   768 x 4096 -> 1024          19.2    24.7
//   256   1024 x 256 -> 1024           5.1     6.1
// A split of 130 tiles' work needs a second round of workgroups.
template <typename T>
void plain_product(const ProductArgs& a, hipStream_t s) {
  const i64 cus = device_cu_count();
  auto tiles = [&](int bm, int bn) { return ceil_div(a.rows, bm) * ceil_div(a.n, bn); };
  const bool direct = aligned_16(a.x, a.x_stride) && aligned_16(a.w, a.w_stride) && a.k % 16 == 0 &&
                      std::max(a.x_stride, a.w_stride) < (1 << 22);  // a tile's offsets stay below 2^31
  if (a.k >= 1024 && tiles(256, 256) >= cus + cus / 2)
    return direct ? launch_tile<T, 256, 256, 128, 4, 2, true>(a, s) : launch_tile<T, 256, 256, 128, 2, 1, false>(a, s);
  if (tiles(256, 128) >= cus)
    return direct ? launch_tile<T, 256, 128, 64, 3, 1, true>(a, s) : launch_tile<T, 256, 128, 64, 2, 1, false>(a, s);
  if (tiles(64, 64) > cus / 2)
    return direct ? launch_tile<T, 64, 64, 32, 4, 1, true>(a, s) : launch_tile<T, 64, 64, 32, 2, 1, false>(a, s);
  // few tiles: the most sharing that still gives every CU a workgroup
  if (tiles(64, 32) >= cus) return launch_few<T, 4, 2>(a, s);
  if (tiles(32, 32) >= cus) return launch_few<T, 2, 2>(a, s);
  if (tiles(32, 16) >= cus) return launch_few<T, 2, 1>(a, s);
  launch_few<T, 1, 1>(a, s);
}

}  // namespace

void product_i8(const ProductArgs& a, hipStream_t s) {
  if (a.rows == 0 || a.n == 0) return;
  if (a.map) return conv_i8(a, s);
  with_dtype(a.out_dtype, [&](auto t) { plain_product<decltype(t)>(a, s); });
}

}  // namespace tc
