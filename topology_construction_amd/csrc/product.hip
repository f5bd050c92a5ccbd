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

// ------------------------------------------------------------------ plain product, many tiles

// Tile t of `total` for this workgroup. Workgroups go to the 8 XCDs in turn, each with
// an L2 of its own: an XCD gets one contiguous range of tiles.
__device__ __forceinline__ i64 xcd_tile(i64 total) {
  const i64 b = blockIdx.x, q = total / 8, r = total % 8, x = b % 8;
  return x * q + min(x, r) + b / 8;
}

// The tile of output rows and of output channels: runs of `kGroup` row tiles
// take all channel tiles before the next run, so that tiles in flight together
// share rows and weights.
__device__ __forceinline__ void tile_place(i64 tile, i64 tiles_m, int tiles_n, i64& tm, int& tn) {
  constexpr int kGroup = 8;
  const i64 per = (i64)kGroup * tiles_n, g = tile / per, first = g * kGroup;
  const int size = (int)min((i64)kGroup, tiles_m - first), at = (int)(tile - g * per);
  tm = first + at % size;
  tn = at / size;
}

// 16 consecutive output channels of one row from n on: dot * (row scale * channel scale) + bias.
template <typename T>
__device__ __forceinline__ void store_16(const ProductArgs& a, i64 row, int n, const float v[16], bool wide) {
  T* out = static_cast<T*>(a.out) + row * a.out_stride + n;
  T r[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = from_f32<T>(v[i]);
  if (wide && n + 16 <= a.n) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(r) / 16; ++i)
      reinterpret_cast<v4i*>(out)[i] = reinterpret_cast<const v4i*>(r)[i];
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (n + i < a.n) out[i] = r[i];
  }
}

template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N < 64, "vmcnt has 6 bits");
  // vmcnt = N, the other counters left alone
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

// LDS keeps a row's 64 bytes of a step in four slots of 16. A wave reads 16 rows
// of the same chunk at once; the chunk's slot depends on the row so that
// neighbours in such a read fall into different banks.
__device__ __forceinline__ int x_key(int row) { return (row >> 1) & 3; }
// Row r of the weights' tile t is channel (r / 4) * 16 + t * 4 + r % 4 of a wave's 64, so
// that a lane's results of four tiles are 16 consecutive channels.
__device__ __forceinline__ int w_key(int row) { return ((row >> 1) & 1) | ((row >> 3) & 2); }

// 16 bytes at row + c, from any address; zeros from k on (c a multiple of 16, k > 0).
__device__ __forceinline__ v4i load_16_tail(const int8_t* row, int c, int k) {
  typedef unsigned long long u64x2 __attribute__((ext_vector_type(2)));
  u64x2 v{0, 0};
  if (k >= 16) {  // the 16 bytes that end the row, or are before its end, moved down
    const int from = min(c, k - 16), by = min(c - from, 16) * 8;
    __builtin_memcpy(&v, row + from, 16);
    const unsigned long long lo = by >= 64 ? v[1] : v[0], hi = by >= 64 ? 0 : v[1];
    const int left = by & 63;
    v[0] = by >= 128 ? 0 : (lo >> left) | (hi << 1 << (63 - left));
    v[1] = hi >> left;
  } else if (c == 0) {
    for (int i = 0; i < k; ++i) v[i >> 3] |= (unsigned long long)(uint8_t)row[i] << (8 * (i & 7));
  }
  return __builtin_bit_cast(v4i, v);
}

// A buffer of at most 2^31 - 1 bytes from `base` on, for loads by 32-bit offsets.
typedef __amdgpu_buffer_rsrc_t Buffer;
constexpr unsigned kOutside = 0x80000000u;  // an offset out of every buffer's range: such a lane loads zeros
__device__ __forceinline__ Buffer buffer_at(const int8_t* base) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(base), 0, 0x7fffffff, 0x00027000);
}

// 16 bytes per lane from the buffer into LDS at `to` + 16 * lane.
__device__ __forceinline__ void load_to_lds(Buffer from, unsigned lane_at, unsigned at, int8_t* to) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void*)to, 16, lane_at, at, 0, 0);
}

// BM x BN outputs per workgroup, (BM / WM) * (BN / 64) waves of WM x 64 each, in
// steps of 64 input channels. kDirect: rows and chunks on 16-byte boundaries go
// straight into LDS, kBufs - 1 steps ahead of the products. Otherwise, from any
// address, through registers: loaded two steps ahead, written one step ahead.
template <typename T, int BM, int BN, int WM, int kBufs, bool kDirect>
__global__ void __launch_bounds__((BM / WM) * (BN / 64) * 64)
    k_product_tile(ProductArgs a, i64 tiles_m, int tiles_n) {
  static_assert(kDirect || kBufs == 2, "one buffer is read, one written");
  constexpr int kWaves = (BM / WM) * (BN / 64);
  constexpr int kLoads = (BM + BN) / 16 / kWaves;  // per wave and step
  constexpr int kBuf = (BM + BN) * 64;
  __shared__ __align__(16) int8_t s_tiles[kBufs * kBuf];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  i64 tm;
  int tn;
  tile_place(xcd_tile(tiles_m * tiles_n), tiles_m, tiles_n, tm, tn);
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
  const int wr = wn + (lr >> 2) * 16 + (lr & 3), xr = wm + lr;
  const int w_at = BM * 64 + wr * 64 + ((lc ^ w_key(wr)) * 16), x_at = xr * 64 + ((lc ^ x_key(xr)) * 16);
  auto multiply = [&](int step) {
    const int8_t* tile = s_tiles + (step % kBufs) * kBuf;
    v4i w[4], x[kRows];
#pragma unroll
    for (int t = 0; t < 4; ++t) w[t] = *reinterpret_cast<const v4i*>(tile + w_at + t * 256);
#pragma unroll
    for (int j = 0; j < kRows; ++j) x[j] = *reinterpret_cast<const v4i*>(tile + x_at + j * 1024);
#pragma unroll
    for (int j = 0; j < kRows; ++j)
#pragma unroll
      for (int t = 0; t < 4; ++t) dot[j][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[t], x[j], dot[j][t], 0, 0, 0);
    // reads two row groups ahead of the products
    __builtin_amdgcn_sched_group_barrier(0x100, kRows > 2 ? 6 : 4 + kRows, 0);
#pragma unroll
    for (int j = 0; j < kRows - 2; ++j) {
      __builtin_amdgcn_sched_group_barrier(0x008, 4, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, kRows > 2 ? 8 : 4 * kRows, 0);
  };
  // every wave has its part of the step in LDS, and has read the step before
  auto meet = [&]() {
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  if constexpr (kDirect) {
#pragma unroll
    for (int s = 0; s < kBufs - 1; ++s)
      if (s < steps) issue(s, true);
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
    put(0);
    if (steps > 1) load(1);
    for (int s = 0; s < steps; ++s) {
      meet();
      if (s + 1 < steps) put(s + 1);
      if (s + 2 < steps) load(s + 2);
      multiply(s);
    }
  }

  const int n = n0 + wn + lc * 16;
  float ws[16], b[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int c = min(n + i, a.n - 1);
    ws[i] = a.w_scale[c];
    b[i] = a.bias ? a.bias[c] : 0.0f;
  }
  const bool wide = ((((uintptr_t)a.out) | (a.out_stride * sizeof(T))) & 15) == 0;
#pragma unroll
  for (int j = 0; j < WM / 16; ++j) {
    const i64 row = row0 + wm + j * 16 + lr;
    if (row >= a.rows) continue;
    const float xs = a.x_scale[row];
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = xs * (float)dot[j][i >> 2][i & 3] * ws[i] + b[i];
    store_16<T>(a, row, n, v, wide);
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
      for (int t = 0; t < kCols; ++t) dot[j][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[t], x[j], dot[j][t], 0, 0, 0);
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

template <typename T, int BM, int BN, int WM, int kBufs, bool kDirect>
void launch_tile(const ProductArgs& a, hipStream_t s) {
  const i64 tm = ceil_div(a.rows, BM);
  const int tn = (int)ceil_div(a.n, BN);
  launch("k_product_tile", k_product_tile<T, BM, BN, WM, kBufs, kDirect>, tm * tn, (BM / WM) * (BN / 64) * 64, s, a,
         tm, tn);
}

template <typename T, int kRows, int kCols>
void launch_few(const ProductArgs& a, hipStream_t s) {
  const i64 blocks = ceil_div(a.rows, kRows * 16) * ceil_div(a.n, kCols * 16);
  launch("k_product_few", k_product_few<T, kRows, kCols>, blocks, kFewWaves * 64, s, a);
}

bool aligned_16(const void* p, i64 stride) { return (((uintptr_t)p | (uintptr_t)stride) & 15) == 0; }

// The variant of a plain product. Timed at 16384 x 4096 -> 4096 (a), 124800 x 256 -> 768 (b),
// 2048 x 1024 -> 1024 (c), 100 x 4096 -> 4096 (d), 64 x 1024 -> 1024 (e), bf16 out, in us:
//   tile        256x256  256x128  64x64  few rows (best split)
//   (a)             236      272    539     -
//   (b)              66       60     88   347
//   (c)              18       12    9.1    17
//   (d)              44       29     19    14
//   (e)              15       10    7.2   4.0
// A tile's loads and products grow as its area, its traffic as its edge: the largest tile that
// fills the card is best, but 256 x 256 runs one workgroup a CU, whose stores nothing hides
// when the input channels are few. Through registers (unaligned) the order is the same
// ((a) with 4095 input channels: 304, 380, 799).
template <typename T>
void plain_product(const ProductArgs& a, hipStream_t s) {
  const i64 cus = device_cu_count();
  auto tiles = [&](int bm, int bn) { return ceil_div(a.rows, bm) * ceil_div(a.n, bn); };
  const bool direct = aligned_16(a.x, a.x_stride) && aligned_16(a.w, a.w_stride) && a.k % 16 == 0 &&
                      std::max(a.x_stride, a.w_stride) < (1 << 22);  // a tile's offsets stay below 2^31
  if (a.k >= 1024 && tiles(256, 256) >= cus + cus / 2)
    return direct ? launch_tile<T, 256, 256, 128, 3, true>(a, s) : launch_tile<T, 256, 256, 128, 2, false>(a, s);
  if (tiles(256, 128) >= cus)
    return direct ? launch_tile<T, 256, 128, 64, 3, true>(a, s) : launch_tile<T, 256, 128, 64, 2, false>(a, s);
  if (tiles(64, 64) > cus / 2)
    return direct ? launch_tile<T, 64, 64, 32, 4, true>(a, s) : launch_tile<T, 64, 64, 32, 2, false>(a, s);
  // few tiles: the most sharing that still gives every CU a workgroup
  if (tiles(64, 32) >= cus) return launch_few<T, 4, 2>(a, s);
  if (tiles(32, 32) >= cus) return launch_few<T, 2, 2>(a, s);
  if (tiles(32, 16) >= cus) return launch_few<T, 2, 1>(a, s);
  launch_few<T, 1, 1>(a, s);
}

}  // namespace

void product_i8(const ProductArgs& a, hipStream_t s) {
  if (a.rows == 0 || a.n == 0) return;
  with_dtype(a.out_dtype, [&](auto t) {
    using T = decltype(t);
    if (!a.map) return plain_product<T>(a, s);
    launch("k_product_any", k_product_any<T>, ceil_div(a.rows, kTile) * ceil_div(a.n, kTile), 256, s, a);
  });
}

}  // namespace tc
