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

// ------------------------------------------------------------------ many tiles

// Row i of the weights' matrix instruction t of a wave's channels, such that a lane's results are 8 consecutive
// channels, twice, and the two lanes of an output row are side by side.
__device__ __forceinline__ constexpr int w_row_32(int t, int i) {
  return t * 32 + (i >> 4) * 16 + (i >> 2 & 1) * 8 + (i >> 3 & 1) * 4 + (i & 3);
}

// LDS keeps a row's 64 bytes of a step in four slots of 16. A chunk's slot depends on the row, so that the 16 lanes
// that are served at a time (0 to 3, 12 to 15, 20 to 27 of each 32, and the others) find their rows' chunk in
// different banks, in either order of the rows.
__device__ __forceinline__ int slot_key(int row) { return (row >> 2) & 3; }

// The exponents of four steps (16 blocks) of a row, as the lanes take them: those of the even blocks, of the odd ones.
__device__ __forceinline__ v4i by_parity(v4i s) {
  return v4i{(int)__builtin_amdgcn_perm(s[1], s[0], 0x06040200), (int)__builtin_amdgcn_perm(s[3], s[2], 0x06040200),
             (int)__builtin_amdgcn_perm(s[1], s[0], 0x07050301), (int)__builtin_amdgcn_perm(s[3], s[2], 0x07050301)};
}

// BM x BN outputs per workgroup, (BM / WM) * (BN / WN) waves of WM x WN each, in steps of 128 input channels (64
// bytes of a row). kDirect: rows and chunks on 16-byte boundaries go straight into LDS, kBufs - 1 steps ahead of the
// products, or (kShort: no more steps than buffers) all at once. Otherwise, from any address, through registers: loaded
// three steps ahead, written two ahead. A step's second half is read while its first is multiplied, and the next step's first
// half while its second is: a barrier is not followed by a wait for LDS.
//
// The blocks' exponents go through registers, eight steps at a time (pieces of 16 bytes a row cost the caches as much as
// whole lines), and are sorted on the way into LDS so that a lane has those of its blocks of four steps in two words, a
// byte of which each matrix instruction picks.
template <typename T, int BM, int BN, int WM, int WN, int kBufs, bool kShort, bool kDirect>
__global__ void __launch_bounds__((BM / WM) * (BN / WN) * 64)
    k_product_mx4_tile(ProductMx4Args a, i64 tiles_m, int tiles_n) {
  constexpr int kThreads = (BM / WM) * (BN / WN) * 64, kWaves = kThreads / 64;
  static_assert(kDirect || (kBufs == 3 && !kShort), "one buffer is read, one waits, one is written");
  constexpr int kLoads = (BM + BN) / 16 / kWaves;  // per wave and step
  constexpr int kBuf = (BM + BN) * 64, kAhead = kShort ? kBufs : kBufs - 1;
  constexpr int kScales = (2 * (BM + BN) + kThreads - 1) / kThreads;  // pieces of exponents per thread
  // one array, as for the 8-bit product: tiles, exponents, bias
  __shared__ __align__(16) int8_t s_tiles[kBufs * kBuf + (BM + BN) * 32 + BN * 4];
  int8_t* const s_scale = s_tiles + kBufs * kBuf;
  float* const s_bias = reinterpret_cast<float*>(s_scale + (BM + BN) * 32);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  i64 tm;
  int tn;
  tile_place(xcd_block(blockIdx.x, tiles_m * tiles_n), tiles_m, tiles_n, tm, tn);
  const i64 row0 = tm * BM;
  const int n0 = tn * BN;
  const int8_t* const x0 = reinterpret_cast<const int8_t*>(a.x) + row0 * a.x_stride;
  const int8_t* const w0 = reinterpret_cast<const int8_t*>(a.w) + n0 * a.w_stride;

  // this lane's part of each load: a row of x or of w, one chunk of it
  const Buffer xb = buffer_at(x0), wb = buffer_at(w0);
  unsigned at[kLoads];  // kDirect
  v4i held[kLoads];     // otherwise
  const int chunk = (lane & 3) ^ slot_key(lane >> 2);  // the same for all loads, whose rows begin at multiples of 16
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int part = (wave * kLoads + i) * 16, r = part + (lane >> 2);
    const i64 row = part < BM ? min((i64)r, a.rows - 1 - row0) : min(r - BM, a.n - 1 - n0);
    at[i] = (unsigned)row * (unsigned)(part < BM ? a.x_stride : a.w_stride) + chunk * 16;
  }
  const int steps = (a.k + 127) / 128;
  auto issue = [&](int step) {
    int8_t* to = s_tiles + (step % kBufs) * kBuf + wave * kLoads * 1024;
    const bool have = step * 128 + chunk * 32 < a.k;
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      load_to_lds((wave * kLoads + i) * 16 < BM ? xb : wb, have ? at[i] : kOutside, step * 64, to + i * 1024);
  };
  // through registers: the rows of this lane's loads; the largest tile makes them anew for every step, since kept they take
  // registers that it has not (it would use scratch memory)
  constexpr bool kAnew = WM * WN >= 128 * 64;
  auto row_of = [&](int i, int lane) {
    const int part = (wave * kLoads + i) * 16, r = part + (lane >> 2);
    return part < BM ? x0 + min((i64)r, a.rows - 1 - row0) * a.x_stride : w0 + (i64)min(r - BM, a.n - 1 - n0) * a.w_stride;
  };
  const int8_t* from[kLoads];
  if constexpr (!kDirect && !kAnew) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) from[i] = row_of(i, lane);
  }
  auto load = [&](int step) {
    if (step >= steps) return;
    int l = lane;
    if constexpr (kAnew) asm volatile("" : "+v"(l));
    const int c = step * 64 + (kAnew ? (l & 3) ^ slot_key(l >> 2) : chunk) * 16;
    if ((step + 1) * 128 <= a.k) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) __builtin_memcpy(&held[i], (kAnew ? row_of(i, l) : from[i]) + c, 16);
    } else {
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        held[i] = load_32_tail(reinterpret_cast<const uint8_t*>(kAnew ? row_of(i, l) : from[i]), c, a.k);
    }
  };
  auto put = [&](int step) {
    if (step >= steps) return;
    int8_t* to = s_tiles + (step % kBufs) * kBuf + wave * kLoads * 1024 + lane * 16;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) *reinterpret_cast<v4i*>(to + i * 1024) = held[i];
  };

  // exponents: this thread's pieces of rows of the tile, x's rows first; in LDS first those of all rows' first four steps
  v4i scale_held[kScales];
  const int blocks = (a.k + 31) / 32, piece = tid & 1;
  auto scales_of = [&](int i, int tid) {
    const int r = (tid + i * kThreads) / 2;
    return r < BM ? a.x_scale + min(row0 + r, a.rows - 1) * a.x_scale_stride
                  : a.w_scale + (i64)min(n0 + r - BM, a.n - 1) * a.w_scale_stride;
  };
  const uint8_t* scale_from[kScales];
  if constexpr (!kAnew) {
#pragma unroll
    for (int i = 0; i < kScales; ++i) scale_from[i] = scales_of(i, tid);
  }
  auto load_scales = [&](int eight) {
    if (eight * 8 >= steps) return;
    int t = tid;
    if constexpr (kAnew) asm volatile("" : "+v"(t));
    const int first = eight * 32 + (t & 1) * 16;
    auto at = [&](int i) { return first + (kAnew ? scales_of(i, t) : scale_from[i]); };
    if ((eight + 1) * 32 <= blocks) {
#pragma unroll
      for (int i = 0; i < kScales; ++i) __builtin_memcpy(&scale_held[i], at(i), 16);
    } else {  // zeros beyond the last
#pragma unroll
      for (int i = 0; i < kScales; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int left = blocks - first - e * 4;
          int v = 0;
          if (left >= 4) __builtin_memcpy(&v, at(i) + e * 4, 4);
          else
            for (int k = 0; k < left; ++k) v |= (int)at(i)[e * 4 + k] << (8 * k);
          scale_held[i][e] = v;
        }
    }
  };
  auto put_scales = [&](int eight) {
    if (eight * 8 >= steps) return;
#pragma unroll
    for (int i = 0; i < kScales; ++i)
      if (tid + i * kThreads < 2 * (BM + BN))
        *reinterpret_cast<v4i*>(s_scale + (piece * (BM + BN) + (tid + i * kThreads) / 2) * 16) = by_parity(scale_held[i]);
  };

  const int wm = (wave / (BN / WN)) * WM, wn = (wave % (BN / WN)) * WN;
  const int lr = lane & 31, lh = lane >> 5;
  constexpr int kRows = WM / 32, kCols = WN / 32;
  using std::integral_constant;
  v16f dot[kRows][kCols];
#pragma unroll
  for (int j = 0; j < kRows; ++j)
#pragma unroll
    for (int t = 0; t < kCols; ++t) dot[j][t] = v16f{};
  // the keys depend on neither t nor j; the chunks of a step's two products
  const int wr = wn + w_row_32(0, lr), xr = wm + lr;
  int w_at[2], x_at[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    w_at[q] = BM * 64 + wr * 64 + (((2 * q + lh) ^ slot_key(wr)) * 16);
    x_at[q] = xr * 64 + (((2 * q + lh) ^ slot_key(xr)) * 16);
  }
  typedef int v2i __attribute__((ext_vector_type(2)));
  v2i ws[kCols], xs[kRows];  // the exponents of four steps
  auto read_scales = [&](int four) {
    const int8_t* const from = s_scale + (four & 1) * (BM + BN) * 16 + lh * 8;
#pragma unroll
    for (int t = 0; t < kCols; ++t) ws[t] = *reinterpret_cast<const v2i*>(from + (BM + wr + t * 32) * 16);
#pragma unroll
    for (int j = 0; j < kRows; ++j) xs[j] = *reinterpret_cast<const v2i*>(from + (xr + j * 32) * 16);
  };
  v4i w[2][kCols], x[2][kRows];  // of the two halves of a step
  auto read = [&](auto q, int step) {
    const int8_t* const tile = s_tiles + (step % kBufs) * kBuf;
#pragma unroll
    for (int t = 0; t < kCols; ++t) w[q][t] = *reinterpret_cast<const v4i*>(tile + w_at[q] + t * 2048);
#pragma unroll
    for (int j = 0; j < kRows; ++j) x[q][j] = *reinterpret_cast<const v4i*>(tile + x_at[q] + j * 2048);
  };
  // Beyond the last channel there are zeros, under exponents of zero.
  auto product = [&](auto of_four, auto q) {
    constexpr int kWord = of_four / 2, kByte = of_four % 2 * 2 + q;
#pragma unroll
    for (int j = 0; j < kRows; ++j)
#pragma unroll
      for (int t = 0; t < kCols; ++t)
        dot[j][t] = product_mx4<kByte>(w[q][t], x[q][j], dot[j][t], ws[t][kWord], xs[j][kWord]);
    // half a step's reads among half a step's products
    constexpr int kReads = kRows + kCols, kEach = kRows * kCols / kReads;
#pragma unroll
    for (int i = 0; i < kReads; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, kEach, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, kRows * kCols - kReads * kEach, 0);
  };
  if (tid < BN) s_bias[tid] = a.bias ? a.bias[min(n0 + tid, a.n - 1)] : 0.0f;
  static_assert(kThreads >= BN, "one thread per channel");
  const integral_constant<int, 0> k0;
  const integral_constant<int, 1> k1;

  load_scales(0);
  if constexpr (kDirect) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) issue(i);
  } else {
    load(0);
    put(0);
    load(1);
    put(1);
    load(2);
  }
  put_scales(0);
  if constexpr (kDirect) wait_loads<0>();
  meet();
  read_scales(0);
  read(k0, 0);
  for (int four = 0; four * 4 < steps; ++four) {
    auto go = [&](auto of_four) {
      const int step = four * 4 + of_four;
      if (step >= steps) return;
      // the next step's loads are done, those of steps after it may be under way (and, for a while, those of exponents)
      if (step > 0) {
        if constexpr (kDirect && !kShort) {
          wait_loads<(kAhead - 2) * kLoads>();
        }
        if constexpr (!kShort) meet();
      }
      if constexpr (kDirect) {
        if (!kShort) issue(step + kAhead);  // beyond the last step: zeros into a buffer that is not read
      } else {
        put(step + 2);
        load(step + 3);
      }
      if (!kShort && of_four == 0 && four % 2 == 0) load_scales(four / 2 + 1);
      __builtin_amdgcn_sched_barrier(0);
      read(k1, step);
      product(of_four, k0);
      __builtin_amdgcn_sched_barrier(0);
      if (!kShort && of_four == 2 && four % 2 == 1) put_scales(four / 2 + 1);  // over those that all waves have read: barriers lie between
      read(k0, step + 1);
      product(of_four, k1);
      if (of_four == 3) read_scales(four + 1);
      __builtin_amdgcn_sched_barrier(0);
    };
    go(integral_constant<int, 0>());
    go(integral_constant<int, 1>());
    go(integral_constant<int, 2>());
    go(integral_constant<int, 3>());
  }

  // Results go through this wave's part of the tiles' and exponents' LDS, so that a store has whole pieces of rows: 32 rows of
  // kSpan channels at a time, rows 16 bytes apart besides (banks).
  constexpr int kPart = (kBufs * kBuf + (BM + BN) * 32) / kWaves / 16 * 16;
  constexpr int kSpan = 32 * (WN * (int)sizeof(T) + 16) <= kPart ? WN : 32;
  constexpr int kPitch = kSpan * sizeof(T) + 16, kEach = 16 / sizeof(T), kLanes = kSpan / kEach;  // a lane's channels, lanes a row
  static_assert(32 * kPitch <= kPart, "a wave's results fit its part");
  int8_t* const part = s_tiles + wave * kPart;
  const bool wide = aligned_16(a.out, a.out_stride * (i64)sizeof(T));
  if constexpr (kDirect) wait_loads<0>();
  meet();  // all waves have read their last tile
#pragma unroll
  for (int j = 0; j < kRows; ++j)
#pragma unroll
    for (int span = 0; span < WN; span += kSpan) {
#pragma unroll
      for (int t = span / 32; t < (span + kSpan) / 32; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c = t * 32 + h * 16 + lh * 8;
          T v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = from_f32<T>(dot[j][t][h * 8 + i] + s_bias[wn + c + i]);
          __builtin_memcpy(__builtin_assume_aligned(part + lr * kPitch + (c - span) * sizeof(T), 16), v, sizeof(v));
        }
#pragma unroll
      for (int i = lane; i < 32 * kLanes; i += 64) {
        const int r = i / kLanes, c = i % kLanes * kEach, n = n0 + wn + span + c;
        const v4i v = *reinterpret_cast<const v4i*>(part + r * kPitch + c * sizeof(T));
        const i64 row = row0 + wm + j * 32 + r;
        if (row >= a.rows || n >= a.n) continue;
        T* out = static_cast<T*>(a.out) + row * a.out_stride + n;
        if (n + kEach > a.n) {
          const T* one = reinterpret_cast<const T*>(&v);
#pragma unroll
          for (int e = 0; e < kEach; ++e)
            if (n + e < a.n) out[e] = one[e];
        } else if (wide) {
          __builtin_nontemporal_store(v, reinterpret_cast<v4i*>(out));
        } else {
          __builtin_memcpy(out, &v, 16);
        }
      }
    }
}

// ------------------------------------------------------------------ few tiles

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
  const int s0 = wave * each, s1 = min(s0 + each, steps), whole = min(s1, a.k / 128);
  auto multiply = [&](const v4i* x, const v4i* w, const int* xs, const int* ws) {
#pragma unroll
    for (int j = 0; j < kRows; ++j)
#pragma unroll
      for (int t = 0; t < kCols; ++t) dot[j][t] = product_mx4<0>(w[t], x[j], dot[j][t], ws[t], xs[j]);
  };
  auto load = [&](const uint8_t* at) {
    v4i v;
    __builtin_memcpy(&v, at, 16);
    return v;
  };
  constexpr int kAhead = 4;  // steps whose loads are in flight together; a row's exponents of four steps are 16 bytes
  int s = s0;
  for (; s + kAhead <= whole; s += kAhead) {
    v4i x[kAhead][kRows], w[kAhead][kCols], xe[kRows], we[kCols];
#pragma unroll
    for (int t = 0; t < kCols; ++t) we[t] = load(wscale[t] + s * 4);
#pragma unroll
    for (int j = 0; j < kRows; ++j) xe[j] = load(xscale[j] + s * 4);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
#pragma unroll
      for (int t = 0; t < kCols; ++t) w[u][t] = load(wrow[t] + (s + u) * 64 + lc * 16);
#pragma unroll
      for (int j = 0; j < kRows; ++j) x[u][j] = load(xrow[j] + (s + u) * 64 + lc * 16);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      int xs[kRows], ws[kCols];
#pragma unroll
      for (int t = 0; t < kCols; ++t) ws[t] = we[t][u] >> (8 * lc);
#pragma unroll
      for (int j = 0; j < kRows; ++j) xs[j] = xe[j][u] >> (8 * lc);
      multiply(x[u], w[u], xs, ws);
    }
  }
  for (; s < s1; ++s) {
    v4i x[kRows], w[kCols];
    int xs[kRows], ws[kCols];
    const int block = s * 4 + lc;
    const bool have = block * 32 < a.k;
#pragma unroll
    for (int t = 0; t < kCols; ++t) {
      w[t] = s < whole ? load(wrow[t] + block * 16) : load_32_tail(wrow[t], block * 16, a.k);
      ws[t] = have ? wscale[t][block] : 0;
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      x[j] = s < whole ? load(xrow[j] + block * 16) : load_32_tail(xrow[j], block * 16, a.k);
      xs[j] = have ? xscale[j][block] : 0;
    }
    multiply(x, w, xs, ws);
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

template <typename T, int BM, int BN, int WM, int WN, int kBufs, bool kShort>
void launch_tile(const ProductMx4Args& a, hipStream_t s) {
  const bool direct = aligned_16(a.x, a.x_stride) && aligned_16(a.w, a.w_stride) && a.k % 32 == 0 &&
                      std::max(a.x_stride, a.w_stride) < (1 << 22);  // a tile's offsets stay below 2^31
  const i64 tm = ceil_div(a.rows, BM);
  const int tn = (int)ceil_div(a.n, BN);
  launch("k_product_mx4_tile",
         direct ? k_product_mx4_tile<T, BM, BN, WM, WN, kBufs, kShort, true> : k_product_mx4_tile<T, BM, BN, WM, WN, 3, false, false>,
         tm * tn, (BM / WM) * (BN / WN) * 64, s, a, tm, tn);
}

// The variant, and what others took (us, bf16 out, captured launches one after another):
//   rows x c_in -> c_out       256x256  128x128  64x64  256x128, all steps at once   32x32  16x16 (few)
//   16384 x 4096 -> 4096           165      204    300
//   16384 x 4095 -> 4096           186      222    334   (through registers)
//   3000 x 4096 -> 4096           34.5     47.1   60.0
//   2048 x 4096 -> 4096           30.4     26.9   42.1
//   2500 x 2048 -> 2048           18.6     13.7   16.1
//   1024 x 4096 -> 4096           28.9     19.3   21.7
//   1500 x 4096 -> 1500                    18.7   15.8
//   400 x 4096 -> 4096            27.4     17.4   12.0
//   124800 x 256 -> 768           55.2     63.1   74.0   42.0
//   124800 x 64 -> 64                      11.4    8.3    8.0
//   4000 x 256 -> 256                              3.9    5.8
//   100 x 4096 -> 4096                             9.8                                  12.5   17.9
//   64 x 4096 -> 4096                              9.9                                   8.1   12.1
//   32 x 4096 -> 1024                              7.0                                   7.2    5.0
//   8 x 8192 -> 8192                              16.2                                  10.9   10.6
//   16 x 4096 -> 4096                              9.6                                   7.0    5.5
//   1 x 1024 -> 4096                               4.0                                          3.4
// The largest tile that gives most CUs one is best; with no more than two steps of input channels the stores are most of the
// time, and two workgroups of eight waves a CU (62 KB of LDS and 112 registers each) have one's under the other's loads.
template <typename T>
void product(const ProductMx4Args& a, hipStream_t s) {
  const i64 cus = device_cu_count();
  auto tiles = [&](int bm, int bn) { return ceil_div(a.rows, bm) * ceil_div(a.n, bn); };
  if (a.rows <= 8 || tiles(64, 64) < cus / 2)
    return a.rows > 16 && tiles(32, 32) >= cus ? launch_few<T, 2, 2>(a, s) : launch_few<T, 1, 1>(a, s);
  if (a.k <= 256)
    return tiles(256, 128) >= 2 * cus ? launch_tile<T, 256, 128, 64, 64, 2, true>(a, s)
                                      : launch_tile<T, 64, 64, 32, 32, 4, false>(a, s);
  if (tiles(256, 256) >= cus * 3 / 4) return launch_tile<T, 256, 256, 128, 64, 4, false>(a, s);
  if (tiles(128, 128) >= cus) return launch_tile<T, 128, 128, 64, 64, 3, false>(a, s);
  launch_tile<T, 64, 64, 32, 32, 4, false>(a, s);
}

}  // namespace

void product_mx4(const ProductMx4Args& a, hipStream_t s) {
  if (a.rows == 0) return;
  with_dtype(a.out_dtype, [&](auto t) { product<decltype(t)>(a, s); });
}

}  // namespace tc
