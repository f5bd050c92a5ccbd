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
// that a lane's results of two instructions are 8 consecutive output channels.
template <int kCols>
__device__ __forceinline__ constexpr int weight_row(int t, int r) {
  if (kCols == 1) return r;
  return (t >> 1) * 32 + (r >> 2) * 8 + (t & 1) * 4 + (r & 3);
}
// The LDS slot key of such a row: a function of r alone that differs between the
// rows one read takes together, two by two.
template <int kCols>
__device__ __forceinline__ constexpr int weight_key(int row) {
  if (kCols == 1) return (row >> 1) & 3;
  return ((row >> 1) & 1) | ((row >> 2) & 2);
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

// The place of row `tid` of a tile in the order of its rows: the Gray rank of its taps' mask,
// a bit a tap, then its number (below 256).
__device__ __forceinline__ uint32_t order_key(uint32_t mask, int taps, int tid) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) mask ^= mask >> d;
  mask <<= taps < 32 ? 32 - taps : 0;
  return (mask & ~255u) | tid;
}
template <int BM>
__device__ __forceinline__ int rank_of(const uint32_t* s_key, int tid) {
  const uint32_t mine = s_key[tid];
  int rank = 0;
#pragma unroll 8
  for (int i = 0; i < BM; i += 4) {
    const uint4 o = *reinterpret_cast<const uint4*>(s_key + i);
    rank += (o.x < mine) + (o.y < mine) + (o.z < mine) + (o.w < mine);
  }
  return rank;
}

// One workgroup of four waves per 64 kRows output rows and 16 kCols output
// channels; a wave has kRows groups of 16 rows.
//
// Order of the rows: a tap is absent for most rows of a surface's map, and a group
// of 16 skips the taps that none of its rows has. The tile's rows are sorted by the
// Gray rank of their masks, so that rows of like masks share a group (16 shells of
// resolution 64, 39% of the entries there: 75% of the groups' taps in the rows' own order,
// 64% sorted; a transposed 2x2x2: 70%, 16%); group g goes to wave g % 4.
//
// A stage is one tap and 64 kSteps input channels (kWide: the rows have more than that, a tap
// takes several stages, and its integer sums are kept across them). Its weights are
// shared by the waves, two stages of them in LDS. Its rows are gathered by each wave into
// LDS of its own, in 16 rows x 64 bytes a load (a lane's 16 bytes of a row of its own, as the
// matrix operand has them, would cost a load three times the time), and read from there as
// operands before the next stage's are asked for. kDirect: rows and weights on 16-byte
// boundaries go straight into LDS, otherwise through registers, from any address.
//
// 116k rows, 27 taps, 128 -> 128: 62 us a call in a row of calls (67 traced alone), 1.8 us a stage beside 14
// for order, first loads and stores (one tap: 15.5). The matrix units are busy 22% of the cycles, 0.53 us
// of a stage: what is left is that two workgroups a CU overlap products, LDS and gathers no better. Sharing
// the rows among waves that split the channels (balanced skips, but three branches for every 64 products)
// took 81 us where this took 69, all groups without branches 78.
//
// kWide keeps integer sums beside the float ones: 309 registers with 64 output channels (358 through
// registers), one workgroup a CU, and rows gathered again for every 64 channels. 65k rows, 27 taps, 256 -> 256:
// 310 us for the 46 that its operations take.
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
    const int32_t* m = a.map + min(row0 + tid, a.rows - 1) * taps;
    const auto has = [&](int e) { return (uint32_t)((uint32_t)e < (uint32_t)a.n_src); };
    if (taps >= 4 && taps <= 32) {  // all loads under way together
      v4i e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i * 4 < taps) __builtin_memcpy(&e[i], m + min(i * 4, taps - 4), 16);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i * 4 < taps)
          mask |= (has(e[i][0]) | has(e[i][1]) << 1 | has(e[i][2]) << 2 | has(e[i][3]) << 3) << min(i * 4, taps - 4);
    } else {
      const int every = (taps + 31) / 32;
#pragma unroll 8
      for (int b = 0; b < 32; ++b)
        if (b * every < taps) mask |= has(m[b * every]) << b;
    }
    s_key[tid] = order_key(row0 + tid < a.rows ? mask : 0, taps, tid);
  }
  __syncthreads();
  if (tid < BM) s_order[rank_of<BM>(s_key, tid)] = tid;
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

  // the map entry of this lane's row at a tap (taps in turn), -1: none
  auto entry_at = [&](int tap) {
    if (tap > 0 && (tap & 3) == 0) {
      entries = entries_ahead;
      entries_ahead = four_entries(tap + 4);
    }
    const int at = tap - (taps >= 4 ? min(tap & ~3, taps - 4) : 0);
    const int e = at == 0 ? entries[0] : at == 1 ? entries[1] : at == 2 ? entries[2] : entries[3];
    return live && (uint32_t)e < (uint32_t)a.n_src ? e : -1;
  };
  auto group_has = [&](unsigned long long h, int j) { return (h >> (16 * j) & 0xffff) != 0; };
  auto ask = [&](int tap, int c0, int buffer, unsigned long long have, const unsigned (&src)[kRows]) {
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
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int c = c0 + s * 64 + load_chunk;
        if constexpr (kDirect) {
          load_to_lds(xb, (src[j] + c) | (c < k ? 0 : kOutside), 0, my_x + (j * kSteps + s) * 1024);
        } else if ((int)src[j] >= 0) {
          const int8_t* row = a.x + (int)src[j] * a.x_stride;
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
  // the rows a lane loads, one of each group, as the lanes that own them have them: kDirect:
  // byte offsets, otherwise their numbers; from 2^31 on: none
  auto rows_of = [&](int entry, unsigned (&src)[kRows]) {
    const unsigned at = entry < 0 ? kOutside : kDirect ? (unsigned)entry * (unsigned)a.x_stride : (unsigned)entry;
#pragma unroll
    for (int j = 0; j < kRows; ++j) src[j] = __shfl(at, j * 16 + load_row, kWave);
  };
  int entry = entry_at(0);
  unsigned src[kRows];
  unsigned long long have = __ballot(entry >= 0);
  float scale = entry >= 0 ? a.x_scale[entry] : 0.0f;  // of this lane's row
  rows_of(entry, src);
  ask(0, 0, 0, have, src);
  put(0);
  int tap = 0, c0 = 0;
  for (int stage = 0; tap < taps; ++stage) {
    const bool last = !kWide || c0 + 64 * kSteps >= k;  // of the tap
    const int next_tap = last ? tap + 1 : tap, next_c0 = last ? 0 : c0 + 64 * kSteps;
    const bool more = next_tap < taps;
    const unsigned long long now = have;
    if (last && more) {
      entry = entry_at(next_tap);
      have = __ballot(entry >= 0);
      rows_of(entry, src);
    }
    wait_loads<0>();
    meet();
    // this stage's operands and scales
    v4i x[kRows][kSteps], w[kPart][kSteps];
    float xs[kRows];
    const int8_t* w_tile = s_w + (stage & 1) * BN * 64 * kSteps;
    auto weights = [&](int part) {
#pragma unroll
      for (int t = 0; t < kPart; ++t) {
        const int r = weight_row<kCols>(part * kPart + t, lr);
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
          w[t][s] = *reinterpret_cast<const v4i*>(w_tile + (s * BN + r) * 64 + ((lc ^ weight_key<kCols>(r)) * 16));
      }
    };
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
        x[j][s] = *reinterpret_cast<const v4i*>(my_x + (j * kSteps + s) * 1024 + x_at);
      xs[j] = last ? __shfl(scale, j * 16 + lr, kWave) : 0.0f;
    }
    weights(0);
    wait_lds();  // the operands' LDS may be written again
    if (more) {
      if (last) scale = entry >= 0 ? a.x_scale[entry] : 0.0f;
      ask(next_tap, next_c0, (stage + 1) & 1, have, src);
    }
    if (now) {
#pragma unroll
      for (int part = 0; part < kCols / kPart; ++part) {
        if (part > 0) weights(part);
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
            __builtin_amdgcn_sched_group_barrier(0x008, kSteps * kPart, 0);
            __builtin_amdgcn_sched_group_barrier(0x002, 8 * kPart, 0);
          }
        }
      }
    }
    if (more) put((stage + 1) & 1);
    tap = next_tap;
    c0 = next_c0;
  }

  constexpr int kPair = kCols < 2 ? 1 : 2;  // instructions of one run of channels
#pragma unroll
  for (int t = 0; t < kCols; t += kPair) {
    const Channels<kPair * 4> out(a, n0 + t * 16 + lc * 4 * kPair);
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const i64 row = row0 + s_order[(j * kConvWaves + wave) * 16 + lr];
      if (row >= a.rows) continue;
      float v[kPair * 4];
#pragma unroll
      for (int i = 0; i < kPair * 4; ++i) v[i] = acc[j][t + i / 4][i % 4];
      out.store(a, row, v);
    }
  }
}

// Few weights: those of all taps stay in LDS, beside the map entries of the workgroup's
// 256 rows. The rows are sorted by their masks as in k_conv_tile; then every wave goes
// through the taps of its four groups by itself, without a barrier, one tap of each group under way
// at a time, rows straight from memory as matrix operands (from any address).
template <int kCols, int kSteps>
__global__ void __launch_bounds__(kConvWaves * 64, 2) k_conv_resident(ProductArgs a) {
  constexpr int BM = kConvWaves * 64, BN = kCols * 16, kGroups = 4;
  extern __shared__ __align__(16) int8_t s_dynamic[];  // weights, then entries [BM][taps | 1]
  __shared__ __align__(16) uint32_t s_key[BM];
  __shared__ uint32_t s_mask[BM];
  __shared__ int s_order[BM];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lc = lane >> 4;
  const i64 row0 = xcd_block(blockIdx.x, gridDim.x) * BM;
  const int taps = a.taps, k = a.k, pitch = taps | 1, parts = taps * kSteps * kCols;
  int32_t* const s_map = reinterpret_cast<int32_t*>(s_dynamic + parts * 1024);

  {
    uint32_t mask = 0;
    const bool live = row0 + tid < a.rows;
    const int32_t* m = a.map + min(row0 + tid, a.rows - 1) * taps;
    int32_t* const mine = s_map + tid * pitch;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i * 4 >= taps) break;
      const int first = taps >= 4 ? min(i * 4, taps - 4) : 0;
      v4i e;
      if (taps >= 4) {
        __builtin_memcpy(&e, m + first, 16);
      } else {
#pragma unroll
        for (int u = 0; u < 4; ++u) e[u] = m[min(u, taps - 1)];
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (first + u >= taps) continue;
        const bool has = live && (uint32_t)e[u] < (uint32_t)a.n_src;
        mine[first + u] = has ? e[u] : -1;
        mask |= (uint32_t)has << (first + u);
      }
    }
    s_mask[tid] = mask;
    s_key[tid] = order_key(mask, taps, tid);
  }
  const int load_row = lane >> 2;
#pragma unroll 4
  for (int part = wave; part < parts; part += kConvWaves) {
    const int r = part % kCols * 16 + load_row;
    const int c = part / kCols % kSteps * 64 + ((lane & 3) ^ weight_key<kCols>(r)) * 16;
    const int8_t* from = a.w + ((i64)(part / (kCols * kSteps)) * a.n + min(r, a.n - 1)) * k;
    *reinterpret_cast<v4i*>(s_dynamic + part * 1024 + lane * 16) =
        k >= 16 ? weight_16_end(from, c, k) : load_16_tail(from, c, k);
  }
  __syncthreads();
  s_order[rank_of<BM>(s_key, tid)] = tid;
  __syncthreads();

  // group j of this wave: rows (4 j + wave) * 16 on of that order
  uint32_t own = s_mask[s_order[(lc * kConvWaves + wave) * 16 + lr]];
  own = lanes_reduce<16>(own, [](uint32_t x, uint32_t y) { return x | y; });
  uint32_t left[kGroups];
  const int32_t* entries[kGroups];
#pragma unroll
  for (int j = 0; j < kGroups; ++j) {
    left[j] = __builtin_amdgcn_readlane(own, j * 16);
    entries[j] = s_map + s_order[(j * kConvWaves + wave) * 16 + lr] * pitch;
  }
  v4i x[kGroups][kSteps];
  float xs[kGroups];
  int at[kGroups];  // the tap under way, -1: none
  auto ask = [&](int j) {
    at[j] = left[j] ? __builtin_ctz(left[j]) : -1;
    if (at[j] < 0) return;
    left[j] &= left[j] - 1;
    const int e = entries[j][at[j]];
    const int8_t* from = a.x + max(e, 0) * a.x_stride;  // any row where there is none: its scale is zero
    xs[j] = e >= 0 ? a.x_scale[e] : 0.0f;
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
      x[j][s] = k >= 16 ? load_16_end(from, s * 64 + lc * 16, k) : load_16_tail(from, s * 64 + lc * 16, k);
  };
  v4f acc[kGroups][kCols];
#pragma unroll
  for (int j = 0; j < kGroups; ++j) {
    ask(j);
#pragma unroll
    for (int t = 0; t < kCols; ++t) acc[j][t] = v4f{0, 0, 0, 0};
  }
  while (max(max(at[0], at[1]), max(at[2], at[3])) >= 0) {
#pragma unroll
    for (int j = 0; j < kGroups; ++j) {
      if (at[j] < 0) continue;
      const int8_t* tile = s_dynamic + at[j] * (kSteps * kCols * 1024);
      v4i d[kCols];
#pragma unroll
      for (int t = 0; t < kCols; ++t) {
        const int r = weight_row<kCols>(t, lr);
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          const v4i w = *reinterpret_cast<const v4i*>(tile + (s * BN + r) * 64 + ((lc ^ weight_key<kCols>(r)) * 16));
          d[t] = product_16(w, x[j][s], s == 0 ? v4i{0, 0, 0, 0} : d[t]);
        }
      }
      const float scale = xs[j];
      ask(j);
#pragma unroll
      for (int t = 0; t < kCols; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][t][i] += scale * (float)d[t][i];
    }
  }

  constexpr int kPair = kCols < 2 ? 1 : 2;
#pragma unroll
  for (int t = 0; t < kCols; t += kPair) {
    const Channels<kPair * 4> out(a, t * 16 + lc * 4 * kPair);
#pragma unroll
    for (int j = 0; j < kGroups; ++j) {
      const i64 row = row0 + s_order[(j * kConvWaves + wave) * 16 + lr];
      if (row >= a.rows) continue;
      float v[kPair * 4];
#pragma unroll
      for (int i = 0; i < kPair * 4; ++i) v[i] = acc[j][t + i / 4][i % 4];
      out.store(a, row, v);
    }
  }
}

// Rows that do not fill the card in tiles of 256: 64 of them a workgroup, 16 a wave, and as
// many taps a stage as registers take, so that their loads are under way together. The loads
// of a stage (through registers, from any address) are asked for while the stage before is
// computed; its weights are shared by the waves, in one buffer of LDS. At most 64 output
// channels: with 128 the registers hold fewer workgroups a CU (14k rows, 100 -> 96: 44 us for 29).
// Far from what its bytes and operations take (those 29 us: 1.4): of nine stages each has two barriers
// and one set of loads to wait for, with few waves a CU to fill the wait (read from the code, not measured apart).
template <int kCols, int kSteps, bool kWide>
__global__ void __launch_bounds__(kConvWaves * 64, kWide ? 2 : 3) k_conv_mid(ProductArgs a, int tiles_n) {
  constexpr int kTaps = kCols * kSteps > 4 ? 3 : 4;  // of a stage
  constexpr int BN = kCols * 16;
  constexpr int kWeightParts = kTaps * kSteps * kCols;  // loads of 16 rows x 64 bytes
  constexpr int kWeightLoads = (kWeightParts + kConvWaves - 1) / kConvWaves, kRowLoads = kTaps * kSteps;  // a wave
  constexpr int kPair = kCols < 2 ? 1 : 2;
  __shared__ __align__(16) int8_t s_all[(kWeightParts + kConvWaves * kRowLoads) * 1024];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lc = lane >> 4, load_row = lane >> 2;
  const i64 tile = xcd_block(blockIdx.x, gridDim.x);
  const i64 row = tile / tiles_n * (kConvWaves * 16) + wave * 16 + lr;
  const int n0 = (int)(tile % tiles_n) * BN;
  const int taps = a.taps, k = a.k;
  int8_t* const my_x = s_all + (kWeightParts + wave * kRowLoads) * 1024;

  // lane (u, r) of four by 16 holds the map entry and the scale of row r at tap u of the stage
  const int32_t* my_map = a.map + min(row, a.rows - 1) * taps;
  auto entry_at = [&](int tap0) {
    const int e = my_map[min(tap0 + lc, taps - 1)];
    return row < a.rows && lc < kTaps && tap0 + lc < taps && (uint32_t)e < (uint32_t)a.n_src ? e : -1;
  };
  v4i x_held[kRowLoads], w_held[kWeightLoads];
#pragma unroll
  for (int i = 0; i < kRowLoads; ++i) x_held[i] = v4i{0, 0, 0, 0};
  auto ask = [&](int entry, int tap0, int c0) {
#pragma unroll
    for (int i = 0; i < kWeightLoads; ++i) {
      const int part = i * kConvWaves + wave;
      if (part < kWeightParts) {
        const int r = part % kCols * 16 + load_row;
        const int c = c0 + part / kCols % kSteps * 64 + ((lane & 3) ^ weight_key<kCols>(r)) * 16;
        const int tap = min(tap0 + part / (kCols * kSteps), taps - 1);
        const int8_t* from = a.w + ((i64)tap * a.n + min(n0 + r, a.n - 1)) * k;
        w_held[i] = k >= 16 ? weight_16_end(from, c, k) : load_16_tail(from, c, k);
      }
    }
    if (!__any(entry >= 0)) return;
#pragma unroll
    for (int u = 0; u < kTaps; ++u) {
      // any row where there is none: its scale is zero
      const int8_t* from = a.x + max(__shfl(entry, u * 16 + load_row, kWave), 0) * a.x_stride;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int c = c0 + s * 64 + ((lane & 3) ^ x_key(load_row)) * 16;
        x_held[u * kSteps + s] = k >= 16 ? load_16_end(from, c, k) : load_16_tail(from, c, k);
      }
    }
  };

  v4f acc[kCols];
  v4i dot[kWide ? kTaps : 1][kCols];
#pragma unroll
  for (int t = 0; t < kCols; ++t) {
    acc[t] = v4f{0, 0, 0, 0};
#pragma unroll
    for (int u = 0; u < (kWide ? kTaps : 1); ++u) dot[u][t] = v4i{0, 0, 0, 0};
  }
  const int x_at = lr * 64 + ((lc ^ x_key(lr)) * 16);
  int entry = entry_at(0), entry_ahead = entry_at(kTaps);
  float scale = entry >= 0 ? a.x_scale[entry] : 0.0f;
  ask(entry, 0, 0);
  for (int tap0 = 0, c0 = 0; tap0 < taps;) {
    const bool last = !kWide || c0 + 64 * kSteps >= k;  // of these taps
    const int next_tap = last ? tap0 + kTaps : tap0, next_c0 = last ? 0 : c0 + 64 * kSteps;
    const unsigned long long now = __ballot(entry >= 0);
    meet();  // the stage before has been read
#pragma unroll
    for (int i = 0; i < kWeightLoads; ++i) {
      const int part = i * kConvWaves + wave;
      if (part < kWeightParts) *reinterpret_cast<v4i*>(s_all + part * 1024 + lane * 16) = w_held[i];
    }
#pragma unroll
    for (int i = 0; i < kRowLoads; ++i) *reinterpret_cast<v4i*>(my_x + i * 1024 + lane * 16) = x_held[i];
    float xs[kTaps];
    if (last) {
#pragma unroll
      for (int u = 0; u < kTaps; ++u) xs[u] = __shfl(scale, u * 16 + lr, kWave);
      entry = entry_ahead;
      if (next_tap < taps) {
        entry_ahead = entry_at(next_tap + kTaps);
        scale = entry >= 0 ? a.x_scale[entry] : 0.0f;
      }
    }
    meet();
    if (next_tap < taps) ask(entry, next_tap, next_c0);
#pragma unroll
    for (int u = 0; u < kTaps; ++u) {
      if (!(now >> (16 * u) & 0xffff)) continue;
      v4i x[kSteps];
#pragma unroll
      for (int s = 0; s < kSteps; ++s) x[s] = *reinterpret_cast<const v4i*>(my_x + (u * kSteps + s) * 1024 + x_at);
#pragma unroll
      for (int t = 0; t < kCols; ++t) {
        const int r = weight_row<kCols>(t, lr);
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          const v4i w = *reinterpret_cast<const v4i*>(s_all + ((u * kSteps + s) * BN + r) * 64 +
                                                      ((lc ^ weight_key<kCols>(r)) * 16));
          v4i& d = dot[kWide ? u : 0][t];
          d = product_16(w, x[s], !kWide && s == 0 ? v4i{0, 0, 0, 0} : d);
        }
      }
      if (last) {
#pragma unroll
        for (int t = 0; t < kCols; ++t) {
          v4i& d = dot[kWide ? u : 0][t];
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[t][i] += xs[u] * (float)d[i];
          if (kWide) d = v4i{0, 0, 0, 0};
        }
      }
    }
    tap0 = next_tap;
    c0 = next_c0;
  }
  if (row >= a.rows) return;
#pragma unroll
  for (int t = 0; t < kCols; t += kPair) {
    const Channels<kPair * 4> out(a, n0 + t * 16 + lc * 4 * kPair);
    float v[kPair * 4];
#pragma unroll
    for (int i = 0; i < kPair * 4; ++i) v[i] = acc[t + i / 4][i % 4];
    out.store(a, row, v);
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

// The registers of a wave hold 64 rows x 128 channels of sums, except where the rows come
// through registers as well, or integer sums are kept beside the float ones.
template <int kCols>
void conv_tile(const ProductArgs& a, bool direct, hipStream_t s) {
  constexpr int kFew = std::min(kCols, 4);  // channels
  if (a.k > 128) return direct ? launch_conv<4, kFew, 2, true, true>(a, s) : launch_conv<4, kFew, 2, false, true>(a, s);
  if (a.k <= 64)
    return direct ? launch_conv<4, kCols, 1, true, false>(a, s) : launch_conv<4, kCols, 1, false, false>(a, s);
  if (direct) return launch_conv<4, kCols, 2, true, false>(a, s);
  launch_conv<kCols == 8 ? 2 : 4, kCols, 2, false, false>(a, s);
}

template <int kCols, int kSteps, bool kWide>
void launch_conv_mid(const ProductArgs& a, hipStream_t s) {
  const int tn = (int)ceil_div(a.n, kCols * 16);
  launch("k_conv_mid", k_conv_mid<kCols, kSteps, kWide>, ceil_div(a.rows, kConvWaves * 16) * tn, kConvWaves * 64, s, a,
         tn);
}
template <int kCols>
void conv_mid(const ProductArgs& a, hipStream_t s) {
  if (a.k > 128) return launch_conv_mid<kCols, 2, true>(a, s);
  if (a.k > 64) return launch_conv_mid<kCols, 2, false>(a, s);
  launch_conv_mid<kCols, 1, false>(a, s);
}

template <int kCols>
void conv_few(const ProductArgs& a, hipStream_t s) {
  const int tn = (int)ceil_div(a.n, kCols * 16);
  launch("k_conv_few", k_conv_few<kCols>, ceil_div(a.rows, 16) * tn, kFewWaves * 64, s, a, tn);
}

// LDS of k_conv_resident; 0 where it does not take the call.
int resident_lds(const ProductArgs& a, int cols) {
  if (a.taps > 32 || a.k > 128 || a.n > 128) return 0;
  const int lds = a.taps * cols * (a.k > 64 ? 2 : 1) * 1024 + kConvWaves * 64 * (a.taps | 1) * 4;
  return lds <= 76 * 1024 ? lds : 0;  // two workgroups a CU, with 3 KiB of their own
}
template <int kCols>
void conv_resident(const ProductArgs& a, hipStream_t s) {
  const i64 blocks = ceil_div(a.rows, kConvWaves * 64);
  const size_t lds = resident_lds(a, kCols);
  auto run = [&](auto kernel) {
    // beyond 64 KiB the kernel has to be told
    if (lds > 60 * 1024) hip_check(hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                                  76 * 1024), "hipFuncSetAttribute");
    launch_lds("k_conv_resident", kernel, blocks, kConvWaves * 64, lds, s, a);
  };
  if (a.k > 64) run(k_conv_resident<kCols, 2>);
  else run(k_conv_resident<kCols, 1>);
}

// Calls f<kCols> for the channels of a tile.
template <typename F>
void with_cols(int n, F&& f) {
  using std::integral_constant;
  if (n <= 16) return f(integral_constant<int, 1>());
  if (n <= 32) return f(integral_constant<int, 2>());
  if (n <= 64) return f(integral_constant<int, 4>());
  f(integral_constant<int, 8>());
}

}  // namespace

// The variant. Timed over 27-tap maps of shells, bf16 out, in us a call:
//   rows    channels     tile  middle  few
//   116k    128 -> 128     69     164
//   116k    64 -> 64       39      47
//   65k     96 -> 96       55      85
//   65k     64 -> 64       33      27
//   37k     60 -> 60       45      24
//   22k     100 -> 96      63      34  100
//   5.5k    60 -> 96               19   23
//   2.7k    60 -> 60               19   12
//   65k     256 -> 256    310     372 1124
//   22k     256 -> 256   *155     144  390
//   8.6k    256 -> 256     82     *95  160
//   8.6k    512 -> 512    270     296  556
// and over 8-tap maps onto refined (up) and halved (down) grids:
//   108k up    64 -> 64     15     17    93
//   69k up     64 -> 64     14     14    58
//   69k up   128 -> 128     21     35   210
//   69k up   256 -> 128     64     74   330
//   22k up   128 -> 128     19     14    67
//   25k up     60 -> 60     12    9.2    29
//   8.4k up    64 -> 64     13    7.1    11
//   82k down   64 -> 64     17     17    76
//   36k down  64 -> 128    *20     16    68
//   36k down   64 -> 64     15     10    35
//   8.9k down 64 -> 128     20    8.3    19
//   2.4k down 64 -> 128     20    7.1  *8.2
// The rule takes the fastest, but the starred where there is one: 8 to 29% over the fastest.
// A tile of 256 rows reads its weights for four times the rows and skips more, and needs
// about one workgroup a CU to be worth it; where it has 64 channels or fewer to share a row
// among, more. Taps split over waves win while the rows leave CUs idle. Of the tiles, those
// with the weights of all taps in LDS are faster where rows would come through registers
// anyway (52 -> 45 onto 108k refined voxels 16 us for 21, 60 -> 60 onto 522k 46 for 72, from 110k to
// half the resolution 28 for 45, 27 taps 12 -> 12 40 for 51), and slower on most aligned ones (64 -> 64
// to half the resolution 26 for 20, 27 taps 16 -> 16 31 for 29; 32 -> 16 onto 522k 21 for 27).
void conv_i8(const ProductArgs& a, hipStream_t s) {
  const i64 cus = device_cu_count();
  auto tiles = [&](int rows, int cols) { return ceil_div(a.rows, rows) * ceil_div(a.n, cols); };
  // the offsets of a gather straight into LDS are 31 bits
  const bool direct = (((uintptr_t)a.x | (uintptr_t)a.x_stride | (uintptr_t)a.w | (uintptr_t)a.k) & 15) == 0 &&
                      a.n_src * a.x_stride + a.k < (1ll << 31);
  if (2 * tiles(256, 128) >= (a.n > 64 ? cus : 3 * cus))
    return with_cols(a.n, [&](auto c) {
      if (!direct && resident_lds(a, decltype(c)::value)) conv_resident<decltype(c)::value>(a, s);
      else conv_tile<decltype(c)::value>(a, direct, s);
    });
  if (tiles(64, 64) >= cus / 2) return with_cols(a.n, [&](auto c) { conv_mid<std::min(decltype(c)::value, 4)>(a, s); });
  if (tiles(16, 64) >= cus) return conv_few<4>(a, s);
  if (tiles(16, 32) >= cus) return conv_few<2>(a, s);
  conv_few<1>(a, s);
}

}  // namespace tc
