// 8-bit rows and weights as the matrix instructions take them: loads, tiles and their order in LDS, stores of results
// (product.hip, conv.hip); packed 4-bit ones share the loads, tiles and waits (mx4.hpp, product_mx4.hip).
#pragma once

#include "rows.hpp"

namespace tc {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));

// CNT consecutive output channels of one row from n on, rounded to T. Rows on 16-byte
// boundaries (`wide`) are stored past the caches, which keeps the inputs there
// (16384 x 4096 -> 4096: 230 for 260 us, 124800 x 256 -> 768: 65 for 106 us, in one run).
template <typename T, int CNT>
__device__ __forceinline__ void store_run(const ProductArgs& a, i64 row, int n, const float v[CNT], bool wide) {
  T* out = static_cast<T*>(a.out) + row * a.out_stride + n;
  T r[CNT];
#pragma unroll
  for (int i = 0; i < CNT; ++i) r[i] = from_f32<T>(v[i]);
  if (n + CNT <= a.n) {
    if (wide && sizeof(r) >= 16) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(r) / 16; ++i)
        __builtin_nontemporal_store(reinterpret_cast<const v4i*>(r)[i], reinterpret_cast<v4i*>(out) + i);
    } else {
      __builtin_memcpy(out, r, sizeof(r));
    }
  } else {
#pragma unroll
    for (int i = 0; i < CNT; ++i)
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
  } else if (c == 0 && k >= 8) {
    unsigned long long lo, hi;
    __builtin_memcpy(&lo, row, 8);
    __builtin_memcpy(&hi, row + k - 8, 8);
    v[0] = lo;
    v[1] = hi >> 1 >> (127 - 8 * k & 63);  // its last k - 8 bytes: 0 for k = 8
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

// One step of products: 16 rows of w by 16 rows of x over 64 input channels. A lane
// holds four rows of w (4 (lane / 16) on) of x's row lane % 16.
__device__ __forceinline__ v4i product_16(v4i w, v4i x, v4i sum) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(w, x, sum, 0, 0, 0);
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

// This wave's LDS reads and writes are done.
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// Every wave has its part in LDS, and has read what it had to.
__device__ __forceinline__ void meet() {
  wait_lds();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

}  // namespace tc
