// Rows held in registers over their reductions, as the norms take them (norm.hip, layer_norm.hip).
#pragma once

#include <type_traits>

#include "rows.hpp"

namespace tc {

namespace {

constexpr int kNormThreads = 256;

__device__ __forceinline__ float weight_at(const void* w, int dt, int c) {
  if (!w) return 1.0f;
  if (dt == TC_F32) return static_cast<const float*>(w)[c];
  if (dt == TC_F16) return to_f32(static_cast<const f16*>(w)[c]);
  return to_f32(static_cast<const bf16*>(w)[c]);
}

// 16 bytes of a row, from any address.
template <typename T>
struct Vec {
  static constexpr int kN = 16 / sizeof(T);
  T v[kN];
  __device__ __forceinline__ void load(const T* p) { __builtin_memcpy(v, p, 16); }
  __device__ __forceinline__ void store(T* p) const { __builtin_memcpy(p, v, 16); }
};

// A group of L threads holds one row, N vectors a thread (vector g + j L for thread
// g). A row that is no whole number of vectors has its last one moved back to end
// the row: `skip` of its elements belong to the vector before as well, are written
// twice with the same value, and are left out of the sums.
template <typename T, int L, int N>
struct RowPlace {
  int c[N];     // first element, -1: none
  int skip[N];
  bool ragged;
  __device__ __forceinline__ RowPlace(int channels) {
    constexpr int V = Vec<T>::kN;
    ragged = channels % V != 0;
    const int g = threadIdx.x % L;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int at = (g + j * L) * V, from = min(at, channels - V);
      c[j] = at < channels ? from : -1;
      skip[j] = at - from;
    }
  }
};

// A row's vectors, loaded where the place has any.
template <typename T, int L, int N>
__device__ __forceinline__ void load_row(Vec<T> (&v)[N], const RowPlace<T, L, N>& at, const void* base, i64 offset) {
#pragma unroll
  for (int j = 0; j < N; ++j)
    if (at.c[j] >= 0) v[j].load(static_cast<const T*>(base) + offset + at.c[j]);
}

// The weights of a place's elements (T's type, or 32 bits; `none` without any; 0 where there is no element).
template <typename T, int L, int N>
__device__ __forceinline__ void load_weights(float (&w)[N][Vec<T>::kN], const RowPlace<T, L, N>& at, const void* p,
                                             int dtype, float none = 1.0f) {
  constexpr int V = Vec<T>::kN;
  Vec<T> raw[N];
  float wide[N][V];
  if (p && dtype == TC_F32) {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (at.c[j] >= 0) __builtin_memcpy(wide[j], static_cast<const float*>(p) + at.c[j], V * 4);
  } else if (p) {
    load_row<T, L, N>(raw, at, p, 0);
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) wide[j][e] = to_f32(raw[j].v[e]);
  }
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int e = 0; e < V; ++e) w[j][e] = at.c[j] < 0 ? 0.0f : p ? wide[j][e] : none;
}

// Sums over the L threads of a group, L a power of two up to a wave, or a workgroup of
// four waves. Every thread gets the sum, in an order that only L decides.
template <typename V>
struct GroupScratch {
  V part[2][4], top[2][4];
};

template <int L, typename V>
__device__ __forceinline__ V group_sum(V v, GroupScratch<V>& s, int turn) {
  v = lanes_reduce<(L < kWave ? L : kWave)>(v, [](V a, V b) { return a + b; });
  if constexpr (L > kWave) {
    if ((threadIdx.x & (kWave - 1)) == 0) s.part[turn][threadIdx.x / kWave] = v;
    __syncthreads();
    v = (s.part[turn][0] + s.part[turn][1]) + (s.part[turn][2] + s.part[turn][3]);
  }
  return v;
}

// s = root * 2^shift: shift is 0 but for rows far from one (above), where it takes the power of
// two, so that s need not fit 32 bits (rows below 2^-126 with eps = 0).
struct InverseRoot {
  float root;
  int shift;
  __device__ __forceinline__ float times(float h) const { return ldexpf(h, shift) * root; }
  __device__ __forceinline__ float value() const { return ldexpf(root, shift); }
};
// Whether the mean of the squares and eps, in 32 bits, is one of a far row: squares below the normal
// range are off by 2^-150, nothing next to 2^-100. Those of f16 are 2^-48 to 2^32, or zero.
template <typename T>
__device__ __forceinline__ bool far(float mean) {
  return !std::is_same<T, f16>::value && !(mean >= 0x1p-100f && mean < INFINITY);
}
// From that mean in 64 bits: the root of a number in [1/2, 2).
__device__ __forceinline__ InverseRoot far_root(double mean) {
  const int half = __builtin_amdgcn_frexp_exp(mean) >> 1;  // 0 for 0, infinity and NaN
  return {1.0f / sqrtf((float)ldexp(mean, -2 * half)), -half};
}

// Calls f<L, N> with the place of rows of `vectors` 16-byte vectors: the fewest
// lanes that hold the row, up to four vectors a lane in one wave, then a workgroup.
// False where a workgroup's registers do not hold the row.
template <typename F>
bool with_place(i64 vectors, F&& f) {
  using std::integral_constant;
  auto go = [&](auto l, auto n) { f(l, n); return true; };
#define TC_PLACE(L, N) go(integral_constant<int, L>(), integral_constant<int, N>())
  if (vectors <= 1) return TC_PLACE(1, 1);
  if (vectors <= 2) return TC_PLACE(2, 1);
  if (vectors <= 4) return TC_PLACE(4, 1);
  if (vectors <= 8) return TC_PLACE(8, 1);
  if (vectors <= 16) return TC_PLACE(16, 1);
  if (vectors <= 32) return TC_PLACE(32, 1);
  if (vectors <= 64) return TC_PLACE(64, 1);
  if (vectors <= 128) return TC_PLACE(64, 2);
  if (vectors <= 256) return TC_PLACE(256, 1);
  if (vectors <= 512) return TC_PLACE(256, 2);
  if (vectors <= 1024) return TC_PLACE(256, 4);
  if (vectors <= 2048) return TC_PLACE(256, 8);
#undef TC_PLACE
  return false;
}

}  // namespace

}  // namespace tc
