// Rotary positions: pair i of every head of a row is turned by the angle p f[i], p the row's coordinate
// along the pair's axis.
//
//   (x1, x2) -> (x1 cos - x2 sin, x1 sin + x2 cos)
//
// The inverse, by the opposite angle, is also the gradient. Coordinates are any 32-bit integers and frequencies any finite
// ones, so an angle can be 2^159 radians: it is reduced in 64 bits, in turns, where subtracting whole turns is exact. Memory
// bounds it: a workgroup puts the sines of its rows into LDS once, for all heads, while its rows are under way.
#include <type_traits>

#include "rows.hpp"

namespace tc {

namespace {

constexpr int kMostThreads = 512;
constexpr int kTableBytes = 32 << 10;  // of sines and cosines in a workgroup

// The first 224 bits of 1 / (2 pi).
__constant__ const uint32_t kTurnBits[7] = {0x28be60db, 0x9391054a, 0x7f09d5f4, 0x7d4d3770, 0x36d8a566, 0x4f10e410, 0x7f9458ea};

// f radians in turns, less whole ones, as hi + lo to 2^-64, for |f| from 2^40 on, by the method of Payne and Hanek: f is
// m 2^e, and of 1 / (2 pi) the bits before number e make whole turns. NaN for what is not finite.
__device__ __forceinline__ void turns_far(float f, double& hi, double& lo) {
  const uint32_t bits = __float_as_uint(f), m = (bits & 0x7fffff) | 0x800000;
  const int e = min((int)(bits >> 23 & 255) - 150, 104), last = (e + 31) >> 5;  // 17 to 104; the word that holds bit e, or the next
  auto word = [&](int i) { return __builtin_amdgcn_alignbit(kTurnBits[last - 1 + i], kTurnBits[last + i], 32 * last - e); };
  const uint64_t turns = ((uint64_t)m * word(2) >> 32) + (uint64_t)m * word(1) + ((uint64_t)(m * word(0)) << 32);
  const float sign = copysignf(1.0f, f) + (f - f);
  hi = (double)(int32_t)(turns >> 32) * 0x1p-32 * sign;
  lo = (double)(uint32_t)turns * 0x1p-64 * sign;
}

// cos and sin of p * f radians. The compiler may not fuse operations by itself here: `whole` less its whole turns has to
// be of the rounded product, whose rounding is added back once (fused, it came in twice: angles near 2^31 radians were
// off by 1.8e-7, of 2^51 radians by 0.1).
__device__ __forceinline__ float2 turn_of(int p, float f) {
#pragma clang fp contract(off)
  constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;  // 1 / (2 pi) as a sum, to 2^-110
  double hi = (double)f * kHi, lo = fma((double)f, kLo, fma((double)f, kHi, -hi));  // f in turns
  if (__builtin_expect(fabsf(f) >= 0x1p40f, 0)) turns_far(f, hi, lo);
  const double x = p, whole = x * hi;
  double t = (whole - rint(whole)) + fma(x, lo, fma(x, hi, -whole));  // turns
  t -= rint(t);
  const double quarter = rint(4.0 * t);
  const float a = (float)(fma(-0.25, quarter, t) * 6.283185307179586), s = a * a;  // within pi / 4
  // Taylor's series; what is left out is below 2^-29
  const float sin = fmaf(a * s, fmaf(s, fmaf(s, fmaf(s, 1.0f / 362880, -1.0f / 5040), 1.0f / 120), -1.0f / 6), a);
  const float cos = fmaf(s, fmaf(s, fmaf(s, fmaf(s, fmaf(s, -1.0f / 3628800, 1.0f / 40320), -1.0f / 720), 1.0f / 24), -0.5f), 1.0f);
  const int q = (int)quarter;  // -2 to 2; 0 for what is no number
  const float c = q & 1 ? sin : cos, d = q & 1 ? cos : sin;
  return {(q + 1) & 2 ? -c : c, q & 2 ? -d : d};
}

// A unit of work is a vector of 16 bytes of firsts of pairs and one of seconds, half the turned channels apart, or two
// vectors of pairs that are side by side (kNeighbours), or one (kWide). The last unit of a head may have fewer pairs,
// which go one by one. A thread has the same unit of kDepth rows, all asked for before the sines are made.
//
// kWide: outputs on 16-byte boundaries, of which a wave has whole lines, go past the caches: 60000 x 8 x 128 bf16
// 42 for 53 us, neighbours 38 for 56; 124800 x 16 x 64, neighbours, 110 for 120 (4.7 TB/s). Halves of 64 bytes
// (124800 x 16 x 64) would take 130 for 115 that way.
template <typename T, bool kNeighbours, bool kWide>
struct UnitOf {
  static constexpr int kVectors = kNeighbours && kWide ? 1 : 2;
  static constexpr int kPairs = 16 / sizeof(T) * kVectors / 2, kDepth = 8 / kVectors;
};

struct Plan {
  int units;        // of a head's pairs
  int heads_each;   // heads of a workgroup
  int head_groups;
  int rows_across;  // rows that the threads of a workgroup are side by side on
  i64 rows_each;    // rows of a workgroup, at most a thread's times rows_across
  int pitch;        // pairs of a row of the table, an even number
  int row_step, pair_step;  // from an entry of the table to the thread's next
};

template <typename T, bool kNeighbours, bool kWide>
__global__ void __launch_bounds__(kMostThreads) k_rotary(RotaryArgs a, Plan plan) {
  using U = UnitOf<T, kNeighbours, kWide>;
  constexpr int V = 16 / sizeof(T), P = U::kPairs, kDepth = U::kDepth, kVectors = U::kVectors;
  extern __shared__ float2 s_turn[];  // [rows][pitch]
  const i64 row0 = blockIdx.x / plan.head_groups * plan.rows_each;
  const int head0 = blockIdx.x % plan.head_groups * plan.heads_each;
  const int rows = (int)min(plan.rows_each, a.rows - row0), heads = min(plan.heads_each, a.heads - head0);
  const int pairs = a.pairs, tid = threadIdx.x;
  const int at = tid / plan.units, r0 = at / plan.heads_each, h = at - r0 * plan.heads_each;
  const int first = (tid - at * plan.units) * P;
  const int count = r0 < plan.rows_across && h < heads ? min(P, pairs - first) : 0;  // pairs of the unit, 0: none
  // channels of the first pair; a unit's vectors, and the pairs of one that has fewer, are side by side or `apart`
  const int c1 = kNeighbours ? 2 * first : first, apart = kNeighbours ? V : pairs;
  const T* x = static_cast<const T*>(a.x) + (row0 + r0) * a.x_row + (i64)(head0 + h) * a.x_head;
  T* out = static_cast<T*>(a.out) + (row0 + r0) * a.out_row + (i64)(head0 + h) * a.out_head;
  auto first_at = [&](int e) { return kNeighbours ? c1 + 2 * e : c1 + e; };
  auto second_at = [&](int e) { return kNeighbours ? c1 + 2 * e + 1 : c1 + pairs + e; };
  auto first_of = [](T (&v)[kVectors][V], int e) -> T& { return kNeighbours ? v[2 * e / V][2 * e % V] : v[0][e]; };
  auto second_of = [](T (&v)[kVectors][V], int e) -> T& { return kNeighbours ? v[2 * e / V][2 * e % V + 1] : v[kVectors - 1][e]; };

  T v[kDepth][kVectors][V];
#pragma unroll
  for (int i = 0; i < kDepth; ++i) {
    if (!count || r0 + i * plan.rows_across >= rows) continue;
    const T* from = x + i * plan.rows_across * a.x_row;
    if (count == P) {
#pragma unroll
      for (int k = 0; k < kVectors; ++k) __builtin_memcpy(v[i][k], from + c1 + k * apart, 16);
    } else {
#pragma unroll
      for (int e = 0; e < P; ++e)
        if (e < count) {
          first_of(v[i], e) = from[first_at(e)];
          second_of(v[i], e) = from[second_at(e)];
        }
    }
  }
  for (int r = tid / pairs, p = tid - r * pairs; r < rows;) {
    const int axis = (p >= a.ends[0]) + (p >= a.ends[1]) + (p >= a.ends[2]);
    const float f = a.freqs[p];
    const int at = a.positions[(row0 + r) * a.position_row + axis];
    float2* const to = s_turn + r * plan.pitch + p;
    // with a division for each entry, the branch for far frequencies cost 10% where the sines bound it (40000 x 2 x 256 bf16)
    r += plan.row_step;
    p += plan.pair_step;
    if (p >= pairs) {
      p -= pairs;
      ++r;
    }
    const float2 t = turn_of(at, f);
    *to = {t.x, a.inverse ? -t.y : t.y};
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kDepth; ++i) {
    const int r = r0 + i * plan.rows_across;
    if (!count || r >= rows) continue;
    T* to = out + i * plan.rows_across * a.out_row;
    float2 t[P];
    if (count == P) {
      __builtin_memcpy(t, __builtin_assume_aligned(s_turn + r * plan.pitch + first, 16), sizeof(t));
    } else {
#pragma unroll
      for (int e = 0; e < P; ++e) t[e] = e < count ? s_turn[r * plan.pitch + first + e] : float2{0.0f, 0.0f};
    }
#pragma unroll
    for (int e = 0; e < P; ++e) {
      T &p1 = first_of(v[i], e), &p2 = second_of(v[i], e);
      const float x1 = to_f32(p1), x2 = to_f32(p2);
      p1 = from_f32<T>(fmaf(x1, t[e].x, -(x2 * t[e].y)));
      p2 = from_f32<T>(fmaf(x1, t[e].y, x2 * t[e].x));
    }
    if (count == P) {
#pragma unroll
      for (int k = 0; k < kVectors; ++k) {
        typedef int v4i __attribute__((ext_vector_type(4)));
        if (kWide) __builtin_nontemporal_store(*reinterpret_cast<const v4i*>(v[i][k]), reinterpret_cast<v4i*>(to + c1 + k * apart));
        else __builtin_memcpy(to + c1 + k * apart, v[i][k], 16);
      }
    } else {
#pragma unroll
      for (int e = 0; e < P; ++e)
        if (e < count) {
          to[first_at(e)] = first_of(v[i], e);
          to[second_at(e)] = second_of(v[i], e);
        }
    }
  }
  // what is not turned, into another tensor, one by one: 60000 x 8 x 48 bf16 with 8 pairs 47 us, for 18 that its bytes take
  const int rest = a.dim - 2 * pairs;
  if (rest == 0 || a.in_place) return;
  for (int i = tid; i < rows * heads * rest; i += blockDim.x) {
    const int at = i / rest, r = at / heads, h = head0 + at - r * heads, c = 2 * pairs + i - at * rest;
    static_cast<T*>(a.out)[(row0 + r) * a.out_row + h * a.out_head + c] =
        static_cast<const T*>(a.x)[(row0 + r) * a.x_row + h * a.x_head + c];
  }
}

}  // namespace

void rotary(const RotaryArgs& a, hipStream_t s) {
  if (a.rows == 0 || a.heads == 0) return;
  with_dtype(a.dtype, [&](auto t) {
    using T = decltype(t);
    auto go = [&](auto neighbours, auto wide) {
      using U = UnitOf<T, decltype(neighbours)::value, decltype(wide)::value>;
      Plan p;
      p.units = (int)ceil_div(a.pairs, U::kPairs);  // at most kMostThreads: dim is at most 4096
      // all heads of a row in one workgroup, where they fit, share its sines
      p.heads_each = std::min(a.heads, kMostThreads / p.units);
      p.head_groups = (int)ceil_div(a.heads, p.heads_each);
      p.pitch = a.pairs + a.pairs % 2;
      // as many rows side by side as leave the fewest lanes of the waves idle
      const int across = p.heads_each * p.units;
      const i64 table_rows = std::max<i64>(1, kTableBytes / ((i64)sizeof(float2) * p.pitch));
      const i64 most = std::min<i64>({kMostThreads / across, a.rows, std::max<i64>(1, table_rows / U::kDepth)});
      p.rows_across = 1;
      auto waves = [&](int rows) { return (rows * across + kWave - 1) / kWave; };
      for (int r = 2; r <= most; ++r)
        if (r * waves(p.rows_across) >= p.rows_across * waves(r)) p.rows_across = r;
      // rows for every CU before depth
      const i64 depth = std::max<i64>(
          1, std::min<i64>({U::kDepth, table_rows / p.rows_across,
                            a.rows * p.head_groups / (p.rows_across * 2 * (i64)device_cu_count())}));
      p.rows_each = depth * p.rows_across;
      const int threads = waves(p.rows_across) * kWave;
      p.row_step = threads / a.pairs;
      p.pair_step = threads % a.pairs;
      launch_lds("k_rotary", k_rotary<T, decltype(neighbours)::value, decltype(wide)::value>,
                 ceil_div(a.rows, p.rows_each) * p.head_groups, threads,
                 sizeof(float2) * (size_t)p.rows_each * (size_t)p.pitch, s, a, p);
    };
    constexpr i64 kSize = sizeof(T);
    const bool aligned = aligned_16(a.out, (a.out_row | a.out_head) * kSize);
    if (a.interleaved) {
      // heads that follow each other, or that are whole lines themselves
      const i64 turned = 2 * a.pairs * kSize;
      const bool lines = turned % 128 == 0 || (2 * a.pairs == a.dim && (a.heads == 1 || a.out_head == a.dim));
      if (aligned && turned % 16 == 0 && turned / 16 <= kMostThreads && lines) go(std::true_type(), std::true_type());
      else go(std::true_type(), std::false_type());
    } else {
      if (aligned && a.pairs * kSize % 128 == 0) go(std::false_type(), std::true_type());
      else go(std::false_type(), std::false_type());
    }
  });
}

}  // namespace tc
