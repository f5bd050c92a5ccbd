// Rotary positions: pair i of every head of a row is turned by the angle p f[i], p the row's coordinate
// along the pair's axis.
//
//   (x1, x2) -> (x1 cos - x2 sin, x1 sin + x2 cos)
//
// The inverse, by the opposite angle, is also the gradient. Coordinates are any 32-bit integers, so an angle can
// be 2^31 radians: it is reduced in 64 bits, in turns, where subtracting whole turns is exact. Memory bounds
// it: a workgroup puts the sines of its rows into LDS once, for all heads, while its rows are under way.
#include "rows.hpp"

namespace tc {

namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;                        // a thread's units of work
constexpr int kMaxUnits = kThreads * kUnits;     // a workgroup's
constexpr int kTableBytes = 16 << 10;            // of sines and cosines in a workgroup

// A quotient by a number below 2^16 of one below 2^16.
struct Divider {
  uint32_t by, magic;
  explicit Divider(uint32_t d) : by(d), magic(d == 1 ? 0 : (uint32_t)((0x100000000ull + d - 1) / d)) {}
  // n (magic d - 2^32) / 2^32 < n d / 2^32 < 1 is all that the rounding up of magic adds to n
  __device__ __forceinline__ uint32_t divide(uint32_t n) const { return by == 1 ? n : __umulhi(n, magic); }
};

// cos and sin of p * f radians.
__device__ __forceinline__ float2 turn_of(int p, float f) {
  constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;  // 1 / (2 pi) as a sum
  const double x = p, hi = (double)f * kHi, lo = fma((double)f, kHi, -hi) + (double)f * kLo;
  const double whole = x * hi;
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

struct Plan {
  i64 rows_each;    // rows of a workgroup
  int heads_each;   // heads of a workgroup
  int head_groups;
  int units;        // of a head's pairs, V pairs each
  Divider by_units, by_heads;
};

// A unit is V pairs: two vectors of 16 bytes, half a head apart or (kNeighbours) side by side. The last
// unit of a head may have fewer, which go one by one.
template <typename T, bool kNeighbours>
__global__ void __launch_bounds__(kThreads) k_rotary(RotaryArgs a, Plan plan) {
  constexpr int V = 16 / sizeof(T);
  extern __shared__ float2 s_turn[];  // [rows][pairs]
  const i64 row0 = blockIdx.x / plan.head_groups * plan.rows_each;
  const int head0 = blockIdx.x % plan.head_groups * plan.heads_each;
  const int rows = (int)min(plan.rows_each, a.rows - row0), heads = min(plan.heads_each, a.heads - head0);
  const int units = rows * plan.heads_each * plan.units;
  const int pairs = a.pairs;

  T v[kUnits][2 * V];
  i64 to[kUnits];
  int count[kUnits], turn[kUnits], first[kUnits];  // pairs of the unit (0: none), its place in s_turn, its first pair
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int unit = threadIdx.x + i * kThreads;
    count[i] = 0;
    if (unit >= units) continue;
    const int at = plan.by_units.divide(unit), r = plan.by_heads.divide(at), h = at - r * plan.heads_each;
    if (h >= heads) continue;
    first[i] = (unit - at * plan.units) * V;
    count[i] = min(V, pairs - first[i]);
    turn[i] = r * pairs + first[i];
    const T* x = static_cast<const T*>(a.x) + (row0 + r) * a.x_row + (i64)(head0 + h) * a.x_head;
    to[i] = (row0 + r) * a.out_row + (i64)(head0 + h) * a.out_head;
    if (count[i] == V) {
      __builtin_memcpy(v[i], x + (kNeighbours ? 2 * first[i] : first[i]), 16);
      __builtin_memcpy(v[i] + V, x + (kNeighbours ? 2 * first[i] + V : pairs + first[i]), 16);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (e >= count[i]) continue;
        v[i][kNeighbours ? 2 * e : e] = x[kNeighbours ? 2 * (first[i] + e) : first[i] + e];
        v[i][kNeighbours ? 2 * e + 1 : V + e] = x[kNeighbours ? 2 * (first[i] + e) + 1 : pairs + first[i] + e];
      }
    }
  }
  for (int i = threadIdx.x; i < rows * pairs; i += kThreads) {
    const int r = i / pairs, p = i - r * pairs;
    const int axis = (p >= a.ends[0]) + (p >= a.ends[1]) + (p >= a.ends[2]);
    const float2 t = turn_of(a.positions[(row0 + r) * a.position_row + axis], a.freqs[p]);
    s_turn[i] = {t.x, a.inverse ? -t.y : t.y};
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    if (!count[i]) continue;
    T* out = static_cast<T*>(a.out) + to[i];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if (e >= count[i]) continue;
      const float2 t = s_turn[turn[i] + e];
      T &p1 = v[i][kNeighbours ? 2 * e : e], &p2 = v[i][kNeighbours ? 2 * e + 1 : V + e];
      const float x1 = to_f32(p1), x2 = to_f32(p2);
      p1 = from_f32<T>(fmaf(x1, t.x, -(x2 * t.y)));
      p2 = from_f32<T>(fmaf(x1, t.y, x2 * t.x));
    }
    if (count[i] == V) {
      __builtin_memcpy(out + (kNeighbours ? 2 * first[i] : first[i]), v[i], 16);
      __builtin_memcpy(out + (kNeighbours ? 2 * first[i] + V : pairs + first[i]), v[i] + V, 16);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (e >= count[i]) continue;
        out[kNeighbours ? 2 * (first[i] + e) : first[i] + e] = v[i][kNeighbours ? 2 * e : e];
        out[kNeighbours ? 2 * (first[i] + e) + 1 : pairs + first[i] + e] = v[i][kNeighbours ? 2 * e + 1 : V + e];
      }
    }
  }
  // what is not turned, into another tensor
  const int rest = a.dim - 2 * pairs;
  if (rest == 0 || a.in_place) return;
  for (int i = threadIdx.x; i < rows * heads * rest; i += kThreads) {
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
    constexpr int V = 16 / sizeof(T);
    const int units = std::max<int>(1, (int)ceil_div(a.pairs, V));
    // all heads of a row in one workgroup share its sines; rows up to the units of a thread, and to the table's size
    const int heads_each = std::min(a.heads, std::max(1, kMaxUnits / units));
    const i64 rows_each = std::max<i64>(1, std::min<i64>({kMaxUnits / ((i64)units * heads_each),
                                                          kTableBytes / ((i64)sizeof(float2) * std::max(a.pairs, 1)), a.rows}));
    const int head_groups = (int)ceil_div(a.heads, heads_each);
    const Plan plan{rows_each, heads_each, head_groups, units, Divider((uint32_t)units), Divider((uint32_t)heads_each)};
    const size_t lds = sizeof(float2) * (size_t)rows_each * (size_t)a.pairs;
    launch_lds("k_rotary", a.interleaved ? k_rotary<T, true> : k_rotary<T, false>, ceil_div(a.rows, rows_each) * head_groups,
               kThreads, lds, s, a, plan);
  });
}

}  // namespace tc
