// Root-mean-square norm of feature rows with the residual's addition, its
// 8-bit form and its gradient.
//
//   h = round(x + r), s = 1 / sqrt(mean(h^2) + eps), out = round(h s w)
//
// h is rounded to the rows' type once and the norm is the norm of that rounded
// h, so the gradient taken from the stored h is the gradient of what was
// computed. The mean is a float sum of float squares; where that leaves 32 bits or nears the end of
// their range (rows from 1.8e19 on, or below 1e-15 with an eps as small), the squares are summed
// again in 64 bits: the norm of a finite row is finite. Memory bounds all of it: every kernel
// reads a row once, holds it in registers over its reductions and writes once.
#include "norm_rows.hpp"

namespace tc {

namespace {

// As group_sum, with the largest `top` beside the sum.
template <int L>
__device__ __forceinline__ void group_sum_max(float& v, double& top, GroupScratch<float>& sums,
                                              GroupScratch<double>& tops, int turn) {
  constexpr int W = L < kWave ? L : kWave;
  v = lanes_reduce<W>(v, [](float a, float b) { return a + b; });
  top = lanes_reduce<W>(top, [](double a, double b) { return fmax(a, b); });
  if constexpr (L > kWave) {
    if ((threadIdx.x & (kWave - 1)) == 0) {
      sums.part[turn][threadIdx.x / kWave] = v;
      tops.top[turn][threadIdx.x / kWave] = top;
    }
    __syncthreads();
    v = (sums.part[turn][0] + sums.part[turn][1]) + (sums.part[turn][2] + sums.part[turn][3]);
    top = fmax(fmax(tops.top[turn][0], tops.top[turn][1]), fmax(tops.top[turn][2], tops.top[turn][3]));
  }
}

// |h w| in 64 bits, where it is exact; infinite for an infinity or NaN.
__device__ __forceinline__ double magnitude(double p) {
  p = fabs(p);
  return p < INFINITY ? p : INFINITY;
}

// The factor of the row's 8-bit values, and its scale.
__device__ __forceinline__ double row_factor(double top, const InverseRoot& s, float& scale) {
  const bool finite = top < INFINITY, some = top > 0.0;
  scale = finite ? (some ? (float)ldexp(top * s.root * (1.0 / 127.0), s.shift) : 0.0f) : NAN;
  return finite && some ? 127.0 / top : 0.0;
}

// p * factor, rounded to 64 bits, then to the nearest integer, ties to even: adding
// 1.5 * 2^52 leaves it in the low bits. One fused operation would skip the first rounding.
__device__ __forceinline__ int8_t nearest_i8(double p, double factor) {
#pragma clang fp contract(off)
  const double q = p * factor;
  return (int8_t)__double2loint(q + 6755399441055744.0);
}

// The row stays in registers between the reductions and the outputs. h is stored
// only after a reduction over the row, when all of x and r is read: it may go over either.
// Memory bounds it: 16384 x 4096 f16 91 us (5.9 TB/s), f32 186 (5.8), 124800 x 128 bf16 21, f32 42,
// in 8 bits 124800 x 64 bf16 13 us (4.2 TB/s; products in 32 bits instead of 64 changed nothing),
// one row of 1024 2.9 us.
//
// N = 4: held to the 168 registers of three waves a SIMD (the 8-bit form of 16-bit rows would take a few
// more: 4096 x 6000 f16 96 us for 92).
template <typename T, int L, int N, bool kI8>
__global__ void __launch_bounds__(kNormThreads, N == 4 ? 3 : 1) k_rms_norm(NormArgs a) {
  constexpr int V = Vec<T>::kN;
  __shared__ GroupScratch<float> s_red;
  __shared__ GroupScratch<double> s_far;
  const RowPlace<T, L, N> at(a.channels);
  const i64 step = (i64)gridDim.x * (kNormThreads / L);
  i64 row = (i64)blockIdx.x * (kNormThreads / L) + threadIdx.x / L;
  Vec<T> x[N], r[N];  // of the next row, asked for before the row at hand is reduced
  auto ask = [&](i64 row) {
    if (row >= a.rows) return;
    load_row<T, L, N>(x, at, a.x, row * a.x_stride);
    if (a.residual) load_row<T, L, N>(r, at, a.residual, row * a.residual_stride);
  };
  ask(row);
  float w[N][V];
  load_weights<T, L, N>(w, at, a.weight, a.weight_dtype);
  int turn = 0;
  for (; row < a.rows; row += step, turn ^= 1) {
    Vec<T> h[N];
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e)
        h[j].v[e] = a.residual ? from_f32<T>(to_f32(x[j].v[e]) + to_f32(r[j].v[e])) : x[j].v[e];
    ask(row + step);
    float ss = 0.0f;
    double top = 0.0;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (at.c[j] < 0) continue;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float f = to_f32(h[j].v[e]);
        if (!at.ragged || e >= at.skip[j]) ss += f * f;
        if constexpr (kI8) top = fmax(top, magnitude((double)f * (double)w[j][e]));
      }
    }
    if constexpr (kI8) group_sum_max<L>(ss, top, s_red, s_far, turn);
    else ss = group_sum<L>(ss, s_red, turn);
    const float mean = ss / (float)a.channels + a.eps;
    InverseRoot s{1.0f / sqrtf(mean), 0};
    const bool again = far<T>(mean);  // the same for the whole row
    if (again) {
      double sum = 0.0;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        if (at.c[j] < 0) continue;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const double f = to_f32(h[j].v[e]);
          if (!at.ragged || e >= at.skip[j]) sum += f * f;
        }
      }
      s = far_root(group_sum<L>(sum, s_far, turn) / a.channels + a.eps);
    }
    const bool first = threadIdx.x % L == 0;
    if (a.sum) {
      T* sum = static_cast<T*>(a.sum) + row * a.channels;
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (at.c[j] >= 0) h[j].store(sum + at.c[j]);
    }
    if constexpr (kI8) {
      float scale;
      const double to_q = row_factor(top, s, scale);
      if (first) a.scale[row] = scale;
      int8_t* q = a.q + row * a.channels;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        if (at.c[j] < 0) continue;
        int8_t b[V];
#pragma unroll
        for (int e = 0; e < V; ++e)
          b[e] = to_q > 0.0 ? nearest_i8((double)to_f32(h[j].v[e]) * (double)w[j][e], to_q) : 0;
        __builtin_memcpy(q + at.c[j], b, V);
      }
    } else {
      if (a.rstd && first) a.rstd[row] = s.value();
      T* out = static_cast<T*>(a.out) + row * a.channels;
      auto write = [&](auto unit) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
          if (at.c[j] < 0) continue;
          Vec<T> o;
#pragma unroll
          for (int e = 0; e < V; ++e) o.v[e] = from_f32<T>(unit(to_f32(h[j].v[e])) * w[j][e]);
          o.store(out + at.c[j]);
        }
      };
      if (again) write([&](float f) { return s.times(f); });
      else write([&](float f) { return f * s.root; });
    }
  }
}

// dx = s g - u (s mean(g u)) + dh with g = dy w and the unit row u = h s, and this workgroup's
// part of dw = sum over rows of dy u: each thread adds up its channels over its rows in
// registers, the workgroup's groups are joined once at the end. Neither a power of s nor a
// product with h is formed: those leave 32 bits (rows of 1e14, s^3 = 1e-42) where u does not.
// 16384 x 4096 f16 113 us (4.8 TB/s) and 5 for the sum of the parts, f32 212 (5.1) and 6, 124800 x 128
// bf16 21 us and 5. N = 8 takes more than 256 registers, one wave a SIMD: 8192 x 8192 f32 211 us (5.1 TB/s)
// all the same.
template <typename T, int L, int N, bool kWeight>
__global__ void __launch_bounds__(kNormThreads) k_rms_norm_grad(NormGradArgs a) {
  constexpr int V = Vec<T>::kN;
  __shared__ GroupScratch<float> s_red;
  const RowPlace<T, L, N> at(a.channels);
  const i64 step = (i64)gridDim.x * (kNormThreads / L);
  i64 row = (i64)blockIdx.x * (kNormThreads / L) + threadIdx.x / L;
  Vec<T> next_dy[N], next_h[N], next_dh[N];  // of the next row
  float next_rstd = 0.0f;
  auto ask = [&](i64 row) {
    if (row >= a.rows) return;
    load_row<T, L, N>(next_dy, at, a.grad_out, row * a.grad_out_stride);
    load_row<T, L, N>(next_h, at, a.h, row * a.h_stride);
    if (a.grad_sum) load_row<T, L, N>(next_dh, at, a.grad_sum, row * a.grad_sum_stride);
    next_rstd = a.rstd[row];
  };
  ask(row);
  float w[N][V], dw[N][V];
  load_weights<T, L, N>(w, at, a.weight, a.weight_dtype);
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int e = 0; e < V; ++e) dw[j][e] = 0.0f;
  int turn = 0;
  for (; row < a.rows; row += step, turn ^= 1) {
    Vec<T> dy[N], h[N], dh[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      dy[j] = next_dy[j];
      h[j] = next_h[j];
      dh[j] = next_dh[j];
    }
    const float rstd = next_rstd;
    ask(row + step);
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (at.c[j] < 0) continue;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float y = to_f32(dy[j].v[e]), u = to_f32(h[j].v[e]) * rstd;
        if (!at.ragged || e >= at.skip[j]) dot += y * w[j][e] * u;
        if constexpr (kWeight) dw[j][e] += y * u;
      }
    }
    dot = group_sum<L>(dot, s_red, turn);
    if (!a.grad_x) continue;
    const float along = rstd * (dot / (float)a.channels);
    T* dx = static_cast<T*>(a.grad_x) + row * a.channels;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (at.c[j] < 0) continue;
      Vec<T> o;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float v = rstd * (to_f32(dy[j].v[e]) * w[j][e]) - to_f32(h[j].v[e]) * rstd * along;
        o.v[e] = from_f32<T>(a.grad_sum ? v + to_f32(dh[j].v[e]) : v);
      }
      o.store(dx + at.c[j]);
    }
  }
  if constexpr (kWeight) {
    float* part = a.partial + (i64)blockIdx.x * a.channels;
    if constexpr (L > kWave) {
#pragma unroll
      for (int j = 0; j < N; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (at.c[j] >= 0) part[at.c[j] + e] = dw[j][e];
    } else {
      constexpr int kWaves = kNormThreads / kWave;
      __shared__ float s_dw[kWaves][L * N * V];
      const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
#pragma unroll
      for (int j = 0; j < N; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float v = dw[j][e];
#pragma unroll
          for (int d = L; d < kWave; d <<= 1) v += __shfl_xor(v, d, kWave);
          if (lane < L) s_dw[wave][(j * L + lane) * V + e] = v;
        }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < N; ++j) {
        // slot i of the row's vectors, as this thread's RowPlace has it where the thread is below L
        for (int i = threadIdx.x; i < L * V; i += kNormThreads) {
          const int vec = j * L + i / V, first = vec * V;
          if (first >= a.channels) continue;
          float v = s_dw[0][j * L * V + i];
#pragma unroll
          for (int k = 1; k < kWaves; ++k) v += s_dw[k][j * L * V + i];
          part[min(first, a.channels - V) + i % V] = v;
        }
      }
    }
  }
}

// Rows of fewer channels than a vector has (L = 1: one thread a row), or of more
// than a workgroup's registers hold (L = a workgroup, the row read twice), element by
// element: such rows are rare, and loads of 2 or 4 bytes a lane bound them. 2048 x 20000 bf16 142 us
// for the 66 that its bytes take, in 8 bits 152 for 58, 2048 x 10000 f32 91 for 66, 124800 x 3 f32 5.
template <typename T, int L, bool kI8>
__global__ void __launch_bounds__(kNormThreads) k_rms_norm_any(NormArgs a) {
  __shared__ GroupScratch<float> s_red;
  __shared__ GroupScratch<double> s_far;
  const int g = threadIdx.x % L;
  int turn = 0;
  for (i64 row = (i64)blockIdx.x * (kNormThreads / L) + threadIdx.x / L; row < a.rows;
       row += (i64)gridDim.x * (kNormThreads / L), turn ^= 1) {
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    const T* r = a.residual ? static_cast<const T*>(a.residual) + row * a.residual_stride : nullptr;
    T* sum = a.sum ? static_cast<T*>(a.sum) + row * a.channels : nullptr;
    float ss = 0.0f;
    double top = 0.0;
    for (int c = g; c < a.channels; c += L) {
      const T h = r ? from_f32<T>(to_f32(x[c]) + to_f32(r[c])) : x[c];
      if (sum) sum[c] = h;
      const float f = to_f32(h);
      ss += f * f;
      if constexpr (kI8) top = fmax(top, magnitude((double)f * (double)weight_at(a.weight, a.weight_dtype, c)));
    }
    if constexpr (kI8) group_sum_max<L>(ss, top, s_red, s_far, turn);
    else ss = group_sum<L>(ss, s_red, turn);
    // h where this thread stored it, else x and r again
    const auto h_at = [&](int c) { return sum ? sum[c] : (r ? from_f32<T>(to_f32(x[c]) + to_f32(r[c])) : x[c]); };
    const float mean = ss / (float)a.channels + a.eps;
    InverseRoot s{1.0f / sqrtf(mean), 0};
    if (far<T>(mean)) {
      double again = 0.0;
      for (int c = g; c < a.channels; c += L) {
        const double f = to_f32(h_at(c));
        again += f * f;
      }
      s = far_root(group_sum<L>(again, s_far, turn) / a.channels + a.eps);
    }
    if (!kI8 && a.rstd && g == 0) a.rstd[row] = s.value();
    double to_q = 0.0;
    if constexpr (kI8) {
      float scale;
      to_q = row_factor(top, s, scale);
      if (g == 0) a.scale[row] = scale;
    }
    for (int c = g; c < a.channels; c += L) {
      const float f = to_f32(h_at(c)), w = weight_at(a.weight, a.weight_dtype, c);
      if constexpr (kI8) a.q[row * a.channels + c] = to_q > 0.0 ? nearest_i8((double)f * (double)w, to_q) : 0;
      else static_cast<T*>(a.out)[row * a.channels + c] = from_f32<T>(s.times(f) * w);
    }
  }
}

template <typename T, int L>
__global__ void __launch_bounds__(kNormThreads) k_rms_norm_grad_any(NormGradArgs a) {
  __shared__ GroupScratch<float> s_red;
  const int g = threadIdx.x % L;
  int turn = 0;
  for (i64 row = (i64)blockIdx.x * (kNormThreads / L) + threadIdx.x / L; row < a.rows;
       row += (i64)gridDim.x * (kNormThreads / L), turn ^= 1) {
    const T* dy = static_cast<const T*>(a.grad_out) + row * a.grad_out_stride;
    const T* h = static_cast<const T*>(a.h) + row * a.h_stride;
    const T* dh = a.grad_sum ? static_cast<const T*>(a.grad_sum) + row * a.grad_sum_stride : nullptr;
    const float rstd = a.rstd[row];
    float dot = 0.0f;
    for (int c = g; c < a.channels; c += L)
      dot += to_f32(dy[c]) * weight_at(a.weight, a.weight_dtype, c) * (to_f32(h[c]) * rstd);
    dot = group_sum<L>(dot, s_red, turn);
    const float along = rstd * (dot / (float)a.channels);
    for (int c = g; c < a.channels; c += L) {
      const float gy = to_f32(dy[c]) * weight_at(a.weight, a.weight_dtype, c);
      const float v = rstd * gy - to_f32(h[c]) * rstd * along;
      static_cast<T*>(a.grad_x)[row * a.channels + c] = from_f32<T>(dh ? v + to_f32(dh[c]) : v);
    }
  }
}

// The weight gradient's parts for the rows of k_rms_norm_grad_any: block (column
// group, part) adds a contiguous range of rows. Beside that kernel's 209 us for 2048 x 20000 bf16 it takes 68
// and the sum of the parts 13; for 124800 x 3 f32, where three threads of a workgroup add, 18 beside 4.
template <typename T>
__global__ void __launch_bounds__(kNormThreads) k_rms_norm_grad_part(NormGradArgs a, int parts, i64 rows_per_part) {
  const int groups = (a.channels + kNormThreads - 1) / kNormThreads;
  const int part = blockIdx.x / groups;
  const int c = (blockIdx.x % groups) * kNormThreads + threadIdx.x;
  if (c >= a.channels) return;
  const i64 r0 = (i64)part * rows_per_part;
  const i64 r1 = min(a.rows, r0 + rows_per_part);
  float acc = 0.0f;
  for (i64 row = r0; row < r1; ++row)
    acc += to_f32(static_cast<const T*>(a.grad_out)[row * a.grad_out_stride + c]) *
           (to_f32(static_cast<const T*>(a.h)[row * a.h_stride + c]) * a.rstd[row]);
  a.partial[(i64)part * a.channels + c] = acc;
}

// dw: the sum of the parts, 32 channels by 32 slices of the parts a workgroup.
constexpr int kSumChannels = 32, kSumSlices = 32;
__global__ void __launch_bounds__(kSumChannels* kSumSlices)
    k_rms_norm_grad_sum(const float* partial, int parts, int channels, float* out) {
  __shared__ float s_part[kSumSlices][kSumChannels];
  const int cl = threadIdx.x % kSumChannels, slice = threadIdx.x / kSumChannels;
  const int c = blockIdx.x * kSumChannels + cl;
  float acc = 0.0f;
  if (c < channels) {
#pragma unroll 8
    for (int p = slice; p < parts; p += kSumSlices) acc += partial[(i64)p * channels + c];
  }
  s_part[slice][cl] = acc;
  __syncthreads();
  if (slice == 0 && c < channels) {
#pragma unroll
    for (int k = 1; k < kSumSlices; ++k) acc += s_part[k][cl];
    out[c] = acc;
  }
}

// Workgroups whose parts of the weight gradient are joined at the end: enough to
// have memory busy, while the parts stay small next to the rows (forward and backward of
// 16384 x 4096 with 512 parts 265 us, 1024: 220, 2048: 238; of 124800 x 128 with 1024: 58, 2048: 64).
constexpr int kGradParts = 1024;
int grad_parts(i64 rows) { return (int)std::max<i64>(1, std::min<i64>(rows, kGradParts)); }

}  // namespace

void rms_norm(const NormArgs& a, hipStream_t s) {
  if (a.rows == 0) return;
  const i64 most = (i64)device_cu_count() * 8;  // workgroups that fill the card; each takes its rows in turn
  with_dtype(a.dtype, [&](auto t) {
    using T = decltype(t);
    constexpr int V = Vec<T>::kN;
    auto blocks = [&](int rows) { return std::min<i64>(ceil_div(a.rows, rows), most); };
    auto any = [&](auto l) {
      constexpr int L = decltype(l)::value;
      launch("k_rms_norm_any", a.q ? k_rms_norm_any<T, L, true> : k_rms_norm_any<T, L, false>, blocks(kNormThreads / L),
             kNormThreads, s, a);
    };
    if (a.channels < V) return any(std::integral_constant<int, 1>());
    const bool held = with_place(ceil_div(a.channels, V), [&](auto l, auto n) {
      constexpr int L = decltype(l)::value, N = decltype(n)::value;
      if (a.q) launch("k_rms_norm", k_rms_norm<T, L, N, true>, blocks(kNormThreads / L), kNormThreads, s, a);
      else launch("k_rms_norm", k_rms_norm<T, L, N, false>, blocks(kNormThreads / L), kNormThreads, s, a);
    });
    if (!held) any(std::integral_constant<int, kNormThreads>());
  });
}

size_t rms_norm_grad_workspace(i64 rows, int channels) {
  return sizeof(float) * (size_t)grad_parts(rows) * (size_t)channels;
}

void rms_norm_grad(const NormGradArgs& a, hipStream_t s) {
  with_dtype(a.dtype, [&](auto t) {
    using T = decltype(t);
    constexpr int V = Vec<T>::kN;
    const i64 most = (i64)device_cu_count() * 8;
    int parts = grad_parts(a.rows);
    bool held = false;
    if (a.channels >= V && a.rows > 0)
      held = with_place(ceil_div(a.channels, V), [&](auto l, auto n) {
        constexpr int L = decltype(l)::value, N = decltype(n)::value;
        const i64 groups = ceil_div(a.rows, kNormThreads / L);
        if (a.grad_weight) {
          parts = (int)std::min<i64>(parts, groups);
          launch("k_rms_norm_grad", k_rms_norm_grad<T, L, N, true>, parts, kNormThreads, s, a);
        } else {
          launch("k_rms_norm_grad", k_rms_norm_grad<T, L, N, false>, std::min(groups, most), kNormThreads, s, a);
        }
      });
    if (!held) {
      const bool narrow = a.channels < V;
      if (a.grad_x && a.rows) {
        if (narrow)
          launch("k_rms_norm_grad_any", k_rms_norm_grad_any<T, 1>,
                 std::min(ceil_div(a.rows, kNormThreads), most), kNormThreads, s, a);
        else
          launch("k_rms_norm_grad_any", k_rms_norm_grad_any<T, kNormThreads>, std::min(a.rows, most), kNormThreads, s,
                 a);
      }
      if (a.grad_weight)
        launch("k_rms_norm_grad_part", k_rms_norm_grad_part<T>, ceil_div(a.channels, kNormThreads) * parts,
               kNormThreads, s, a, parts, ceil_div(a.rows, parts));
    }
    if (a.grad_weight)
      launch("k_rms_norm_grad_sum", k_rms_norm_grad_sum, ceil_div(a.channels, kSumChannels), kSumChannels * kSumSlices,
             s, (const float*)a.partial, parts, a.channels, a.grad_weight);
  });
}

}  // namespace tc
