// Layer norm of feature rows with the residual's addition, and its gradient.
//
//   h = round(x + r), m = mean(h), s = 1 / sqrt(mean((h - m)^2) + eps), out = round((h - m) s w + b)
//
// The norm is that of the rounded h, as its gradient is taken from the stored h. The mean is a 64-bit
// sum, split into two floats, so that rows far from zero next to their spread keep the spread's digits
// (a 32-bit mean alone is off by 2^-25 of itself); the squares of the differences are a float sum. Where
// that nears the ends of 32 bits (spreads from 1.8e19 on, or below 1e-15 with an eps as small) they are
// summed again in 64 bits. Memory bounds all of it: a row is read once and held in registers.
#include "norm_rows.hpp"

namespace tc {

namespace {

// A 64-bit mean as two floats: h - m = (h - hi) - lo, each difference rounded once.
struct Centre {
  float hi, lo;
  __device__ __forceinline__ explicit Centre(double m) : hi((float)m), lo((float)(m - (double)hi)) {}
  __device__ __forceinline__ float from(float h) const { return (h - hi) - lo; }
};

// The weights of N channels from c on (T's type, or 32 bits; `none` without any).
template <typename T, int N>
__device__ __forceinline__ void weights_at(float (&w)[N], const void* p, int dtype, int c, float none) {
  if (!p) {
#pragma unroll
    for (int e = 0; e < N; ++e) w[e] = none;
  } else if (dtype == TC_F32) {
    __builtin_memcpy(w, static_cast<const float*>(p) + c, sizeof(w));
  } else {
    T t[N];
    __builtin_memcpy(t, static_cast<const T*>(p) + c, sizeof(t));
#pragma unroll
    for (int e = 0; e < N; ++e) w[e] = to_f32(t[e]);
  }
}

// The row stays in registers between the reductions and the outputs. h is stored only after a reduction over the row,
// when all of x and r is read: it may go over either. The 64-bit additions cost 3 to 7% of the time.
// Memory bounds it: 16384 x 4096 f16 95 us (5.6 TB/s), f32 205 (5.2), 124800 x 128 bf16 22 (5.9), f32 41 (6.2), one row of
// 1024 3.3 us.
template <typename T, int L, int N>
__global__ void __launch_bounds__(kNormThreads) k_layer_norm(LayerNormArgs a) {
  constexpr int V = Vec<T>::kN;
  __shared__ GroupScratch<double> s_mean, s_far;
  __shared__ GroupScratch<float> s_red;
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
  float w[N][V], b[N][V];
  load_weights<T, L, N>(w, at, a.weight, a.weight_dtype);
  load_weights<T, L, N>(b, at, a.bias, a.bias_dtype, 0.0f);
  int turn = 0;
  for (; row < a.rows; row += step, turn ^= 1) {
    Vec<T> h[N];
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e)
        h[j].v[e] = a.residual ? from_f32<T>(to_f32(x[j].v[e]) + to_f32(r[j].v[e])) : x[j].v[e];
    ask(row + step);
    // f(element) over the row's own elements, each once
    auto each = [&](auto&& f) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        if (at.c[j] < 0) continue;
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (!at.ragged || e >= at.skip[j]) f(to_f32(h[j].v[e]));
      }
    };
    double sum = 0.0;
    each([&](float f) { sum += f; });
    const double mean = group_sum<L>(sum, s_mean, turn) / a.channels;
    const Centre m(mean);
    float ss = 0.0f;
    each([&](float f) { ss += m.from(f) * m.from(f); });
    const float spread = group_sum<L>(ss, s_red, turn) / (float)a.channels + a.eps;
    InverseRoot s{1.0f / sqrtf(spread), 0};
    const bool again = far<T>(spread);  // the same for the whole row
    if (again) {
      double sum = 0.0;
      each([&](float f) { sum += ((double)f - mean) * ((double)f - mean); });
      s = far_root(group_sum<L>(sum, s_far, turn) / a.channels + a.eps);
    }
    if (a.sum) {
      T* to = static_cast<T*>(a.sum) + row * a.channels;
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (at.c[j] >= 0) h[j].store(to + at.c[j]);
    }
    if (threadIdx.x % L == 0) {
      if (a.mean) a.mean[row] = m.hi;
      if (a.rstd) a.rstd[row] = s.value();
    }
    T* out = static_cast<T*>(a.out) + row * a.channels;
    auto write = [&](auto unit) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        if (at.c[j] < 0) continue;
        Vec<T> o;
#pragma unroll
        for (int e = 0; e < V; ++e) o.v[e] = from_f32<T>(fmaf(unit(to_f32(h[j].v[e])), w[j][e], b[j][e]));
        o.store(out + at.c[j]);
      }
    };
    if (again) write([&](float f) { return (float)ldexp((double)f - mean, s.shift) * s.root; });
    else write([&](float f) { return m.from(f) * s.root; });
  }
}

// Rows of fewer channels than a vector has (L = 1: one thread a row), or of more than a workgroup's
// registers hold (L = a workgroup, the row read three times): whole vectors, the rest by elements. 2048 x 20000 bf16 97 us
// for the 65 that its bytes take (weights one by one: 166), 124800 x 3 f32 5.4.
template <typename T, int L>
__global__ void __launch_bounds__(kNormThreads) k_layer_norm_any(LayerNormArgs a) {
  constexpr int V = Vec<T>::kN;
  __shared__ GroupScratch<double> s_mean, s_far;
  __shared__ GroupScratch<float> s_red;
  const int g = threadIdx.x % L, whole = a.channels / V * V;
  int turn = 0;
  for (i64 row = (i64)blockIdx.x * (kNormThreads / L) + threadIdx.x / L; row < a.rows;
       row += (i64)gridDim.x * (kNormThreads / L), turn ^= 1) {
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    const T* r = a.residual ? static_cast<const T*>(a.residual) + row * a.residual_stride : nullptr;
    T* sum = a.sum ? static_cast<T*>(a.sum) + row * a.channels : nullptr;
    T* out = static_cast<T*>(a.out) + row * a.channels;
    // f(h, first channel) over vectors and elements of h = x + r, or of what this thread stored of it
    auto each = [&](bool stored, auto&& f) {
      for (int c = g * V; c < whole; c += L * V) {
        Vec<T> v;
        v.load(stored ? sum + c : x + c);
        if (r && !stored) {
          Vec<T> o;
          o.load(r + c);
#pragma unroll
          for (int e = 0; e < V; ++e) v.v[e] = from_f32<T>(to_f32(v.v[e]) + to_f32(o.v[e]));
        }
        f(v.v, c, std::integral_constant<int, V>());
      }
      for (int c = whole + g; c < a.channels; c += L) {
        T v[1] = {stored ? sum[c] : r ? from_f32<T>(to_f32(x[c]) + to_f32(r[c])) : x[c]};
        f(v, c, std::integral_constant<int, 1>());
      }
    };
    double total = 0.0;
    each(false, [&](const T* v, int c, auto n) {
#pragma unroll
      for (int e = 0; e < n; ++e) total += to_f32(v[e]);
      if (sum) __builtin_memcpy(sum + c, v, n * sizeof(T));
    });
    const double mean = group_sum<L>(total, s_mean, turn) / a.channels;
    const Centre m(mean);
    float ss = 0.0f;
    each(sum, [&](const T* v, int c, auto n) {
#pragma unroll
      for (int e = 0; e < n; ++e) ss += m.from(to_f32(v[e])) * m.from(to_f32(v[e]));
    });
    const float spread = group_sum<L>(ss, s_red, turn) / (float)a.channels + a.eps;
    InverseRoot s{1.0f / sqrtf(spread), 0};
    const bool again = far<T>(spread);
    if (again) {
      total = 0.0;
      each(sum, [&](const T* v, int c, auto n) {
#pragma unroll
        for (int e = 0; e < n; ++e) total += ((double)to_f32(v[e]) - mean) * ((double)to_f32(v[e]) - mean);
      });
      s = far_root(group_sum<L>(total, s_far, turn) / a.channels + a.eps);
    }
    if (g == 0) {
      if (a.mean) a.mean[row] = m.hi;
      if (a.rstd) a.rstd[row] = s.value();
    }
    each(sum, [&](const T* v, int c, auto n) {
      T o[n];
      float w[n], b[n];
      weights_at<T, n>(w, a.weight, a.weight_dtype, c, 1.0f);
      weights_at<T, n>(b, a.bias, a.bias_dtype, c, 0.0f);
#pragma unroll
      for (int e = 0; e < n; ++e) {
        const float f = to_f32(v[e]);
        const float u = again ? (float)ldexp((double)f - mean, s.shift) * s.root : m.from(f) * s.root;
        o[e] = from_f32<T>(fmaf(u, w[e], b[e]));
      }
      __builtin_memcpy(out + c, o, n * sizeof(T));
    });
  }
}

// ------------------------------------------------------------------ gradient

// dx = s (g - mean(g) - u mean(g u)) + dh with g = dy w and the unit row u = (h - m) s. m comes as one float: with
// v = (h - m) s, u is v - mean(v), and mean(g u) = mean(g v) - mean(v) mean(g), so one pass over the
// row gives all three sums.
struct GradSums {
  float g, gv, v;
  __device__ __forceinline__ void add(float gy, float unit) {
    g += gy;
    gv += gy * unit;
    v += unit;
  }
  // of the row: means of g, of g u, and of v
  __device__ __forceinline__ void finish(float channels) {
    g /= channels;
    v /= channels;
    gv = gv / channels - v * g;
  }
};
struct GradScratch {
  float part[2][3][kNormThreads / kWave];
};
template <int L>
__device__ __forceinline__ GradSums group_sums(GradSums s, GradScratch& scratch, int turn) {
  constexpr int W = L < kWave ? L : kWave;
  auto add = [](float a, float b) { return a + b; };
  s.g = lanes_reduce<W>(s.g, add);
  s.gv = lanes_reduce<W>(s.gv, add);
  s.v = lanes_reduce<W>(s.v, add);
  if constexpr (L > kWave) {
    auto& p = scratch.part[turn];
    if ((threadIdx.x & (kWave - 1)) == 0) {
      p[0][threadIdx.x / kWave] = s.g;
      p[1][threadIdx.x / kWave] = s.gv;
      p[2][threadIdx.x / kWave] = s.v;
    }
    __syncthreads();
    s.g = (p[0][0] + p[0][1]) + (p[0][2] + p[0][3]);
    s.gv = (p[1][0] + p[1][1]) + (p[1][2] + p[1][3]);
    s.v = (p[2][0] + p[2][1]) + (p[2][2] + p[2][3]);
  }
  return s;
}

// (h - m) s of a row's elements. The difference leaves 32 bits for rows beyond half their range, and s the normal
// numbers for spreads from 2^126 on: a power of two, 1 but for rows of such sizes, goes from one to the other.
struct Unit {
  float by, centre, rstd;
  __device__ __forceinline__ Unit(float mean, float s) {
    const bool large = s < 0x1p-62f;
    by = large ? 0x1p-64f : 1.0f;
    centre = -(mean * by);
    rstd = s * (large ? 0x1p64f : 1.0f);
  }
  __device__ __forceinline__ float of(float h) const { return fmaf(h, by, centre) * rstd; }
};

// This workgroup's parts of dw = sum dy u and of db = sum dy: each thread adds up its channels over its rows
// in registers, the workgroup's groups are joined once at the end. 16384 x 4096 f16 115 us (4.7 TB/s) and 6 for the sum of
// the parts, f32 205 and 8, 124800 x 128 bf16 23 and 4.
template <typename T, int L, int N, bool kParams>
__global__ void __launch_bounds__(kNormThreads) k_layer_norm_grad(LayerNormGradArgs a) {
  constexpr int V = Vec<T>::kN;
  __shared__ GradScratch s_red;
  const RowPlace<T, L, N> at(a.channels);
  const i64 step = (i64)gridDim.x * (kNormThreads / L);
  i64 row = (i64)blockIdx.x * (kNormThreads / L) + threadIdx.x / L;
  Vec<T> next_dy[N], next_h[N], next_dh[N];  // of the next row
  float next_mean = 0.0f, next_rstd = 0.0f;
  auto ask = [&](i64 row) {
    if (row >= a.rows) return;
    load_row<T, L, N>(next_dy, at, a.grad_out, row * a.grad_out_stride);
    load_row<T, L, N>(next_h, at, a.h, row * a.h_stride);
    if (a.grad_sum) load_row<T, L, N>(next_dh, at, a.grad_sum, row * a.grad_sum_stride);
    next_mean = a.mean[row];
    next_rstd = a.rstd[row];
  };
  ask(row);
  float w[N][V], dw[N][V], db[N][V];
  load_weights<T, L, N>(w, at, a.weight, a.weight_dtype);
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int e = 0; e < V; ++e) dw[j][e] = db[j][e] = 0.0f;
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
    const Unit unit(next_mean, rstd);
    ask(row + step);
    GradSums s{0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (at.c[j] < 0) continue;
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (!at.ragged || e >= at.skip[j]) s.add(to_f32(dy[j].v[e]) * w[j][e], unit.of(to_f32(h[j].v[e])));
    }
    s = group_sums<L>(s, s_red, turn);
    s.finish((float)a.channels);
    T* dx = static_cast<T*>(a.grad_x) + row * a.channels;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (at.c[j] < 0) continue;
      Vec<T> o;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float y = to_f32(dy[j].v[e]), u = unit.of(to_f32(h[j].v[e])) - s.v;
        if constexpr (kParams) {
          dw[j][e] += y * u;
          db[j][e] += y;
        }
        const float v = rstd * ((y * w[j][e] - s.g) - u * s.gv);
        o.v[e] = from_f32<T>(a.grad_sum ? v + to_f32(dh[j].v[e]) : v);
      }
      if (a.grad_x) o.store(dx + at.c[j]);
    }
  }
  if constexpr (kParams) {
    float* part = a.partial + (i64)blockIdx.x * 2 * a.channels;
    if constexpr (L > kWave) {
#pragma unroll
      for (int j = 0; j < N; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (at.c[j] >= 0) {
            part[at.c[j] + e] = dw[j][e];
            part[a.channels + at.c[j] + e] = db[j][e];
          }
    } else {
      constexpr int kWaves = kNormThreads / kWave;
      __shared__ float s_part[2][kWaves][L * N * V];
      const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
#pragma unroll
      for (int j = 0; j < N; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float v = dw[j][e], b = db[j][e];
#pragma unroll
          for (int d = L; d < kWave; d <<= 1) {
            v += __shfl_xor(v, d, kWave);
            b += __shfl_xor(b, d, kWave);
          }
          if (lane < L) {
            s_part[0][wave][(j * L + lane) * V + e] = v;
            s_part[1][wave][(j * L + lane) * V + e] = b;
          }
        }
      __syncthreads();
      // slot i of the row's vectors, placed as RowPlace has it
      for (int i = threadIdx.x; i < 2 * L * N * V; i += kNormThreads) {
        const int which = i / (L * N * V), slot = i % (L * N * V), first = slot / V * V;
        if (first >= a.channels) continue;
        float v = s_part[which][0][slot];
#pragma unroll
        for (int k = 1; k < kWaves; ++k) v += s_part[which][k][slot];
        part[which * a.channels + min(first, a.channels - V) + slot % V] = v;
      }
    }
  }
}

// Rows of fewer channels than a vector has, one thread a row: 124800 x 3 f32 8 us with the sum.
template <typename T, bool kParams>
__global__ void __launch_bounds__(kNormThreads) k_layer_norm_grad_narrow(LayerNormGradArgs a) {
  constexpr int C = Vec<T>::kN - 1;  // the most channels
  float w[C], dw[C], db[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    w[c] = c < a.channels && a.weight ? weight_at(a.weight, a.weight_dtype, c) : 1.0f;
    dw[c] = db[c] = 0.0f;
  }
  for (i64 row = (i64)blockIdx.x * kNormThreads + threadIdx.x; row < a.rows; row += (i64)gridDim.x * kNormThreads) {
    const T* dy = static_cast<const T*>(a.grad_out) + row * a.grad_out_stride;
    const T* h = static_cast<const T*>(a.h) + row * a.h_stride;
    const T* dh = a.grad_sum ? static_cast<const T*>(a.grad_sum) + row * a.grad_sum_stride : nullptr;
    const float rstd = a.rstd[row];
    const Unit unit(a.mean[row], rstd);
    float y[C], v[C];
    GradSums s{0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (c >= a.channels) continue;
      y[c] = to_f32(dy[c]);
      v[c] = unit.of(to_f32(h[c]));
      s.add(y[c] * w[c], v[c]);
    }
    s.finish((float)a.channels);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (c >= a.channels) continue;
      const float u = v[c] - s.v, d = rstd * ((y[c] * w[c] - s.g) - u * s.gv);
      dw[c] += y[c] * u;
      db[c] += y[c];
      if (a.grad_x) static_cast<T*>(a.grad_x)[row * a.channels + c] = from_f32<T>(dh ? d + to_f32(dh[c]) : d);
    }
  }
  if constexpr (kParams) {
    constexpr int kWaves = kNormThreads / kWave;
    __shared__ float s_part[kWaves][2][C];
    auto add = [](float a, float b) { return a + b; };
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float x = lanes_reduce<kWave>(dw[c], add), b = lanes_reduce<kWave>(db[c], add);
      if ((threadIdx.x & (kWave - 1)) == 0) {
        s_part[threadIdx.x / kWave][0][c] = x;
        s_part[threadIdx.x / kWave][1][c] = b;
      }
    }
    __syncthreads();
    const int which = threadIdx.x / a.channels, c = threadIdx.x % a.channels;
    if (which < 2) {
      float v = s_part[0][which][c];
#pragma unroll
      for (int k = 1; k < kWaves; ++k) v += s_part[k][which][c];
      a.partial[((i64)blockIdx.x * 2 + which) * a.channels + c] = v;
    }
  }
}

// Rows that a workgroup's registers do not hold: a workgroup a row, the row read twice; mean(v), which the
// parts of dw need, is left for k_layer_norm_grad_part (which reads both once more): 2048 x 20000 bf16 206 us
// together (weights one by one: 333).
template <typename T>
__global__ void __launch_bounds__(kNormThreads) k_layer_norm_grad_wide(LayerNormGradArgs a, float* unit_mean) {
  constexpr int V = Vec<T>::kN;
  __shared__ GradScratch s_red;
  const int whole = a.channels / V * V;
  int turn = 0;
  for (i64 row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    const T* dy = static_cast<const T*>(a.grad_out) + row * a.grad_out_stride;
    const T* h = static_cast<const T*>(a.h) + row * a.h_stride;
    const T* dh = a.grad_sum ? static_cast<const T*>(a.grad_sum) + row * a.grad_sum_stride : nullptr;
    const float rstd = a.rstd[row];
    const Unit unit(a.mean[row], rstd);
    auto each = [&](auto&& f) {
      for (int c = threadIdx.x * V; c < whole; c += kNormThreads * V) {
        Vec<T> y, v;
        y.load(dy + c);
        v.load(h + c);
        f(y.v, v.v, c, std::integral_constant<int, V>());
      }
      for (int c = whole + threadIdx.x; c < a.channels; c += kNormThreads)
        f(dy + c, h + c, c, std::integral_constant<int, 1>());
    };
    GradSums s{0.0f, 0.0f, 0.0f};
    each([&](const T* y, const T* v, int c, auto n) {
      float w[n];
      weights_at<T, n>(w, a.weight, a.weight_dtype, c, 1.0f);
#pragma unroll
      for (int e = 0; e < n; ++e) s.add(to_f32(y[e]) * w[e], unit.of(to_f32(v[e])));
    });
    s = group_sums<kNormThreads>(s, s_red, turn);
    s.finish((float)a.channels);
    if (unit_mean && threadIdx.x == 0) unit_mean[row] = s.v;
    if (!a.grad_x) continue;
    T* dx = static_cast<T*>(a.grad_x) + row * a.channels;
    each([&](const T* y, const T* v, int c, auto n) {
      T o[n], add[n];
      float w[n];
      weights_at<T, n>(w, a.weight, a.weight_dtype, c, 1.0f);
      if (dh) __builtin_memcpy(add, dh + c, n * sizeof(T));
#pragma unroll
      for (int e = 0; e < n; ++e) {
        const float u = unit.of(to_f32(v[e])) - s.v;
        const float d = rstd * ((to_f32(y[e]) * w[e] - s.g) - u * s.gv);
        o[e] = from_f32<T>(dh ? d + to_f32(add[e]) : d);
      }
      __builtin_memcpy(dx + c, o, n * sizeof(T));
    });
  }
}

// The parts of dw and db for those rows: block (column group, part) adds a contiguous range of rows.
template <typename T>
__global__ void __launch_bounds__(kNormThreads)
    k_layer_norm_grad_part(LayerNormGradArgs a, const float* unit_mean, int groups, i64 rows_per_part) {
  const int part = blockIdx.x / groups, c = (blockIdx.x % groups) * kNormThreads + threadIdx.x;
  if (c >= a.channels) return;
  const i64 r0 = (i64)part * rows_per_part, r1 = min(a.rows, r0 + rows_per_part);
  float dw = 0.0f, db = 0.0f;
  for (i64 row = r0; row < r1; ++row) {
    const float y = to_f32(static_cast<const T*>(a.grad_out)[row * a.grad_out_stride + c]);
    const T h = static_cast<const T*>(a.h)[row * a.h_stride + c];
    dw += y * (Unit(a.mean[row], a.rstd[row]).of(to_f32(h)) - unit_mean[row]);
    db += y;
  }
  a.partial[(i64)part * 2 * a.channels + c] = dw;
  a.partial[((i64)part * 2 + 1) * a.channels + c] = db;
}

// dw and db: the sums of the parts, 32 channels by 32 slices of the parts a workgroup, the slices by eights. 768 parts of
// 8192 5.6 us (16 channels by 64 slices 8.7: half lines), 1024 of 256 4.7.
constexpr int kSumChannels = 32, kSumSlices = 32, kSumFirst = 4, kSumGroup = kSumSlices / kSumFirst;
__global__ void __launch_bounds__(kSumChannels* kSumSlices)
    k_layer_norm_grad_sum(const float* partial, int parts, int channels, float* dw, float* db) {
  __shared__ float s_part[kSumSlices][kSumChannels], s_first[kSumFirst][kSumChannels];
  const int cl = threadIdx.x % kSumChannels, slice = threadIdx.x / kSumChannels;
  const i64 c = (i64)blockIdx.x * kSumChannels + cl;  // of both, one after the other
  const bool bias = c >= channels;
  float* out = bias ? db : dw;
  float acc = 0.0f;
  if (c < 2 * (i64)channels) {
#pragma unroll 8
    for (int p = slice; p < parts; p += kSumSlices) acc += partial[(i64)p * 2 * channels + c];
  }
  s_part[slice][cl] = acc;
  __syncthreads();
  if (slice < kSumFirst) {
    acc = s_part[slice * kSumGroup][cl];
#pragma unroll
    for (int k = 1; k < kSumGroup; ++k) acc += s_part[slice * kSumGroup + k][cl];
    s_first[slice][cl] = acc;
  }
  __syncthreads();
  if (slice == 0 && c < 2 * (i64)channels && out) {
#pragma unroll
    for (int k = 1; k < kSumFirst; ++k) acc += s_first[k][cl];
    out[bias ? c - channels : c] = acc;
  }
}

// Workgroups whose parts of the weights' gradients are joined at the end.
constexpr int kGradParts = 1024;
int grad_parts(i64 rows) { return (int)std::max<i64>(1, std::min<i64>(rows, kGradParts)); }

// Workgroups a CU that k_layer_norm_grad's registers leave room for, and no more than four: as many parts are one round, with
// the least traffic of the parts themselves (16384 x 4096 f16: 121 us, in 1024 parts 127; 8192 x 8192 bf16 128, 155;
// 8192 x 8192 f32 216, 242).
template <typename T>
int resident(int vectors) {
  return vectors >= 8 ? 1 : vectors >= 4 ? 2 : vectors == 2 && sizeof(T) == 2 ? 3 : 4;
}

// The most channels that the registers of a workgroup hold for every type: wider rows may need a
// float each in the workspace.
constexpr int kHeldChannels = 2048 * 16 / sizeof(float);

}  // namespace

void layer_norm(const LayerNormArgs& a, hipStream_t s) {
  if (a.rows == 0) return;
  const i64 most = (i64)device_cu_count() * 8;  // workgroups that fill the card; each takes its rows in turn
  with_dtype(a.dtype, [&](auto t) {
    using T = decltype(t);
    constexpr int V = Vec<T>::kN;
    auto blocks = [&](int rows) { return std::min<i64>(ceil_div(a.rows, rows), most); };
    if (a.channels < V)
      return launch("k_layer_norm_any", k_layer_norm_any<T, 1>, blocks(kNormThreads), kNormThreads, s, a);
    const bool held = with_place(ceil_div(a.channels, V), [&](auto l, auto n) {
      constexpr int L = decltype(l)::value, N = decltype(n)::value;
      launch("k_layer_norm", k_layer_norm<T, L, N>, blocks(kNormThreads / L), kNormThreads, s, a);
    });
    if (!held) launch("k_layer_norm_any", k_layer_norm_any<T, kNormThreads>, blocks(1), kNormThreads, s, a);
  });
}

size_t layer_norm_grad_workspace(i64 rows, int channels) {
  return sizeof(float) * ((size_t)grad_parts(rows) * 2 * (size_t)channels +
                          (channels > kHeldChannels ? (size_t)rows : 0));
}

void layer_norm_grad(const LayerNormGradArgs& a, hipStream_t s) {
  const bool params = a.grad_weight || a.grad_bias;
  with_dtype(a.dtype, [&](auto t) {
    using T = decltype(t);
    constexpr int V = Vec<T>::kN;
    const i64 most = (i64)device_cu_count() * 8;
    int parts = grad_parts(a.rows);
    if (a.rows == 0) {
      parts = 0;
    } else if (a.channels < V) {
      const i64 groups = ceil_div(a.rows, kNormThreads);
      parts = (int)std::min<i64>(parts, groups);
      if (params) launch("k_layer_norm_grad_narrow", k_layer_norm_grad_narrow<T, true>, parts, kNormThreads, s, a);
      else launch("k_layer_norm_grad_narrow", k_layer_norm_grad_narrow<T, false>, std::min(groups, most), kNormThreads, s, a);
    } else if (!with_place(ceil_div(a.channels, V), [&](auto l, auto n) {
                 constexpr int L = decltype(l)::value, N = decltype(n)::value;
                 const i64 groups = ceil_div(a.rows, kNormThreads / L);
                 if (params) {
                   const i64 most_parts = resident<T>(N) * (i64)device_cu_count();
                   parts = (int)std::min<i64>({parts, groups, most_parts});
                   launch("k_layer_norm_grad", k_layer_norm_grad<T, L, N, true>, parts, kNormThreads, s, a);
                 } else {
                   launch("k_layer_norm_grad", k_layer_norm_grad<T, L, N, false>, std::min(groups, most), kNormThreads,
                          s, a);
                 }
               })) {
      float* unit_mean = params ? a.partial + (i64)parts * 2 * a.channels : nullptr;
      const int groups = (int)ceil_div(a.channels, kNormThreads);
      launch("k_layer_norm_grad_wide", k_layer_norm_grad_wide<T>, std::min(a.rows, most), kNormThreads, s, a, unit_mean);
      if (params)
        launch("k_layer_norm_grad_part", k_layer_norm_grad_part<T>, (i64)groups * parts, kNormThreads, s, a,
               (const float*)unit_mean, groups, ceil_div(a.rows, parts));
    }
    if (params)
      launch("k_layer_norm_grad_sum", k_layer_norm_grad_sum, ceil_div(2 * (i64)a.channels, kSumChannels),
             kSumChannels * kSumSlices, s, (const float*)a.partial, parts, a.channels, a.grad_weight, a.grad_bias);
  });
}

}  // namespace tc
