// Root-mean-square norm of feature rows with the residual's addition, its
// 8-bit form and its gradient.
//
//   h = round(x + r), s = 1 / sqrt(mean(h^2) + eps), out = round(h s w)
//
// h is rounded to the rows' type once and the norm is the norm of that rounded
// h, so the gradient taken from the stored h is the gradient of what was
// computed. The mean is a float sum of float squares.
#include "rows.hpp"

namespace tc {

namespace {

constexpr int kNormThreads = 256;
constexpr int kNormRows = kNormThreads / kWave;  // one wave per row

__device__ __forceinline__ float weight_at(const void* w, int dt, int c) {
  if (!w) return 1.0f;
  if (dt == TC_F32) return static_cast<const float*>(w)[c];
  if (dt == TC_F16) return to_f32(static_cast<const f16*>(w)[c]);
  return to_f32(static_cast<const bf16*>(w)[c]);
}

// One wave per row, one element per lane and step. The second pass reads h
// where the first one stored it (the same lane's elements), else x and r again.
template <typename T>
__global__ void __launch_bounds__(kNormThreads) k_rms_norm_any(NormArgs a) {
  const int lane = threadIdx.x & (kWave - 1);
  for (i64 row = (i64)blockIdx.x * kNormRows + threadIdx.x / kWave; row < a.rows; row += (i64)gridDim.x * kNormRows) {
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    const T* r = a.residual ? static_cast<const T*>(a.residual) + row * a.residual_stride : nullptr;
    T* sum = a.sum ? static_cast<T*>(a.sum) + row * a.channels : nullptr;
    float ss = 0.0f;
    double top = 0.0;
    for (int c = lane; c < a.channels; c += kWave) {
      const T h = r ? from_f32<T>(to_f32(x[c]) + to_f32(r[c])) : x[c];
      if (sum) sum[c] = h;
      const float f = to_f32(h);
      ss += f * f;
      if (a.q) {
        // h w is exact in 64 bits; an infinity or NaN makes `top` infinite
        const double p = fabs((double)f * (double)weight_at(a.weight, a.weight_dtype, c));
        top = p < INFINITY ? fmax(top, p) : INFINITY;
      }
    }
    ss = wave_sum_f32(ss);
    const float rstd = 1.0f / sqrtf(ss / (float)a.channels + a.eps);
    if (a.rstd && lane == 0) a.rstd[row] = rstd;
    double to_q = 0.0;
    if (a.q) {
      top = wave_max_f64(top);
      const bool finite = top < INFINITY;
      to_q = finite && top > 0.0 ? 127.0 / top : 0.0;
      if (lane == 0) a.scale[row] = finite ? (top > 0.0 ? (float)top * rstd / 127.0f : 0.0f) : NAN;
    }
    for (int c = lane; c < a.channels; c += kWave) {
      const T h = sum ? sum[c] : (r ? from_f32<T>(to_f32(x[c]) + to_f32(r[c])) : x[c]);
      const float f = to_f32(h), w = weight_at(a.weight, a.weight_dtype, c);
      if (a.out) static_cast<T*>(a.out)[row * a.channels + c] = from_f32<T>(f * rstd * w);
      if (a.q) a.q[row * a.channels + c] = to_q > 0.0 ? (int8_t)(int)rint((double)f * (double)w * to_q) : 0;
    }
  }
}

// dx = s g - h s^3 mean(g h) + dh with g = dy w; one wave per row.
template <typename T>
__global__ void __launch_bounds__(kNormThreads) k_rms_norm_grad_any(NormGradArgs a) {
  const int lane = threadIdx.x & (kWave - 1);
  for (i64 row = (i64)blockIdx.x * kNormRows + threadIdx.x / kWave; row < a.rows; row += (i64)gridDim.x * kNormRows) {
    const T* dy = static_cast<const T*>(a.grad_out) + row * a.grad_out_stride;
    const T* h = static_cast<const T*>(a.h) + row * a.h_stride;
    const T* dh = a.grad_sum ? static_cast<const T*>(a.grad_sum) + row * a.grad_sum_stride : nullptr;
    const float rstd = a.rstd[row];
    float dot = 0.0f;
    for (int c = lane; c < a.channels; c += kWave)
      dot += to_f32(dy[c]) * weight_at(a.weight, a.weight_dtype, c) * to_f32(h[c]);
    dot = wave_sum_f32(dot);
    const float k = rstd * rstd * rstd * (dot / (float)a.channels);
    for (int c = lane; c < a.channels; c += kWave) {
      const float g = to_f32(dy[c]) * weight_at(a.weight, a.weight_dtype, c);
      const float v = rstd * g - to_f32(h[c]) * k + (dh ? to_f32(dh[c]) : 0.0f);
      static_cast<T*>(a.grad_x)[row * a.channels + c] = from_f32<T>(v);
    }
  }
}

// dw = sum over rows of dy h s, in two steps with a fixed order: block (column
// group, part) adds a contiguous range of rows, then one thread per channel
// adds the parts.
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
           to_f32(static_cast<const T*>(a.h)[row * a.h_stride + c]) * a.rstd[row];
  a.partial[(i64)part * a.channels + c] = acc;
}

__global__ void __launch_bounds__(kNormThreads) k_rms_norm_grad_sum(const float* partial, int parts, int channels,
                                                                    float* out) {
  const int c = blockIdx.x * kNormThreads + threadIdx.x;
  if (c >= channels) return;
  float acc = 0.0f;
  for (int p = 0; p < parts; ++p) acc += partial[(i64)p * channels + c];
  out[c] = acc;
}

// Parts of the weight gradient's sum over rows.
int grad_parts(i64 rows) { return (int)std::max<i64>(1, std::min<i64>(256, ceil_div(rows, 64))); }

}  // namespace

void rms_norm(const NormArgs& a, hipStream_t s) {
  if (a.rows == 0) return;
  const i64 blocks = std::min<i64>(ceil_div(a.rows, kNormRows), (i64)device_cu_count() * 64);
  with_dtype(a.dtype, [&](auto t) {
    using T = decltype(t);
    launch("k_rms_norm_any", k_rms_norm_any<T>, blocks, kNormThreads, s, a);
  });
}

size_t rms_norm_grad_workspace(i64 rows, int channels) {
  return sizeof(float) * (size_t)grad_parts(rows) * (size_t)channels;
}

void rms_norm_grad(const NormGradArgs& a, hipStream_t s) {
  with_dtype(a.dtype, [&](auto t) {
    using T = decltype(t);
    if (a.grad_x && a.rows)
      launch("k_rms_norm_grad_any", k_rms_norm_grad_any<T>,
             std::min<i64>(ceil_div(a.rows, kNormRows), (i64)device_cu_count() * 64), kNormThreads, s, a);
    if (a.grad_weight) {
      const int parts = grad_parts(a.rows);
      const i64 groups = ceil_div(a.channels, kNormThreads);
      launch("k_rms_norm_grad_part", k_rms_norm_grad_part<T>, groups * parts, kNormThreads, s, a, parts,
             ceil_div(a.rows, parts));
      launch("k_rms_norm_grad_sum", k_rms_norm_grad_sum, groups, kNormThreads, s, (const float*)a.partial, parts,
             a.channels, a.grad_weight);
    }
  });
}

}  // namespace tc
