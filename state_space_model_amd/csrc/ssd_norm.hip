// The norms around a block's scan for gfx950, forward and backward, and the
// quantiser of 8-bit rows.
//
// Source: "Compiler-First State Space Duality and Portable O(1)
// Autoregressive Caching", Implementation choices, "precision management" (the
// residual stream and the norms in float32).
//
//   add norm    r' = r + s x;          y   = r' c w,  c = 1/sqrt(mean(r'^2) + eps)
//   gated norm  g  = y z / (1+e^-z);   out = g c w,   c per group of columns
//   8-bit rows  a = max|v|;  q = rint(v 127/a), scale a/127
#include "ssd_device.h"
#include "ssd_launch.h"

namespace ssd {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kParts = 256;  // rows of dweight partial sums

// Sum (or NaN-keeping maximum) over the workgroup, returned to every lane.
__device__ __forceinline__ float block_sum(float v, float* sm) {
  v = group_sum(v, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
  for (int i = 0; i < kThreads / 64; ++i) s += sm[i];
  return s;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  return (a != a || a > b) ? a : b;
}
__device__ __forceinline__ float block_max(float v, float* sm) {
  for (int off = 32; off > 0; off >>= 1) v = max_nan(v, __shfl_xor(v, off, 64));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
  for (int i = 0; i < kThreads / 64; ++i) s = max_nan(sm[i], s);
  return s;
}

__device__ __forceinline__ float silu(float z) { return z / (1.0f + expf(-z)); }

struct Q8Scale {
  float inv, scale;
};
__device__ __forceinline__ Q8Scale q8_scale(float a) {
  if (!(a < INFINITY)) return {0.0f, NAN};
  if (a < 0x1p-100f) return {0.0f, 0.0f};
  return {127.0f / a, a / 127.0f};
}
__device__ __forceinline__ int8_t q8_of(float v, Q8Scale s) {
  if (s.inv == 0.0f) return 0;
  return (int8_t)fminf(fmaxf(rintf(v * s.inv), -127.0f), 127.0f);
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_add_norm(AddNormArgs a) {
  __shared__ float sm[kThreads / 64];
  const int64_t o = (int64_t)blockIdx.x * a.D;
  const T* x = reinterpret_cast<const T*>(a.x) + o;
  auto rp = [&](int c) {
    const float r = a.residual ? a.residual[o + c] : 0.0f;
    return __fmaf_rn(a.scale, to_f32(x[c]), r);
  };
  float ss = 0.0f;
  for (int c = threadIdx.x; c < a.D; c += kThreads) ss += rp(c) * rp(c);
  const float rstd = 1.0f / sqrtf(block_sum(ss, sm) / (float)a.D + a.eps);
  Q8Scale qs = {};
  if (a.q) {
    float m = 0.0f;
    for (int c = threadIdx.x; c < a.D; c += kThreads) m = max_nan(fabsf(rp(c) * rstd * a.weight[c]), m);
    qs = q8_scale(block_max(m, sm));
    if (threadIdx.x == 0) a.qscale[blockIdx.x] = qs.scale;
    for (int c = a.D + threadIdx.x; c < a.Dp; c += kThreads) a.q[(int64_t)blockIdx.x * a.Dp + c] = 0;
  }
  for (int c = threadIdx.x; c < a.D; c += kThreads) {
    const float r = rp(c), n = r * rstd * a.weight[c];
    if (a.q) a.q[(int64_t)blockIdx.x * a.Dp + c] = q8_of(n, qs);
    else reinterpret_cast<T*>(a.y)[o + c] = to_io<T>(n);
    if (a.residual_out) a.residual_out[o + c] = r;
  }
}

// one workgroup per part: rows part, part + parts, ...
template <typename T>
__global__ __launch_bounds__(kThreads) void k_add_norm_backward(AddNormArgs a) {
  __shared__ float sm[kThreads / 64];
  float* part = a.part + (int64_t)blockIdx.x * a.D;
  for (int c = threadIdx.x; c < a.D; c += kThreads) part[c] = 0.0f;
  for (int64_t row = blockIdx.x; row < a.R; row += gridDim.x) {
    const int64_t o = row * a.D;
    const float* r = a.residual_out + o;
    const T* dy = reinterpret_cast<const T*>(a.dy) + o;
    float ss = 0.0f, pr = 0.0f;
    for (int c = threadIdx.x; c < a.D; c += kThreads) {
      ss += r[c] * r[c];
      pr += to_f32(dy[c]) * a.weight[c] * r[c];
    }
    const float rstd = 1.0f / sqrtf(block_sum(ss, sm) / (float)a.D + a.eps);
    const float m = block_sum(pr, sm) / (float)a.D * rstd;
    for (int c = threadIdx.x; c < a.D; c += kThreads) {
      const float xh = r[c] * rstd, d = to_f32(dy[c]);
      const float dr = rstd * (d * a.weight[c] - xh * m) + (a.dres_out ? a.dres_out[o + c] : 0.0f);
      part[c] += d * xh;
      if (a.dres) a.dres[o + c] = dr;
      if (a.dx) reinterpret_cast<T*>(a.dx)[o + c] = to_io<T>(a.scale * dr);
    }
  }
}

__global__ __launch_bounds__(kThreads) void k_sum_parts(const float* part, float* out, int64_t parts,
                                                        int64_t D) {
  const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (c >= D) return;
  float s = 0.0f;
  for (int64_t p = 0; p < parts; ++p) s += part[p * D + c];
  out[c] = s;
}

// one workgroup per row (its groups in order)
template <typename T>
__global__ __launch_bounds__(kThreads) void k_gated_norm(GatedNormArgs a) {
  __shared__ float sm[kThreads / 64];
  const int64_t o = (int64_t)blockIdx.x * a.D;
  const T* y = reinterpret_cast<const T*>(a.y) + o;
  const T* z = reinterpret_cast<const T*>(a.z) + (int64_t)blockIdx.x * a.z_stride;
  auto gated = [&](int c) { return to_f32(y[c]) * silu(to_f32(z[c])); };
  float m = 0.0f;
  Q8Scale qs = {};
  for (int pass = a.q ? 0 : 1; pass < 2; ++pass) {
    for (int g = 0; g < a.G; ++g) {
      const int c0 = g * a.W;
      float ss = 0.0f;
      for (int c = threadIdx.x; c < a.W; c += kThreads) ss += gated(c0 + c) * gated(c0 + c);
      const float rstd = 1.0f / sqrtf(block_sum(ss, sm) / (float)a.W + a.eps);
      for (int c = c0 + threadIdx.x; c < c0 + a.W; c += kThreads) {
        const float n = gated(c) * rstd * a.weight[c];
        if (pass == 0) m = max_nan(fabsf(n), m);
        else if (a.q) a.q[(int64_t)blockIdx.x * a.Dp + c] = q8_of(n, qs);
        else reinterpret_cast<T*>(a.out)[o + c] = to_io<T>(n);
      }
    }
    if (pass == 0) {
      qs = q8_scale(block_max(m, sm));
      if (threadIdx.x == 0) a.qscale[blockIdx.x] = qs.scale;
      for (int c = (int)a.D + threadIdx.x; c < a.Dp; c += kThreads)
        a.q[(int64_t)blockIdx.x * a.Dp + c] = 0;
    }
  }
}

// grid (parts, G)
template <typename T>
__global__ __launch_bounds__(kThreads) void k_gated_norm_backward(GatedNormArgs a) {
  __shared__ float sm[kThreads / 64];
  const int c0 = (int)blockIdx.y * a.W;
  const float* w = a.weight + c0;
  float* part = a.part + (int64_t)blockIdx.x * a.D + c0;
  for (int c = threadIdx.x; c < a.W; c += kThreads) part[c] = 0.0f;
  for (int64_t row = blockIdx.x; row < a.R; row += gridDim.x) {
    const int64_t o = row * a.D + c0;
    const T* y = reinterpret_cast<const T*>(a.y) + o;
    const T* z = reinterpret_cast<const T*>(a.z) + row * a.z_stride + c0;
    const T* dout = reinterpret_cast<const T*>(a.dout) + o;
    float ss = 0.0f, pg = 0.0f;
    for (int c = threadIdx.x; c < a.W; c += kThreads) {
      const float g = to_f32(y[c]) * silu(to_f32(z[c]));
      ss += g * g;
      pg += to_f32(dout[c]) * w[c] * g;
    }
    const float rstd = 1.0f / sqrtf(block_sum(ss, sm) / (float)a.W + a.eps);
    const float m = block_sum(pg, sm) / (float)a.W * rstd;
    for (int c = threadIdx.x; c < a.W; c += kThreads) {
      const float yv = to_f32(y[c]), zv = to_f32(z[c]), d = to_f32(dout[c]);
      const float s = 1.0f / (1.0f + expf(-zv)), act = zv * s;
      const float gh = yv * act * rstd;
      const float dg = rstd * (d * w[c] - gh * m);
      part[c] += d * gh;
      reinterpret_cast<T*>(a.dy)[o + c] = to_io<T>(dg * act);
      reinterpret_cast<T*>(a.dz)[row * a.dz_stride + c0 + c] =
          to_io<T>(dg * yv * s * (1.0f + zv * (1.0f - s)));
    }
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_quantize_q8(const T* v, int32_t K, int32_t Kp,
                                                          int8_t* q, float* qscale) {
  __shared__ float sm[kThreads / 64];
  v += (int64_t)blockIdx.x * K;
  q += (int64_t)blockIdx.x * Kp;
  float m = 0.0f;
  for (int c = threadIdx.x; c < K; c += kThreads) m = max_nan(fabsf(to_f32(v[c])), m);
  const Q8Scale s = q8_scale(block_max(m, sm));
  if (threadIdx.x == 0) qscale[blockIdx.x] = s.scale;
  for (int c = threadIdx.x; c < Kp; c += kThreads) q[c] = c < K ? q8_of(to_f32(v[c]), s) : 0;
}

hipError_t sum_parts(const float* part, float* out, int64_t parts, int64_t D, hipStream_t s) {
  hipLaunchKernelGGL(k_sum_parts, dim3((unsigned)((D + kThreads - 1) / kThreads)), dim3(kThreads),
                     0, s, part, out, parts, D);
  return hipGetLastError();
}

}  // namespace

int64_t add_norm_backward_parts(int64_t R, int64_t D) { return R < kParts ? R : kParts; }
int64_t gated_norm_backward_parts(int64_t R, int64_t G, int64_t W) { return R < kParts ? R : kParts; }

hipError_t launch_add_norm(const AddNormArgs& a, bool io_bf16, hipStream_t s) {
  const dim3 grid((unsigned)a.R), block(kThreads);
  if (io_bf16) hipLaunchKernelGGL(k_add_norm<bf16>, grid, block, 0, s, a);
  else hipLaunchKernelGGL(k_add_norm<float>, grid, block, 0, s, a);
  return hipGetLastError();
}

hipError_t launch_add_norm_backward(const AddNormArgs& a, bool io_bf16, hipStream_t s) {
  const int64_t parts = add_norm_backward_parts(a.R, a.D);
  const dim3 grid((unsigned)parts), block(kThreads);
  if (io_bf16) hipLaunchKernelGGL(k_add_norm_backward<bf16>, grid, block, 0, s, a);
  else hipLaunchKernelGGL(k_add_norm_backward<float>, grid, block, 0, s, a);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? e : sum_parts(a.part, a.dweight, parts, a.D, s);
}

hipError_t launch_gated_norm(const GatedNormArgs& a, bool io_bf16, hipStream_t s) {
  const dim3 grid((unsigned)a.R), block(kThreads);
  if (io_bf16) hipLaunchKernelGGL(k_gated_norm<bf16>, grid, block, 0, s, a);
  else hipLaunchKernelGGL(k_gated_norm<float>, grid, block, 0, s, a);
  return hipGetLastError();
}

hipError_t launch_gated_norm_backward(const GatedNormArgs& a, bool io_bf16, hipStream_t s) {
  const int64_t parts = gated_norm_backward_parts(a.R, a.G, a.W);
  const dim3 grid((unsigned)parts, (unsigned)a.G), block(kThreads);
  if (io_bf16) hipLaunchKernelGGL(k_gated_norm_backward<bf16>, grid, block, 0, s, a);
  else hipLaunchKernelGGL(k_gated_norm_backward<float>, grid, block, 0, s, a);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? e : sum_parts(a.part, a.dweight, parts, a.D, s);
}

hipError_t launch_quantize_q8(const void* v, bool v_bf16, int64_t R, int32_t K, int32_t Kp,
                              int8_t* q, float* qscale, hipStream_t s) {
  const dim3 grid((unsigned)R), block(kThreads);
  if (v_bf16)
    hipLaunchKernelGGL(k_quantize_q8<bf16>, grid, block, 0, s, static_cast<const bf16*>(v), K, Kp, q,
                       qscale);
  else
    hipLaunchKernelGGL(k_quantize_q8<float>, grid, block, 0, s, static_cast<const float*>(v), K, Kp,
                       q, qscale);
  return hipGetLastError();
}

}  // namespace ssd
