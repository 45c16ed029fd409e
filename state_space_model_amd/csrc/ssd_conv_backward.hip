// Gradients of the depthwise causal convolution for gfx950.
//
// With xp the cached window followed by x, z[t] = bias + sum_i w[i] xp[t+i]
// (recomputed) and dz[t] = dy[t] act'(z[t]):
//   dxp[u] = sum_i w[i] dz[u-i];  dx[t] = dxp[t+k-1];  dstate[j] = dxp[j]
//   dw[i]  = sum_{b,t} dz[t] xp[t+i];  dbias = sum_{b,t} dz[t]
#include "ssd_device.h"
#include "ssd_launch.h"

namespace ssd {
namespace {

constexpr int kThreads = 64;

// lane -> channel, block y -> batch row: the whole sequence in order
template <typename T, typename TG, int K>
__global__ __launch_bounds__(kThreads) void k_conv_backward(ConvBwdArgs a) {
  const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (c >= a.D) return;
  const int64_t b = blockIdx.y;
  const T* x = reinterpret_cast<const T*>(a.x) + b * a.T * a.D + c;
  const TG* dy = reinterpret_cast<const TG*>(a.dy) + b * a.T * a.D + c;
  T* dx = reinterpret_cast<T*>(a.dx) + b * a.T * a.D + c;
  const int64_t so = (b * a.D + c) * (K - 1);
  const T* win = reinterpret_cast<const T*>(a.state_in);
  const T* dso = reinterpret_cast<const T*>(a.dstate_out);
  float w[K], xp[K], dxp[K], dw[K], db = 0.0f;
  const float bias = a.bias ? a.bias[c] : 0.0f;
#pragma unroll
  for (int i = 0; i < K; ++i) {
    w[i] = a.w[c * K + i];
    dw[i] = 0.0f;
    dxp[i] = 0.0f;
    xp[i] = (i < K - 1 && win) ? to_f32(win[so + i]) : 0.0f;
  }
  // position u = t of xp leaves the window after token t
  auto put = [&](int64_t u, float v) {
    if (u >= a.T && dso) v += to_f32(dso[so + u - a.T]);
    if (u >= K - 1) dx[(u - (K - 1)) * a.D] = to_io<T>(v);
    else if (a.dstate) reinterpret_cast<T*>(a.dstate)[so + u] = to_io<T>(v);
  };
  for (int64_t t = 0; t < a.T; ++t) {
    xp[K - 1] = to_f32(x[t * a.D]);
    float z = bias;
#pragma unroll
    for (int i = 0; i < K; ++i) z = __fmaf_rn(w[i], xp[i], z);
    float dz = to_f32(dy[t * a.D]);
    if (a.silu) {
      const float s = 1.0f / (1.0f + expf(-z));
      dz *= s * (1.0f + z * (1.0f - s));
    }
    db += dz;
#pragma unroll
    for (int i = 0; i < K; ++i) {
      dw[i] = __fmaf_rn(dz, xp[i], dw[i]);
      dxp[i] = __fmaf_rn(w[i], dz, dxp[i]);
    }
    put(t, dxp[0]);
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
      xp[i] = xp[i + 1];
      dxp[i] = dxp[i + 1];
    }
    dxp[K - 1] = 0.0f;
  }
#pragma unroll
  for (int i = 0; i < K - 1; ++i) put(a.T + i, dxp[i]);
  float* part = a.part + b * (K + 1) * a.D + c;
#pragma unroll
  for (int i = 0; i < K; ++i) part[i * a.D] = dw[i];
  part[K * a.D] = db;
}

// parts [parts][K+1][D] -> dw [D][K], dbias [D]
__global__ __launch_bounds__(kThreads) void k_conv_sum_parts(ConvBwdArgs a, int64_t parts) {
  const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (c >= a.D) return;
  const int i = blockIdx.y;
  float s = 0.0f;
  for (int64_t p = 0; p < parts; ++p) s += a.part[(p * (a.K + 1) + i) * a.D + c];
  if (i < a.K) a.dw[c * a.K + i] = s;
  else if (a.dbias) a.dbias[c] = s;
}

// seqlen == 0: the window's gradient is handed on
template <typename T>
__global__ __launch_bounds__(kThreads) void k_conv_hand_on(const T* src, T* dst, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i < n) dst[i] = src ? src[i] : to_io<T>(0.0f);
}

template <typename T, typename TG>
hipError_t launch_t(const ConvBwdArgs& a, hipStream_t s) {
  const unsigned blocks = (unsigned)((a.D + kThreads - 1) / kThreads);
  const int64_t parts = conv_backward_parts(a.Bt, a.T, a.D);
  if (parts > 0) {
    const dim3 grid(blocks, (unsigned)a.Bt), block(kThreads);
    if (a.K == 2) hipLaunchKernelGGL((k_conv_backward<T, TG, 2>), grid, block, 0, s, a);
    else if (a.K == 3) hipLaunchKernelGGL((k_conv_backward<T, TG, 3>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_conv_backward<T, TG, 4>), grid, block, 0, s, a);
    if (hipGetLastError() != hipSuccess) return hipErrorLaunchFailure;
  } else if (a.dstate && a.Bt > 0) {
    const int64_t n = a.Bt * a.D * (a.K - 1);
    hipLaunchKernelGGL(k_conv_hand_on<T>, dim3((unsigned)((n + kThreads - 1) / kThreads)),
                       dim3(kThreads), 0, s, reinterpret_cast<const T*>(a.dstate_out),
                       reinterpret_cast<T*>(a.dstate), n);
    if (hipGetLastError() != hipSuccess) return hipErrorLaunchFailure;
  }
  hipLaunchKernelGGL(k_conv_sum_parts, dim3(blocks, (unsigned)a.K + 1), dim3(kThreads), 0, s, a,
                     parts);
  return hipGetLastError();
}

}  // namespace

int64_t conv_backward_parts(int64_t Bt, int64_t T, int64_t D) { return T > 0 ? Bt : 0; }

hipError_t launch_conv_backward(const ConvBwdArgs& a, bool io_bf16, bool dy_bf16, hipStream_t s) {
  if (!io_bf16) return launch_t<float, float>(a, s);
  return dy_bf16 ? launch_t<bf16, bf16>(a, s) : launch_t<bf16, float>(a, s);
}

}  // namespace ssd
