// Gradients of the depthwise causal convolution for gfx950.
//
// With xp the cached window followed by x, z[t] = bias + sum_i w[i] xp[t+i]
// (recomputed) and dz[t] = dy[t] act'(z[t]):
//   dxp[u] = sum_i w[i] dz[u-i];  dx[t] = dxp[t+k-1];  dstate[j] = dxp[j]
//   dw[i]  = sum_{b,t} dz[t] xp[t+i];  dbias = sum_{b,t} dz[t]
//
// Some 40 operations per element moved (most of them the slope of silu): the
// layer is bound by memory when they are spread well.  A thread owns VEC
// adjacent channels and walks a run of tokens with the window of k inputs and
// k pending sums of dxp in registers; the next tokens' rows are requested a
// batch ahead.  A run starts k-1 tokens early (their dz feed its first dx) and
// the weight's gradient counts only the run's own tokens; the runs' sums are
// added by a second launch.
//
// Measured (kernel time in a HIP graph, inputs rotated through HBM): 4096 x 5376
// bfloat16 with float32 dy 42 us, 38 to 40 of them the first launch (4.9 TB/s
// with the tokens read twice); 3 x 1001 x 1793 float32 with a window 22-23 us.
// Four channels per lane (164 registers, three wavefronts per SIMD, 1.9
// resident on average) took 46-49 us however the runs were split, eight tokens
// per batch 46-65 us, and runs shared out over the wavefronts of a workgroup
// (their rows apart) 46 us: what counts is that neighbouring wavefronts read
// neighbouring columns of the same rows and that enough of them are resident.
#include <type_traits>

#include "ssd_launch.h"
#include "ssd_rows.h"

namespace ssd {
namespace {

constexpr int kThreads = 256;
constexpr int kVec = 2;   // channels per lane

// grid (ceil(NG / 256), runs, Bt): lane -> VEC channels, workgroup -> run of R
// tokens.  Where VEC does not divide D the last lane moves back to the
// last VEC channels and writes the values its neighbour writes.
template <typename T, typename TG, int K, int VEC>
__global__ __launch_bounds__(kThreads) void k_conv_backward(ConvBwdArgs a, int32_t NG, int64_t R) {
  constexpr int U = 4;   // tokens requested and worked on at a time
  typedef typename Pack<T, VEC>::V VT;
  typedef typename Pack<TG, VEC>::V VG;
  typedef fvec<VEC> F;
  const int32_t g = (int32_t)blockIdx.x * kThreads + threadIdx.x;
  const bool live = g < NG;
  const int64_t c0 = g * VEC + VEC <= a.D ? g * VEC : a.D - VEC;
  const int64_t b = blockIdx.z, run = blockIdx.y;
  const int64_t t0 = run * R, t1 = t0 + R < a.T ? t0 + R : a.T;
  const T* x = reinterpret_cast<const T*>(a.x) + b * a.T * a.D + c0;
  const TG* dy = reinterpret_cast<const TG*>(a.dy) + b * a.T * a.D + c0;
  T* dx = reinterpret_cast<T*>(a.dx) + b * a.T * a.D + c0;
  const int64_t so = (b * a.D + c0) * (K - 1);
  const T* win = reinterpret_cast<const T*>(a.state_in);
  const T* dso = reinterpret_cast<const T*>(a.dstate_out);
  F w[K], dw[K], db = F(0.0f), bias;
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
#pragma unroll
    for (int i = 0; i < K; ++i) w[i][v] = a.w[(c0 + v) * K + i];
    bias[v] = a.bias ? a.bias[c0 + v] : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < K; ++i) dw[i] = F(0.0f);
  // xp[u], u < K-1: the window; beyond, x
  auto input = [&](int64_t u) {
    F f;
    if (u >= K - 1) {
      f = convert_pack<float, VEC>(load_pack<VEC>(x + (u - (K - 1)) * a.D));
    } else {
#pragma unroll
      for (int v = 0; v < VEC; ++v) f[v] = win ? to_f32(win[so + v * (K - 1) + u]) : 0.0f;
    }
    return f;
  };
  // the finished sum of position u of xp
  auto put = [&](int64_t u, F s) {
    if (!live) return;
    if (u >= a.T && dso) {
#pragma unroll
      for (int v = 0; v < VEC; ++v) s[v] += to_f32(dso[so + v * (K - 1) + u - a.T]);
    }
    if (u >= K - 1) {
      store_pack<VEC>(dx + (u - (K - 1)) * a.D, convert_pack<T, VEC>(s));
    } else if (a.dstate) {
#pragma unroll
      for (int v = 0; v < VEC; ++v)
        reinterpret_cast<T*>(a.dstate)[so + v * (K - 1) + u] = to_io<T>(s[v]);
    }
  };
  if (t0 < t1) {
    // Positions [t0, t1) of xp belong to this run, the last run's also
    // [T, T+K-1).  xs[j], xs[j+1], ... are token t+j's taps, ps[j] the sum of
    // dxp at position t+j.
    F xs[U + K - 1], ps[U + K - 1];
    // dz of token t + j, added to its positions' sums
    auto point = [&](int j, F dz) {
      F z = bias;
#pragma unroll
      for (int i = 0; i < K; ++i) z += w[i] * xs[j + i];
      if (a.silu) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          const float s = logistic(z[v]), act = z[v] * s;
          dz[v] *= s + act * (1.0f - s);
        }
      }
#pragma unroll
      for (int i = 0; i < K - 1; ++i) ps[j + i] += w[i] * dz;
      ps[j + K - 1] = w[K - 1] * dz;
      return dz;
    };
    auto count = [&](int j, F dz) {
      db += dz;
#pragma unroll
      for (int i = 0; i < K; ++i) dw[i] += dz * xs[j + i];
    };
    // the window moves on by n tokens
    auto advance = [&](int n) {
#pragma unroll
      for (int i = 0; i < K - 1; ++i) {
        xs[i] = xs[i + n];
        ps[i] = ps[i + n];
      }
    };
#pragma unroll
    for (int i = 0; i < K - 1; ++i) ps[i] = F(0.0f);
    // the K-1 tokens before the run feed its first positions only
    if (t0 > 0) {
#pragma unroll
      for (int i = 0; i < K - 1; ++i) xs[i] = input(t0 - (K - 1) + i);
#pragma unroll
      for (int h = 0; h < K - 1; ++h) {
        const int64_t t = t0 - (K - 1) + h;      // R >= K-1: never before token 0
        xs[K - 1] = convert_pack<float, VEC>(load_pack<VEC>(x + t * a.D));
        point(0, convert_pack<float, VEC>(load_pack<VEC>(dy + t * a.D)));
        advance(1);
      }
    } else {
#pragma unroll
      for (int i = 0; i < K - 1; ++i) xs[i] = input(i);
    }
    VT xr[U];
    VG gr[U];
    auto fetch = [&](int64_t t) {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int64_t r = (t + j < t1 ? t + j : t1 - 1) * a.D;
        xr[j] = load_pack<VEC>(x + r);
        gr[j] = load_pack<VEC>(dy + r);
      }
    };
    fetch(t0);
    int64_t t = t0;
    for (; t + U <= t1; t += U) {
      F gf[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        xs[K - 1 + j] = convert_pack<float, VEC>(xr[j]);
        gf[j] = convert_pack<float, VEC>(gr[j]);
      }
      fetch(t + U);
#pragma unroll
      for (int j = 0; j < U; ++j) count(j, point(j, gf[j]));
      if (t >= K - 1) {
        if (live) {
#pragma unroll
          for (int j = 0; j < U; ++j)
            store_pack<VEC>(dx + (t + j - (K - 1)) * a.D, convert_pack<T, VEC>(ps[j]));
        }
      } else {
#pragma unroll
        for (int j = 0; j < U; ++j) put(t + j, ps[j]);
      }
      advance(U);
    }
    for (int left = (int)(t1 - t), j0 = 0; j0 < left; ++j0, ++t) {
      VT xt = xr[0];
      VG gt = gr[0];
#pragma unroll
      for (int j = 1; j < U - 1; ++j)
        if (j == j0) xt = xr[j], gt = gr[j];
      xs[K - 1] = convert_pack<float, VEC>(xt);
      count(0, point(0, convert_pack<float, VEC>(gt)));
      put(t, ps[0]);
      advance(1);
    }
    if (t1 == a.T) {
#pragma unroll
      for (int i = 0; i < K - 1; ++i) put(a.T + i, ps[i]);
    }
  }
  if (!live) return;
  // the run's part of dw and dbias: [part][K+1][D]
  float* part = a.part + (b * gridDim.y + blockIdx.y) * (K + 1) * a.D + c0;
#pragma unroll
  for (int i = 0; i <= K; ++i) {
    store_pack<VEC>(part + i * a.D, i < K ? dw[i < K ? i : 0] : db);
  }
}

// parts [parts][K+1][D] -> dw [D][K], dbias [D]: 64 channels per workgroup, its
// SPLIT wavefronts take parts in turn, then their sums are added in order
constexpr int SPLIT = 8;
__global__ __launch_bounds__(64 * SPLIT) void k_conv_sum_parts(ConvBwdArgs a, int32_t parts) {
  __shared__ float sm[SPLIT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = blockIdx.y;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (c < a.D) {
#pragma unroll 8
    for (int p = wave; p < parts; p += SPLIT) s += a.part[((int64_t)p * (a.K + 1) + i) * a.D + c];
  }
  sm[wave][lane] = s;
  __syncthreads();
  if (wave != 0 || c >= a.D) return;
#pragma unroll
  for (int o = 1; o < SPLIT; ++o) s += sm[o][lane];
  if (i < a.K) a.dw[c * a.K + i] = s;
  else if (a.dbias) a.dbias[c] = s;
}

// seqlen == 0: the window's gradient is handed on
template <typename T>
__global__ __launch_bounds__(kThreads) void k_conv_hand_on(const T* src, T* dst, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i < n) dst[i] = src ? src[i] : to_io<T>(0.0f);
}

// How the tokens are split: `groups` runs of R tokens along time, the fewest
// that give three workgroups to a compute unit (five fit, at up to 92
// registers), each long against the k-1 tokens it reads twice.  All workgroups
// are resident at once up to 640 blocks of columns over the batch; between
// 641 and 767 the two runs of each are up to 1534 workgroups, a part of which
// waits.  With the quotient rounded down, at most three to a unit, 11 x 3000 x
// 1500 took 99 us against 109, 64 x 256 x 5376 153 against 164 and 4096 x 5376
// the same, but 26 x 512 x 5120 (two runs instead of three) 130 against 126 and
// 260 x 512 x 512 134 against 129.
struct Runs {
  int64_t R, groups;
};
Runs runs_of(int64_t Bt, int64_t T, int64_t D) {
  constexpr int64_t kResident = 3 * 256, kShortest = 24;
  const int64_t cols = (D + kThreads * kVec - 1) / (kThreads * kVec) * Bt;
  const int64_t groups = (kResident + cols - 1) / cols;
  const int64_t R = (T + groups - 1) / groups < kShortest ? kShortest : (T + groups - 1) / groups;
  return {R, (T + R - 1) / R};
}

template <typename T, typename TG, int VEC>
hipError_t launch_v(const ConvBwdArgs& a, hipStream_t s) {
  const Runs r = runs_of(a.Bt, a.T, a.D);
  const int32_t NG = (int32_t)((a.D + VEC - 1) / VEC);
  const dim3 grid((unsigned)((NG + kThreads - 1) / kThreads), (unsigned)r.groups, (unsigned)a.Bt), block(kThreads);
  if (a.K == 2) hipLaunchKernelGGL((k_conv_backward<T, TG, 2, VEC>), grid, block, 0, s, a, NG, r.R);
  else if (a.K == 3) hipLaunchKernelGGL((k_conv_backward<T, TG, 3, VEC>), grid, block, 0, s, a, NG, r.R);
  else hipLaunchKernelGGL((k_conv_backward<T, TG, 4, VEC>), grid, block, 0, s, a, NG, r.R);
  return hipGetLastError();
}

template <typename T, typename TG>
hipError_t launch_t(const ConvBwdArgs& a, hipStream_t s) {
  const int64_t parts = conv_backward_parts(a.Bt, a.T, a.D);
  if (parts > 0) {
    const hipError_t e = a.D >= kVec ? launch_v<T, TG, kVec>(a, s) : launch_v<T, TG, 1>(a, s);
    if (e != hipSuccess) return e;
  } else if (a.dstate && a.Bt > 0) {
    const int64_t n = a.Bt * a.D * (a.K - 1);
    hipLaunchKernelGGL(k_conv_hand_on<T>, dim3((unsigned)((n + kThreads - 1) / kThreads)),
                       dim3(kThreads), 0, s, reinterpret_cast<const T*>(a.dstate_out),
                       reinterpret_cast<T*>(a.dstate), n);
    if (hipGetLastError() != hipSuccess) return hipErrorLaunchFailure;
  }
  hipLaunchKernelGGL(k_conv_sum_parts, dim3((unsigned)((a.D + 63) / 64), (unsigned)a.K + 1),
                     dim3(64 * SPLIT), 0, s, a, (int32_t)parts);
  return hipGetLastError();
}

}  // namespace

// A grid's threads are counted in 32 bits: those of the sum of the parts and,
// for an empty sequence, of the window's gradient.
bool conv_backward_shape_supported(int64_t Bt, int64_t T, int64_t D, int64_t K) {
  const int64_t windows = Bt * D * (K - 1);
  return conv_shape_supported(Bt, T, D) && (D + 63) / 64 * (64 * SPLIT) <= UINT32_MAX &&
         (T > 0 || (windows + kThreads - 1) / kThreads * kThreads <= UINT32_MAX);
}

int64_t conv_backward_parts(int64_t Bt, int64_t T, int64_t D) {
  return Bt > 0 && T > 0 ? Bt * runs_of(Bt, T, D).groups : 0;
}

hipError_t launch_conv_backward(const ConvBwdArgs& a, bool io_bf16, bool dy_bf16, hipStream_t s) {
  if (!io_bf16) return launch_t<float, float>(a, s);
  return dy_bf16 ? launch_t<bf16, bf16>(a, s) : launch_t<bf16, float>(a, s);
}

}  // namespace ssd
