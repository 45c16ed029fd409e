// Product of 8-bit rows on the integer matrix cores of gfx950:
//   out[m][n] = sx[m] sw[n] sum_k x[m][k] w[n][k]
//
// v_mfma_i32_16x16x64_i8 contracts 64 columns: lane l holds 16 adjacent bytes
// of row l % 16 of each operand, columns 16 (l / 16) ..., and register r of
// lane l is element [4 (l / 16) + r][l % 16] of the product, as for the
// float matrix instructions.  The sum is exact, so its order is free.
#include "ssd_device.h"
#include "ssd_launch.h"

namespace ssd {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// one wavefront per 16 x 16 tile
template <typename T>
__global__ __launch_bounds__(64) void k_linear_q8(LinearQ8Args a, int64_t nt) {
  const int l = threadIdx.x, i = l & 15, g = l >> 4;
  const int64_t m0 = (int64_t)(blockIdx.x / nt) * 16, n0 = (int64_t)(blockIdx.x % nt) * 16;
  const int64_t m = m0 + i < a.M ? m0 + i : a.M - 1, n = n0 + i < a.N ? n0 + i : a.N - 1;
  const int8_t* x = a.q + m * a.K + g * 16;
  const int8_t* w = a.wq + n * a.K + g * 16;
  i32x4 acc = {0, 0, 0, 0};
  for (int k = 0; k < a.K; k += 64)
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(*reinterpret_cast<const i32x4*>(x + k),
                                                *reinterpret_cast<const i32x4*>(w + k), acc, 0, 0, 0);
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int64_t mm = m0 + 4 * g + r;
    if (mm < a.M && n0 + i < a.N)
      reinterpret_cast<T*>(a.out)[mm * a.N + n0 + i] =
          to_io<T>((float)acc[r] * a.wscale[n0 + i] * a.qscale[mm]);
  }
}

}  // namespace

hipError_t launch_linear_q8(const LinearQ8Args& a, bool out_bf16, hipStream_t s) {
  const int64_t nt = (a.N + 15) / 16, mt = (a.M + 15) / 16;
  const dim3 grid((unsigned)(nt * mt)), block(64);
  if (out_bf16) hipLaunchKernelGGL(k_linear_q8<bf16>, grid, block, 0, s, a, nt);
  else hipLaunchKernelGGL(k_linear_q8<float>, grid, block, 0, s, a, nt);
  return hipGetLastError();
}

}  // namespace ssd
