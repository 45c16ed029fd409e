// Building blocks of the row kernels (norms and the 8-bit quantiser): vectors
// of columns held in registers, and reductions over the lanes that share a row.
#pragma once

#include "ssd_device.h"

namespace ssd {

// N elements of T in a register, and the same in memory at the alignment of
// one element: rows of odd width or a sliced gate start anywhere, and global
// loads and stores of 16 bytes need no more than that on gfx950.
template <typename T, int N>
struct Pack {
  typedef T V __attribute__((ext_vector_type(N)));
  typedef V U __attribute__((aligned(sizeof(T))));
};
template <int N> using fvec = typename Pack<float, N>::V;

template <int N, typename T>
__device__ __forceinline__ typename Pack<T, N>::V load_pack(const T* p) {
  return *reinterpret_cast<const typename Pack<T, N>::U*>(p);
}
template <int N, typename T>
__device__ __forceinline__ void store_pack(T* p, typename Pack<T, N>::V v) {
  *reinterpret_cast<typename Pack<T, N>::U*>(p) = v;
}
template <typename To, int N, typename V>
__device__ __forceinline__ typename Pack<To, N>::V convert_pack(V v) {
  return __builtin_convertvector(v, typename Pack<To, N>::V);
}

// The columns of one row of width W that a lane holds: NV vectors of VEC
// columns, vector k at column VEC (k team + lane), where `team` lanes share
// the row.  A vector that would end beyond the row is moved back to the row's
// last VEC columns; its first `dup` columns then repeat another lane's (all of
// them, when dup >= VEC) and are left out of every sum.  Both lanes store the
// same values there, after a reduction that every lane's loads precede.  Only
// the last two vectors of a lane can be moved (the dispatch sees to it), and
// VEC <= W.
template <int VEC, int NV>
struct RowCols {
  int base[NV], dup[NV];
  __device__ __forceinline__ RowCols(int W, int team, int lane) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = VEC * (k * team + lane);
      base[k] = min(c, W - VEC);
      dup[k] = c - base[k];
    }
  }
  static constexpr bool may_move(int k) { return k + 2 >= NV; }
  __device__ __forceinline__ bool kept(int k) const { return !may_move(k) || dup[k] < VEC; }
  // v with the repeated columns zeroed
  __device__ __forceinline__ fvec<VEC> own(int k, fvec<VEC> v) const {
    if (may_move(k)) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = e < dup[k] ? 0.0f : v[e];
    }
    return v;
  }
};

template <int VEC>
__device__ __forceinline__ float sum_of(fvec<VEC> v) {
  float s = v[0];
#pragma unroll
  for (int e = 1; e < VEC; ++e) s += v[e];
  return s;
}

// ---------------------------------------------------------------------------
// Reductions over a wavefront: data-parallel moves within the rows of 16
// lanes, then the four row results through scalar registers.
// ---------------------------------------------------------------------------
template <int CTRL>
__device__ __forceinline__ int dpp_int(int v) {
  return __builtin_amdgcn_mov_dpp(v, CTRL, 0xF, 0xF, false);
}
__device__ __forceinline__ float wave_sum(float v) {
  auto add = [&](int o) { v += __int_as_float(o); };
  add(dpp_int<0xB1>(__float_as_int(v)));   // quad_perm [1,0,3,2]
  add(dpp_int<0x4E>(__float_as_int(v)));   // quad_perm [2,3,0,1]
  add(dpp_int<0x141>(__float_as_int(v)));  // row_half_mirror
  add(dpp_int<0x140>(__float_as_int(v)));  // row_mirror
  auto lane = [&](int l) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
  };
  return (lane(0) + lane(16)) + (lane(32) + lane(48));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, (uint32_t)dpp_int<0xB1>((int)v));
  v = max(v, (uint32_t)dpp_int<0x4E>((int)v));
  v = max(v, (uint32_t)dpp_int<0x141>((int)v));
  v = max(v, (uint32_t)dpp_int<0x140>((int)v));
  auto lane = [&](int l) { return (uint32_t)__builtin_amdgcn_readlane((int)v, l); };
  return max(max(lane(0), lane(16)), max(lane(32), lane(48)));
}

// Reductions over the lanes that share a row: one wavefront, or the whole
// workgroup (BLOCK) through `sm`, one slot of kMaxWaves per reduction.  A slot
// is written again two barriers after it was read at the earliest, as long as
// a caller alternates between two slots.
constexpr int kMaxWaves = 16;
template <bool BLOCK>
__device__ __forceinline__ float team_sum(float v, float* sm) {
  v = wave_sum(v);
  if constexpr (BLOCK) {
    if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = v;
    __syncthreads();
    v = sm[0];
    for (int w = 1; w < (int)(blockDim.x >> 6); ++w) v += sm[w];
  }
  return v;
}
template <bool BLOCK>
__device__ __forceinline__ void team_sum2(float& a, float& b, float* sm) {
  a = wave_sum(a);
  b = wave_sum(b);
  if constexpr (BLOCK) {
    float2* s2 = reinterpret_cast<float2*>(sm);
    if ((threadIdx.x & 63) == 0) s2[threadIdx.x >> 6] = make_float2(a, b);
    __syncthreads();
    float2 t = s2[0];
    for (int w = 1; w < (int)(blockDim.x >> 6); ++w) {
      const float2 o = s2[w];
      t.x += o.x;
      t.y += o.y;
    }
    a = t.x;
    b = t.y;
  }
}
template <bool BLOCK>
__device__ __forceinline__ uint32_t team_max(uint32_t v, float* sm) {
  v = wave_max(v);
  if constexpr (BLOCK) {
    uint32_t* su = reinterpret_cast<uint32_t*>(sm);
    if ((threadIdx.x & 63) == 0) su[threadIdx.x >> 6] = v;
    __syncthreads();
    v = su[0];
    for (int w = 1; w < (int)(blockDim.x >> 6); ++w) v = max(v, su[w]);
  }
  return v;
}

// ---------------------------------------------------------------------------
// Elementwise pieces
// ---------------------------------------------------------------------------
// logistic(z) = 1 / (1 + 2^(-z log2 e)) on the hardware base-2 exponential and
// reciprocal.  Large negative z: 2^(+big) = inf and the result is 0.
__device__ __forceinline__ float logistic(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-z * kLog2e));
}

// 8-bit rows: magnitudes are compared as integers, where an infinity and
// every NaN lie above all finite values, so that neither is lost in a maximum.
struct Q8Row {
  float inv, scale;
  // from the row's largest magnitude
  __device__ __forceinline__ explicit Q8Row(uint32_t amax_bits) {
    const float a = __uint_as_float(amax_bits);
    const bool finite = amax_bits < 0x7F800000u, none = a < 0x1p-100f;
    inv = finite && !none ? 127.0f / a : 0.0f;
    scale = !finite ? __uint_as_float(0x7FC00000u) : none ? 0.0f : a / 127.0f;
  }
  // NaN only where inv is 0 and v is not finite; the clamp's order sends it to
  // -127 or 127, so such rows are zeroed by the caller's inv == 0 test
  __device__ __forceinline__ int8_t operator()(float v) const {
    return inv == 0.0f ? (int8_t)0 : (int8_t)(int)fminf(fmaxf(rintf(v * inv), -127.0f), 127.0f);
  }
};
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

template <int VEC>
__device__ __forceinline__ void store_q8(int8_t* p, fvec<VEC> v, const Q8Row& s) {
  typename Pack<int8_t, VEC>::V q;
#pragma unroll
  for (int e = 0; e < VEC; ++e) q[e] = s(v[e]);
  store_pack<VEC>(p, q);
}

}  // namespace ssd
