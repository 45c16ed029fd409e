// What the kernels of the gated delta rule share (ssd_delta.hip: the scan and
// the step; ssd_delta_backward.hip: the gradients): float32 matrix products on
// the bfloat16 matrix cores, and the layout of the chunks' workspace.
//
// Products.  A float32 number is the exact sum of three bfloat16 numbers of 8
// significant bits each ("planes": h, m, l).  A product of two such
// operands is formed from the plane products whose indices add to at most 2
// (hh, hm, mh, hl, mm, lh; the rest is below 2^-26 of it), each exact in the
// matrix core and accumulated in float32: six v_mfma_f32_16x16x32_bf16 (16
// cycles each) where v_mfma_f32_16x16x4_f32 takes eight of 32 cycles.  An
// operand that is bfloat16 already is one plane, and its product with a
// float32 operand is exact up to the sum with three.  So states, writes and
// their gradients keep float32 accuracy for both io types; only what ends in a
// bfloat16 output is formed from two planes (2^-17 of it, against 2^-8 by the
// rounding of the output).
#pragma once

#include "ssd_device.h"
#include "ssd_launch.h"

namespace ssd {
namespace delta {

constexpr int C = kDeltaChunk;     // tokens of a chunk
constexpr int kThreads = 256;      // four wavefronts; wavefront w owns tokens 16 w .. 16 w + 15
constexpr int kTokStride = C + 8;  // LDS rows of C token-contiguous bfloat16
constexpr int kPairStride = C + 4; // LDS rows of C float32
// Fragments of a triangular [C, C] operand: 16-row tiles x 32-column steps
// that hold anything.  Lower: row tiles 0, 1 need columns 0-31 only; upper:
// row tiles 2, 3 need columns 32-63 only.
constexpr int kTriFrags = 6;
constexpr int kFrag = 512;         // elements of one fragment: 8 per lane

template <typename IO> struct Planes;
template <> struct Planes<float> { static constexpr int in = 3, y = 3; };
template <> struct Planes<bf16> { static constexpr int in = 1, y = 2; };

template <int NP> struct Frag { bf16x8 p[NP]; };

__device__ __forceinline__ f32x4 mma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// acc += A B over the plane products that count, the smallest first
template <int NA, int NB>
__device__ __forceinline__ f32x4 mma(const Frag<NA>& a, const Frag<NB>& b, f32x4 acc) {
  constexpr int top = (NA > NB ? NA : NB) - 1;
#pragma unroll
  for (int s = top; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (s - i >= 0 && s - i < NB) acc = mma(a.p[i], b.p[s - i], acc);
  return acc;
}

// The planes of a pair, plane by plane in one word.  Each is rounded to nearest
// (v_cvt_pk_bf16_f32), so what the dropped products leave out has no sign of its
// own; the remainders are exact.  An infinity or a NaN leaves NaN behind.
struct Split2 {
  uint32_t p[3];
  __device__ __forceinline__ Split2(float a, float b) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
      p[i] = __builtin_bit_cast(uint32_t, bf16x2{(bf16)a, (bf16)b});
      a -= __uint_as_float(p[i] << 16);
      b -= __uint_as_float(p[i] & 0xFFFF0000u);
    }
  }
};

// 8 float32 values as a fragment of NP planes
template <int NP>
__device__ __forceinline__ Frag<NP> split8(const float (&x)[8]) {
  const Split2 a(x[0], x[1]), b(x[2], x[3]), c(x[4], x[5]), d(x[6], x[7]);
  Frag<NP> f;
#pragma unroll
  for (int i = 0; i < NP; ++i)
    f.p[i] = __builtin_bit_cast(bf16x8, make_uint4(a.p[i], b.p[i], c.p[i], d.p[i]));
  return f;
}

// 4 consecutive values to NP planes `plane` elements apart (8-byte stores)
template <int NP>
__device__ __forceinline__ void store_split4(bf16* p, int plane, f32x4 v) {
  const Split2 a(v[0], v[1]), b(v[2], v[3]);
#pragma unroll
  for (int i = 0; i < NP; ++i) *reinterpret_cast<uint2*>(p + i * plane) = make_uint2(a.p[i], b.p[i]);
}

__device__ __forceinline__ bf16x8 ld8(const bf16* p) { return *reinterpret_cast<const bf16x8*>(p); }

template <int NP>
__device__ __forceinline__ Frag<NP> load_planes(const bf16* p, int plane) {
  Frag<NP> f;
#pragma unroll
  for (int i = 0; i < NP; ++i) f.p[i] = ld8(p + i * plane);
  return f;
}

// 8 consecutive io elements of a row as a fragment (16-byte loads), zeros when
// !ok; `p` is a valid address either way.
template <typename IO>
__device__ __forceinline__ Frag<Planes<IO>::in> load_io8(const IO* p, bool ok) {
  if constexpr (sizeof(IO) == 2) {
    uint4 v = *reinterpret_cast<const uint4*>(p);
    v.x = ok ? v.x : 0u; v.y = ok ? v.y : 0u; v.z = ok ? v.z : 0u; v.w = ok ? v.w : 0u;
    Frag<1> f;
    f.p[0] = __builtin_bit_cast(bf16x8, v);
    return f;
  } else {
    const float4 lo = *reinterpret_cast<const float4*>(p);
    const float4 hi = *reinterpret_cast<const float4*>(p + 4);
    const float x[8] = {ok ? lo.x : 0.f, ok ? lo.y : 0.f, ok ? lo.z : 0.f, ok ? lo.w : 0.f,
                        ok ? hi.x : 0.f, ok ? hi.y : 0.f, ok ? hi.z : 0.f, ok ? hi.w : 0.f};
    return split8<3>(x);
  }
}

// ds_read_b64_tr_b16: within each group of 16 lanes, lane j addresses 4
// elements and receives element j % 4 of the vectors addressed by lanes j / 4,
// 4 + j / 4, 8 + j / 4 and 12 + j / 4.
typedef short s16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ bf16x4 lds_read_tr4(const bf16* p) {
  const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) s16x4*)(const_cast<bf16*>(p)));
  return __builtin_bit_cast(bf16x4, v);
}
// The operand that contracts over the rows of a row-major LDS tile: lane j of
// group q gets m[r0 + 8 q .. + 7][c0 + j].
template <int NP>
__device__ __forceinline__ Frag<NP> load_planes_tr(const bf16* m, int plane, int stride, int r0,
                                                   int c0, int lane) {
  const int j = lane & 15, q = lane >> 4;
  const bf16* p = m + (r0 + 8 * q + (j >> 2)) * stride + c0 + 4 * (j & 3);
  Frag<NP> f;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const bf16x4 lo = lds_read_tr4(p + i * plane), hi = lds_read_tr4(p + i * plane + 4 * stride);
    f.p[i] = bf16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  }
  return f;
}

// A 16 x 16 float32 product on the float32 matrix core, its right operand and
// result in the register layout of a result: lane l holds rows 4 (l / 16) + r
// of column l % 16.  Slot s of lane group q is contraction index 4 q + s, so
// the right operand's registers are used as they are and the left one's row is
// one 16-byte vector, `a` = A[l % 16][4 (l / 16) .. + 3].
__device__ __forceinline__ f32x4 mma16(f32x4 a, f32x4 b, f32x4 acc) {
#pragma unroll
  for (int s = 0; s < 4; ++s)
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[s], b[s], acc, 0, 0, 0);
  return acc;
}

__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

// 1 / (1 + e^-z), also for -infinity (0)
__device__ __forceinline__ float sigmoid_of(float z) {
  return 1.0f / (1.0f + exp2_of(-z * kLog2e));
}

// Wavefront w holds tokens 16 w .. + 15 of k and q as matrix operands: row
// lane % 16, key columns 32 s + 8 (lane / 16) .. + 7 of step s.
template <typename IO, int KP>
__device__ __forceinline__ void load_rows(Frag<Planes<IO>::in> (&f)[KP / 32], const void* base,
                                          int64_t stride, int64_t row0, int64_t left, int N, int r,
                                          int q) {
  const bool in = r < left;   // token r of the chunk that starts at row0
  const IO* row = static_cast<const IO*>(base) + (row0 + (in ? r : 0)) * stride;
#pragma unroll
  for (int s = 0; s < KP / 32; ++s) {
    const int col = 32 * s + 8 * q;
    f[s] = load_io8<IO>(row + (col < N ? col : 0), in && col < N);
  }
}

// Where the 32 columns from 32 s on of row tile w are among a triangular
// operand's fragments, and these in the workspace
__device__ __forceinline__ int lower_frag(int w, int s) { return w < 2 ? w : 2 * w - 2 + s; }
__device__ __forceinline__ int upper_frag(int w, int s) { return w < 2 ? 2 * w + s : w + 2; }
template <int NP>
__device__ __forceinline__ void store_frag(bf16* base, int64_t at, int f, int lane, const Frag<NP>& v) {
#pragma unroll
  for (int i = 0; i < NP; ++i)
    *reinterpret_cast<bf16x8*>(base + ((at * NP + i) * kTriFrags + f) * kFrag + lane * 8) = v.p[i];
}
template <int NP>
__device__ __forceinline__ Frag<NP> load_frag(const bf16* base, int64_t at, int f, int lane) {
  return load_planes<NP>(base + (at * NP * kTriFrags + f) * kFrag + lane * 8, kTriFrags * kFrag);
}

// State tiles of a chain's wavefront to [P, N]: keys 16 (KT w + t) + 4 q .. + 3
// of value column col[n]
template <int NT, int KT>
__device__ __forceinline__ void store_state(float* to, const f32x4 (&st)[NT][KT], int N,
                                            const int (&col)[NT], const bool (&col_in)[NT], int w,
                                            int q) {
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const int key = 16 * (KT * w + t) + 4 * q;
      if (col_in[n] && key < N)
        *reinterpret_cast<f32x4*>(to + (int64_t)col[n] * N + key) = st[n][t];
    }
}

// sum over a wavefront
__device__ __forceinline__ float wave_sum64(float v) {
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// Position of a (b, h, chunk)
__device__ __forceinline__ int64_t chunk_at(const DeltaArgs& a, int64_t bh, int64_t c) {
  return bh * a.Nc + c;
}

}  // namespace delta
}  // namespace ssd
