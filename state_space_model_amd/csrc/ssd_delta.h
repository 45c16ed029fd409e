// What the kernels of the gated delta rule share (ssd_delta.hip: the scan and
// the step; ssd_delta_backward.hip: the gradients): float32 matrix products on
// the bfloat16 matrix cores, and the layout of the chunks' workspace.
//
// Products.  A float32 number is the exact sum of three bfloat16 numbers of 8
// significant bits each ("planes": h, m, l), where none of them leaves bfloat16's
// range: a magnitude past its largest number, 3.39e38, becomes infinite, and below
// 2^-110 the last bits may be lost.  A product of two such
// operands is formed from the plane products whose indices add to at most 2
// (hh, hm, mh, hl, mm, lh; ml and lm, the most of the rest, are 2^-8 2^-17 of it
// each: 2^-24, half a step of float32), each exact in the
// matrix core and accumulated in float32: six v_mfma_f32_16x16x32_bf16 (16
// cycles each) where v_mfma_f32_16x16x4_f32 takes eight of 32 cycles.  An
// operand that is bfloat16 already is one plane, and its product with a
// float32 operand is exact up to the sum with three.  So states, writes, outputs
// and all gradients keep float32 accuracy for both io types, and a bfloat16
// output is rounded once, at its store.  (Outputs from two planes of the state,
// the writes and q k^T would take a tenth less, 225 against 245 us for 4096 tokens
// of 80 heads and 3210 against 3640 for 8 x 16384 of 64, and be off by up to 2^-15 of
// the terms' magnitudes.)
#pragma once

#include <type_traits>

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

template <typename IO> struct Planes;   // of an element of q, k or v
template <> struct Planes<float> { static constexpr int in = 3; };
template <> struct Planes<bf16> { static constexpr int in = 1; };

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

// acc[i] += A[i] B for independent tiles, plane product by plane product over
// all of them: a tile's next product depends on its last one, whose result takes
// longer than its issue
template <int NT, int NA, int NB>
__device__ __forceinline__ void mma_tiles(const Frag<NA> (&a)[NT], const Frag<NB>& b, f32x4* acc) {
  constexpr int top = (NA > NB ? NA : NB) - 1;
#pragma unroll
  for (int s = top; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (s - i >= 0 && s - i < NB)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[t] = mma(a[t].p[i], b.p[s - i], acc[t]);
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
      asm("" : "+v"(p[i]));   // one conversion: not a's again for the remainder
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

// 8 consecutive io elements of a row as loaded (16-byte loads), and as a
// fragment.
template <typename IO> struct Raw8;
template <> struct Raw8<bf16> {
  uint4 v;
  __device__ __forceinline__ void load(const bf16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void keep(bool in) {
    v.x = in ? v.x : 0u; v.y = in ? v.y : 0u; v.z = in ? v.z : 0u; v.w = in ? v.w : 0u;
  }
  __device__ __forceinline__ Frag<1> frag() const {
    Frag<1> f;
    f.p[0] = __builtin_bit_cast(bf16x8, v);
    return f;
  }
};
template <> struct Raw8<float> {
  f32x4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const f32x4*>(p);
    b = *reinterpret_cast<const f32x4*>(p + 4);
  }
  __device__ __forceinline__ void keep(bool in) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a[e] = in ? a[e] : 0.0f;
      b[e] = in ? b[e] : 0.0f;
    }
  }
  __device__ __forceinline__ Frag<3> frag() const {
    const float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    return split8<3>(x);
  }
};
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
// group q gets rows r0 + 8 q .. + 7 of column c0 + j, from its own address (row 8 q
// + j / 4 past r0, column 4 (j % 4) past c0; `second` away for the other four
// rows) or from the tile's.
template <int NP>
__device__ __forceinline__ Frag<NP> read_tr(const bf16* p, int plane, int second) {
  Frag<NP> f;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const bf16x4 lo = lds_read_tr4(p + i * plane), hi = lds_read_tr4(p + i * plane + second);
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

// Delta of z = dt + dt_bias.  The clip's minimum and maximum return the other
// operand of a NaN, which would make it a bound, an ordinary gate: it stays a NaN.
__device__ __forceinline__ float rate_of(const DeltaArgs& a, float z) {
  const float d = delta_of(z, a.softplus, a.dt_min, a.dt_max);
  return z == z ? d : z;
}

// 1 / (1 + e^-z), also for -infinity (0)
__device__ __forceinline__ float sigmoid_of(float z) {
  return 1.0f / (1.0f + exp2_of(-z * kLog2e));
}

// One row of k or q as a matrix operand: key columns 32 s + 8 (lane / 16) .. + 7
// of step s, zeros from N on (FULL: N is KP).  `p` points at the lane's columns
// of step 0.  Wavefront w holds rows 16 w + lane % 16 of a chunk; tokens past a
// sequence's end are its last one again, which factors of zero keep out of
// everything.
template <typename IO, int KP, bool FULL> struct KeyRow {
  Raw8<IO> f[KP / 32];
  __device__ __forceinline__ void load(const IO* p, int N, int q) {
#pragma unroll
    for (int s = 0; s < KP / 32; ++s) f[s].load(p + (FULL || 32 * s + 8 * q < N ? 32 * s : -8 * q));
  }
  __device__ __forceinline__ Frag<Planes<IO>::in> frag(int s, int N, int q) const {
    Raw8<IO> r = f[s];
    if constexpr (!FULL) r.keep(32 * s + 8 * q < N);
    return r.frag();
  }
};

// f(io, KP, FULL) with the compiled variant of these keys as constants
template <typename F>
hipError_t with_keys(int N, bool io_bf16, F&& f) {
  using std::integral_constant;
  auto keys = [&](auto io) {
    if (N == 128) return f(io, integral_constant<int, 128>{}, integral_constant<bool, true>{});
    if (N > 64) return f(io, integral_constant<int, 128>{}, integral_constant<bool, false>{});
    if (N == 64) return f(io, integral_constant<int, 64>{}, integral_constant<bool, true>{});
    return f(io, integral_constant<int, 64>{}, integral_constant<bool, false>{});
  };
  return io_bf16 ? keys(bf16{}) : keys(float{});
}

// A gate component's 64 tokens
enum Gate { kBeta = 0, kRight = C, kEnd = 2 * C, kOut = 3 * C, kGates = 4 * C };

// Where the 32 columns from 32 s on of row tile w are among a triangular
// operand's fragments, and these in the workspace
// (a fragment's planes next to each other)
__device__ __forceinline__ int lower_frag(int w, int s) { return w < 2 ? w : 2 * w - 2 + s; }
__device__ __forceinline__ int upper_frag(int w, int s) { return w < 2 ? 2 * w + s : w + 2; }
template <int NP>
__device__ __forceinline__ void store_frag(bf16* base, int64_t at, int f, int lane, const Frag<NP>& v) {
#pragma unroll
  for (int i = 0; i < NP; ++i)
    *reinterpret_cast<bf16x8*>(base + ((at * kTriFrags + f) * NP + i) * kFrag + lane * 8) = v.p[i];
}

// The wavefront's index, in a scalar register
__device__ __forceinline__ int wave_of(int tid) { return __builtin_amdgcn_readfirstlane(tid >> 6); }

// f with the wavefront's index as a constant
template <typename F> __device__ __forceinline__ void by_wave(int w, F&& f) {
  if (w == 0) f(std::integral_constant<int, 0>{});
  else if (w == 1) f(std::integral_constant<int, 1>{});
  else if (w == 2) f(std::integral_constant<int, 2>{});
  else f(std::integral_constant<int, 3>{});
}

template <int CTRL> __device__ __forceinline__ float dpp_add(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
// sum over 16 lanes by neighbours (quads, halves of 8, of 16), without a trip through LDS
__device__ __forceinline__ float sum_of_16(float v) {
  v = dpp_add<0xb1>(v);           // lane ^ 1
  v = dpp_add<0x4e>(v);           // lane ^ 2
  v = dpp_add<0x141>(v);          // mirrored within 8
  return dpp_add<0x140>(v);       // mirrored within 16
}

// sum over a wavefront
__device__ __forceinline__ float wave_sum64(float v) {
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// ---------------------------------------------------------------------------
// Chains of wavefronts that own whole value columns (bfloat16 io).
//
// A result of a matrix product becomes the right operand of the next one
// without leaving the lane: the result of row tiles 2 s and 2 s + 1 gives lane
// group q the rows 4 q .. + 3 of each, and a right operand of 32 contraction
// indices wants 8 per lane group, in any order that the left operand shares.
// Over tokens that order is as the tiles lie: 32 s + 4 q .. + 3, then 32 s + 16
// + 4 q .. + 3; left operands come as such (the triangular fragments) or are read
// so.  Over keys row i of tiles 2 u and 2 u + 1 stands for keys 32 u + 8 (i / 4) +
// i % 4 and 4 more, so that the order is 32 u + 8 q .. + 7 and a left operand's
// row one 16-byte vector: key_of(t, i).
// ---------------------------------------------------------------------------
__device__ __forceinline__ int key_of(int t, int i) {
  return 32 * (t >> 1) + 8 * (i >> 2) + 4 * (t & 1) + (i & 3);
}
// where a token lies in that order, counted in the LDS rows of the chains
__device__ __forceinline__ int token_slot(int t, int q) { return 32 * (t >> 1) + 8 * q + 4 * (t & 1); }

// One plane of a transposed operand from the lane's two addresses
__device__ __forceinline__ Frag<1> read_tr2(const bf16* p, int second) {
  const bf16x4 lo = lds_read_tr4(p), hi = lds_read_tr4(p + second);
  Frag<1> f;
  f.p[0] = bf16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  return f;
}

// 16 bytes per lane from global memory (a uniform address and a lane's offset)
// straight to LDS, 1 KB from byte address `to` + AT on in lane order.  The wait is
// the caller's (landed()): for the builtin the compiler would put one for
// everything requested before the next read of LDS.  s_nop: the base may come from
// a vector instruction (v_readlane), five cycles before a load may use it.
template <int AT = 0>
__device__ __forceinline__ void request16(const void* from, uint32_t offset, uint32_t to) {
  asm volatile("s_add_u32 m0, %0, %3\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2"
               :: "s"(to), "v"(offset), "s"(from), "n"(AT) : "memory", "m0", "scc");
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

// LDS banks.  A 16-byte read takes lanes 0-3, 12-15, 20-23 and 24-27 at a time
// (then the other half of 0-31, and 32-63 alike; found from the conflict counter
// over row strides): rows j of one lane group with those of the next, whose
// vector number differs in bit 0.  So rows are not padded; the 16-byte vectors
// of a row are permuted by exclusive or with a function of its number that takes
// {0-3, 12-15} and {4-11} each to a set closed under changing bit 0.
//
// Rows that are only written 8 bytes and read 16 bytes at a time, R elements
// each: the row's number itself.
template <int R>
__device__ __forceinline__ int row_vec(int row, int vec) {
  return row * R + 8 * (vec ^ (R == 128 ? row & 15 : row >> 1 & 7));
}

// The keys or queries of a chunk: read transposed, too, 4 x 4 (row 4 q + d, vector
// 4 u + b) at a time, which wants different upper bits for each d.
template <int KP, int NW> struct KeyTile {
  static constexpr int kVecs = KP / 8, kRows = 64 / kVecs;   // vectors of a row, rows of 1 KB
  static constexpr int kElems = C * KP, kLoads = C / kRows / NW;
  __device__ __forceinline__ static int swizzle(int row) {
    const int q = row >> 2 & 3, low = (0x78 >> (2 * q) & 3);   // 0, 2, 3, 1
    return (KP == 128 ? 4 * (row & 3) : 4 * (row >> 1 & 1)) + low;
  }
  // The lane's part of a wavefront's requests: byte offsets from the chunk's
  // first row; past row `last` that row again.  64 rows count in 32 bits.
  struct Offsets {
    uint32_t at[kLoads];
    bool in[kLoads];
  };
  __device__ __forceinline__ static void offsets(Offsets& o, int stride, int last, int N, int w, int lane) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int row = (i * NW + w) * kRows + lane / kVecs, vec = lane % kVecs ^ swizzle(row);
      o.at[i] = (uint32_t)min(row, last) * (uint32_t)stride * 2u + 16u * vec;
      o.in[i] = 8 * vec < N;
    }
  }
  // `tile`: the LDS address plus w KB.  Columns from N on (FULL: there are none)
  // are left as they are, zero.
  template <bool FULL, int I = 0>
  __device__ __forceinline__ static void request(const bf16* base, const Offsets& o, uint32_t tile) {
    if constexpr (I < kLoads) {
      if (FULL || o.in[I]) request16<I * NW * 1024>(base, o.at[I], tile);
      request<FULL, I + 1>(base, o, tile);
    }
  }
  // lane's address of row tile 0 of the left operand's step s (tile t: 16 t rows on)
  __device__ __forceinline__ static int row_at(int s, int j, int q) { return j * KP + 8 * ((4 * s + q) ^ swizzle(j)); }
  // lane's address of key tiles 2 u and 2 u + 1 (4 elements further) as left
  // operand of the first 32 tokens, contracted over them (read transposed)
  __device__ __forceinline__ static int col_at(int u, int j, int q) {
    const int row = 4 * q + (j >> 2);
    return row * KP + 8 * ((4 * u + (j & 3)) ^ swizzle(row));
  }
  // rows 16 further on have the same permutation
  __device__ __forceinline__ static Frag<1> columns(const bf16* p) { return read_tr2(p, 16 * KP); }
};

// N KB, lane-linear, over NW wavefronts; `from` and `to` point w KB on
template <int N, int NW, int I = 0>
__device__ __forceinline__ void request_linear(const void* from, uint32_t to, int w, int lane) {
  if constexpr (I * NW < N) {
    if (I * NW + NW <= N || w < N - I * NW)
      request16<I * NW * 1024>(static_cast<const char*>(from) + I * NW * 1024, 16 * lane, to);
    request_linear<N, NW, I + 1>(from, to, w, lane);
  }
}

// The same with as many requests from every wavefront: past the N-th KB the ones
// from the start again, the same bytes to the same place
template <int N, int NW, int I = 0>
__device__ __forceinline__ void request_evenly(const void* from, uint32_t to, int w, int lane) {
  if constexpr (I * NW < N) {
    const int back = I * NW + NW <= N || w < N - I * NW ? 0 : N * 1024;
    request16<I * NW * 1024>(static_cast<const char*>(from) + (I * NW * 1024 - back), 16 * lane, to - back);
    request_evenly<N, NW, I + 1>(from, to, w, lane);
  }
}

// Value columns of a chunk in LDS: [C][16 NW], as KeyTile, not permuted
template <int NW> struct ColumnTile {
  static constexpr int kVecs = 2 * NW, kRows = 64 / kVecs, kLoads = C / kRows / NW;
  struct Offsets {
    uint32_t at[kLoads];
    bool in;
  };
  __device__ __forceinline__ static void offsets(Offsets& o, int stride, int last, int left, int w, int lane) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      o.at[i] = (uint32_t)min((i * NW + w) * kRows + lane / kVecs, last) * (uint32_t)stride * 2u + 16u * (lane % kVecs);
    o.in = 8 * (lane % kVecs) < left;
  }
  template <bool ALL, int I = 0>
  __device__ __forceinline__ static void request(const bf16* base, const Offsets& o, uint32_t tile) {
    if constexpr (I < kLoads) {
      if (ALL || o.in) request16<I * NW * 1024>(base, o.at[I], tile);
      request<ALL, I + 1>(base, o, tile);
    }
  }
};

// acc += A B for a triangular left operand, whose fragments lie from the lane's
// address `a` on (lower: row tiles 0, 1 stop after the first 32 columns; upper:
// tiles 2, 3 begin behind them)
template <int NP, int NB>
__device__ __forceinline__ void mma_lower(const bf16* a, const Frag<NB> (&b)[2], f32x4 (&acc)[4]) {
  Frag<NP> f[4], g[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = load_planes<NP>(a + lower_frag(i, 0) * (NP * kFrag), kFrag);
#pragma unroll
  for (int i = 0; i < 2; ++i) g[i] = load_planes<NP>(a + lower_frag(i + 2, 1) * (NP * kFrag), kFrag);
  mma_tiles(f, b[0], acc);
  mma_tiles(g, b[1], acc + 2);
}
template <int NP, int NB>
__device__ __forceinline__ void mma_upper(const bf16* a, const Frag<NB> (&b)[2], f32x4 (&acc)[4]) {
  Frag<NP> f[2], g[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) f[i] = load_planes<NP>(a + upper_frag(i, 0) * (NP * kFrag), kFrag);
#pragma unroll
  for (int i = 0; i < 4; ++i) g[i] = load_planes<NP>(a + upper_frag(i, 1) * (NP * kFrag), kFrag);
  mma_tiles(f, b[0], acc);
  mma_tiles(g, b[1], acc);
}

// two result tiles as a right operand
template <int NP>
__device__ __forceinline__ Frag<NP> right_of(f32x4 a, f32x4 b) {
  const float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  return split8<NP>(x);
}

// `x` has been waited for: the compiler does not see the waits of landed() and
// would put one of its own before x's first use in a loop, for whatever is in
// flight there
__device__ __forceinline__ void pin(f32x4& x) { asm volatile("" : "+v"(x)); }

// A value that the launch before left, the same for the whole wavefront, through
// the scalar unit: a vector load's wait would be for every request before it too
__device__ __forceinline__ float load_uniform(const float* p) {
  return *(const __attribute__((address_space(4))) float*)p;
}

// Everything but the last STORES memory operations of the wavefront has landed,
// its LDS reads are done, and every wavefront is here.
template <int STORES>
__device__ __forceinline__ void landed() {
  static_assert(STORES < 64, "the counter's range");
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_waitcnt lgkmcnt(0)\n\ts_barrier" ::"n"(STORES) : "memory");
}

// Everyone has read what it will of LDS: requests may overwrite it
__device__ __forceinline__ void lds_free() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Value columns of a chain whose four wavefronts share them and split the tokens
// (tokens(NG): NG such groups of 16 columns to a workgroup, which fills a compute
// unit's LDS), or a chain of wavefronts that own 16 each (columns()).  Sharing
// makes a step as short as it gets and is taken while every chain has a unit to
// itself; owning needs less than half the work of LDS and VALU for as many
// columns, and two workgroups share a unit.  bfloat16, 4096 tokens, shared in pairs
// against owned, in us: scans with 128 keys, 160 pairs 209 against 336, 256 pairs
// 257 / 356, 272 384 / 359, 320 410 / 377, 384 440 / 406; with 64 keys, 256 177 / 293,
// 272 310 / 297; 8 x 16384 tokens of 64 heads (1024 pairs) 3120 / 2145.  The gradients'
// chains with 128 keys, 256 pairs 285 / 390, 288 353 / 410, 320 369 / 425, 384 447 / 438,
// 512 486 / 455; with 64, 256 223 / 311, 288 274 / 322: between 256 and 384 pairs the rule
// loses up to a seventh there.
//
// `ways`: chains that one launch runs for every column (the gradients' both of 32
// heads: 128 and 187 us one after the other, 265 to 285 us together in pairs)
template <typename F, typename G>
hipError_t chain_of(const DeltaArgs& a, int ways, F&& tokens, G&& columns) {
  const int64_t heads = ways * a.Bt * a.H, groups = heads * ((a.P + 15) / 16), pairs = heads * ((a.P + 31) / 32);
  if (groups <= 256) tokens(std::integral_constant<int, 1>{}, (unsigned)groups);
  else if (pairs <= 256) tokens(std::integral_constant<int, 2>{}, (unsigned)pairs);
  else columns((unsigned)(heads * ((a.P + 63) / 64)));
  return hipGetLastError();
}

// Columns and keys that the chains keep of a head in the gradients' workspace:
// whole tiles, so that no store is conditional
__device__ __forceinline__ int padded_cols(int P) { return (P + 15) / 16 * 16; }

// What a workgroup of one chunk and head works on.  Workgroups count below 2^24,
// H and Nc no further: divisions of 32 bits (64-bit ones were a tenth of
// k_delta_prep's instructions).
struct ChunkHead { int64_t b, c, h, g; };
__device__ __forceinline__ ChunkHead chunk_head(const DeltaArgs& a) {
  const uint32_t id = (uint32_t)xcd_remap(blockIdx.x, gridDim.x), H = (uint32_t)a.H, Nc = (uint32_t)a.Nc;
  const uint32_t h = id % H, rest = id / H;
  return {rest / Nc, rest % Nc, h, h / (H / (uint32_t)a.G)};
}

// Position of a (b, h, chunk)
__device__ __forceinline__ int64_t chunk_at(const DeltaArgs& a, int64_t bh, int64_t c) {
  return bh * a.Nc + c;
}

}  // namespace delta
}  // namespace ssd
