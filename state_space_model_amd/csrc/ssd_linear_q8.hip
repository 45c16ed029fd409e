// Product of 8-bit rows on the integer matrix cores of gfx950:
//   out[m][n] = sx[m] sw[n] sum_k x[m][k] w[n][k]
//
// The weight is the instruction's first operand, so that a lane ends with
// four adjacent outputs of one token.  Both matrix instructions used contract
// 16 adjacent bytes per lane, any assignment of columns to lanes being valid
// as long as both operands share it; the integer sum is exact, so its order is
// free and every shape gives the same bits.
//   v_mfma_i32_16x16x64_i8  lane l: row l % 16, bytes 16 (l / 16) of 64;
//                           register r: element [4 (l / 16) + r][l % 16]
//   v_mfma_i32_32x32x32_i8  lane l: row l % 32, bytes 16 (l / 32) of 32;
//                           register r: [8 (r / 4) + 4 (l / 32) + r % 4][l % 32]
#include "ssd_launch.h"
#include "ssd_rows.h"

namespace ssd {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ i32x4 load16(const int8_t* p) { return *reinterpret_cast<const i32x4*>(p); }

// four adjacent outputs of one token, of which `n` exist
template <typename T>
__device__ __forceinline__ void store_quad(T* p, i32x4 acc, const float* ws, float xs, int n) {
  if (n >= 4) {
    const fvec<4> w = load_pack<4>(ws);
    fvec<4> v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (float)acc[e] * xs * w[e];
    store_pack<4>(p, convert_pack<T, 4>(v));
  } else {
    for (int e = 0; e < n; ++e) p[e] = to_io<T>((float)acc[e] * xs * ws[e]);
  }
}

// ---------------------------------------------------------------------------
// Few tokens: the weights stream once from memory.  A workgroup of eight
// wavefronts owns 16 outputs and all (up to 16) tokens; the wavefronts split
// the columns, 128 bytes (a line of each weight row) at a time, load straight
// into registers and add up through LDS.  What counts is how many bytes are in
// flight: many wavefronts with few loads each.  Two, three and five times 128
// bytes at a time took the same or more (one token: 10576 x 2560 8.3-8.7 us,
// 2560 x 5120 6.4-6.8, against 8.5 and 6.5), and so did 4 and 16 wavefronts
// (2048 x 4096: 7.4 and 5.2 against 5.4 us; 16 x 10576 x 2560: 11.0 and 12.1
// against 11.2).
// ---------------------------------------------------------------------------
template <typename T>
__global__ __launch_bounds__(512) void k_linear_q8_stream(LinearQ8Args a) {
  constexpr int NW = 8;
  __shared__ i32x4 part[NW - 1][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, g = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int64_t n = n0 + i < a.N ? n0 + i : a.N - 1, m = i < a.M ? i : a.M - 1;
  const int units = a.K / 128;
  const int u0 = units * wave / NW, u1 = units * (wave + 1) / NW;
  const int8_t* w = a.wq + n * a.K + g * 16;
  const int8_t* x = a.q + m * a.K + g * 16;
  i32x4 acc = {};
  for (int u = u0; u < u1; ++u) {
    const i32x4 w0 = load16(w + u * 128), w1 = load16(w + u * 128 + 64);
    const i32x4 x0 = load16(x + u * 128), x1 = load16(x + u * 128 + 64);
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(w0, x0, acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(w1, x1, acc, 0, 0, 0);
  }
  if (wave > 0) part[wave - 1][lane] = acc;
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int o = 0; o < NW - 1; ++o) acc += part[o][lane];
  const int64_t nn = n0 + 4 * g;
  if (i < a.M && nn < a.N)
    store_quad(reinterpret_cast<T*>(a.out) + i * a.N + nn, acc, a.wscale + nn, a.qscale[i],
               (int)(a.N - nn < 4 ? a.N - nn : 4));
}

// The k-th tile in launch order, of nt x mt: those of one XCD are consecutive, in
// groups of 8 tile rows, so that the tiles it holds at a time share both
// operands' panels in its L2.
struct TileOf {
  int32_t n, m;
  __device__ __forceinline__ TileOf(int32_t nt, int32_t mt, int32_t k) {
    constexpr int32_t kRows = 8;
    const uint32_t id = (uint32_t)xcd_remap(k, (int64_t)nt * mt);
    const uint32_t per = kRows * nt, group = id / per, in = id % per, first = group * kRows;
    const uint32_t size = min((uint32_t)mt - first, (uint32_t)kRows);
    // divisions are done on the vector unit; the results are the same in every lane
    m = __builtin_amdgcn_readfirstlane((int)(first + in % size));
    n = __builtin_amdgcn_readfirstlane((int)(in / size));
  }
};

// A wavefront's 32 TN x 32 TM outputs, through its own kOutBytes of LDS: 64
// columns of 32 tokens at a time, scaled by the token on the way in and by the
// column on the way out, where a lane's four columns stay the same; each
// token's columns then leave as whole lines.
constexpr int kOutPitch = 256 + 16, kOutBytes = 32 * kOutPitch;
template <typename T, int TN, int TM>
__device__ __forceinline__ void store_tile(const LinearQ8Args& a, const i32x16 (&acc)[TN][TM],
                                           int8_t* lds, int64_t n0, int64_t m0, int lane) {
  const int half = lane >> 5, tok = lane & 31, c = (lane & 15) * 4;
  float xs[TM];
#pragma unroll
  for (int tm = 0; tm < TM; ++tm) {
    const int64_t m = m0 + 32 * tm + tok;
    xs[tm] = a.qscale[m < a.M ? m : a.M - 1];
  }
#pragma unroll
  for (int t0 = 0; t0 < TN; t0 += 2) {
    const int64_t n = n0 + 32 * t0 + c;
    const int left = (TN - t0 >= 2 || c < 32) && n < a.N ? (int)(a.N - n < 4 ? a.N - n : 4) : 0;
    fvec<4> ws;
#pragma unroll
    for (int e = 0; e < 4; ++e) ws[e] = a.wscale[e < left ? n + e : a.N - 1];
#pragma unroll
    for (int tm = 0; tm < TM; ++tm) {
#pragma unroll
      for (int t = t0; t < t0 + 2 && t < TN; ++t)
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          fvec<4> v;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = (float)acc[t][tm][4 * p + e] * xs[tm];
          *reinterpret_cast<fvec<4>*>(lds + tok * kOutPitch + (32 * (t - t0) + 8 * p + 4 * half) * 4) = v;
        }
      // (LDS operations of one wavefront complete in order)
#pragma unroll
      for (int r = 0; r < 32; r += 4) {
        const int row = r + lane / 16;
        const fvec<4> v = *reinterpret_cast<const fvec<4>*>(lds + row * kOutPitch + c * 4) * ws;
        const int64_t m = m0 + 32 * tm + row;
        if (m < a.M) {
          T* out = reinterpret_cast<T*>(a.out) + m * a.N + n;
          const typename Pack<T, 4>::V o = convert_pack<T, 4>(v);
          if (left == 4) {
            store_pack<4>(out, o);
          } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
              if (e < left) out[e] = o[e];
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Many tokens: BN outputs x BM tokens per workgroup, WN x WM wavefronts, the
// operands staged through LDS 128 columns at a time in a ring of NS buffers.
//
// Global loads write LDS directly, 16 bytes per lane: a wavefront's load fills
// 8 rows of 128 bytes.  The 16-byte chunk c of row r is kept at position
// c ^ (r / 2 % 8) of its row, so that the 16 lanes of a read phase, which take
// one chunk of 16 adjacent rows, meet 16 different quarter-banks; the swizzle
// is applied to the global address, as the LDS side of such a load is linear.
// (Columns go 128 at a time because a cache line holds them: with 64, every
// line is requested twice, 8192 x 8192 x 8192: 515 -> 555 us.)
// ---------------------------------------------------------------------------
template <typename T, int BN, int BM, int WN, int WM, int NS>
__global__ __launch_bounds__(64 * WN * WM) void k_linear_q8_tile(LinearQ8Args a, int32_t nt,
                                                                  int32_t mt) {
  constexpr int NW = WN * WM, BK = 128, KK = BK / 32;
  constexpr int TN = BN / WN / 32, TM = BM / WM / 32;   // 32 x 32 tiles of a wavefront
  constexpr int STAGE = (BN + BM) * BK, LOADS = (BN + BM) / 8 / NW;
  static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0 && (NS - 2) * LOADS < 64);
  // (the outputs pass through the same memory afterwards)
  __shared__ __align__(1024) int8_t sm[NS * STAGE > NW * kOutBytes ? NS * STAGE : NW * kOutBytes];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const TileOf at(nt, mt, blockIdx.x);
  const int64_t m0 = (int64_t)at.m * BM, n0 = (int64_t)at.n * BN;

  // rows past the end repeat the last one (their outputs are not stored)
  const int8_t* wp = a.wq + n0 * a.K;
  const int8_t* xp = a.q + m0 * a.K;
  const int nlast = (int)(a.N - n0 < BN ? a.N - n0 : BN) - 1;
  const int mlast = (int)(a.M - m0 < BM ? a.M - m0 : BM) - 1;
  uint32_t off[LOADS];
#pragma unroll
  for (int j = 0; j < LOADS; ++j) {
    const int r = (j * NW + wave) * 8 + lane / 8, chunk = (lane % 8) ^ (r / 2 % 8);
    const int row = j * NW * 8 < BN ? min(r, nlast) : min(r - BN, mlast);
    off[j] = (uint32_t)row * (uint32_t)a.K + chunk * 16;
  }
  // part of the loads of the step wp and xp point at
  auto stage = [&](int buf, int j0, int j1) {
#pragma unroll
    for (int j = j0; j < j1; ++j)
      __builtin_amdgcn_global_load_lds(
          (const __attribute__((address_space(1))) void*)((j * NW * 8 < BN ? wp : xp) + off[j]),
          (__attribute__((address_space(3))) void*)(sm + buf * STAGE + (j * NW + wave) * 1024), 16, 0, 0);
  };
  const int steps = a.K / BK;
  // past the end the last step is loaded again, into a buffer that no one reads
  auto advance = [&](int s) {
    wp += s < steps ? BK : 0;
    xp += s < steps ? BK : 0;
  };
  const int wn = wave % WN, wm = wave / WN, half = lane >> 5;
  const int rw = wn * (BN / WN) + (lane & 31), rx = BN + wm * (BM / WM) + (lane & 31);
  i32x16 acc[TN][TM] = {};
#pragma unroll
  for (int p = 0; p < NS - 1; ++p) {
    stage(p, 0, LOADS);
    advance(p + 1);
  }
  int cur = 0;
  for (int s = 0; s < steps; ++s) {
    // step s has landed everywhere, and step s - 1 has been read
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_waitcnt lgkmcnt(0)\n\ts_barrier" ::"n"((NS - 2) * LOADS)
                 : "memory");
    const int8_t* b = sm + cur * STAGE;
    i32x4 wf[KK][TN], xf[KK][TM];
    auto frags = [&](int kk) {
#pragma unroll
      for (int t = 0; t < TN; ++t)
        wf[kk][t] = load16(b + (rw + 32 * t) * BK + (((2 * kk + half) ^ (rw / 2 % 8)) << 4));
#pragma unroll
      for (int t = 0; t < TM; ++t)
        xf[kk][t] = load16(b + (rx + 32 * t) * BK + (((2 * kk + half) ^ (rx / 2 % 8)) << 4));
    };
    const int free = cur == 0 ? NS - 1 : cur - 1;
    frags(0);
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      auto product = [&](int i0, int i1) {
#pragma unroll
        for (int i = i0; i < i1; ++i)
          acc[i / TM][i % TM] = __builtin_amdgcn_mfma_i32_32x32x32_i8(
              wf[kk][i / TM], xf[kk][i % TM], acc[i / TM][i % TM], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
      };
      // the next operands and a share of the loads behind the first product
      product(0, 1);
      if (kk + 1 < KK) frags(kk + 1);
      stage(free, LOADS * kk / KK, LOADS * (kk + 1) / KK);
      __builtin_amdgcn_sched_barrier(0);
      product(1, TN * TM);
    }
    advance(s + NS);
    cur = cur + 1 == NS ? 0 : cur + 1;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // no load may reach LDS after this
  __syncthreads();
  store_tile<T, TN, TM>(a, acc, sm + wave * kOutBytes, n0 + wn * (BN / WN), m0 + wm * (BM / WM), lane);
}

// Few tiles: the KS wavefronts of a workgroup share one BN x BM tile and split
// its columns; each stages its part through a ring of its own, without
// barriers, and the sums meet in LDS.  Workgroups next to each other on an XCD
// start their columns three steps apart: all of them read the same tokens, and
// in step they would ask the same channels of the L2 for the same lines
// (64 x 2560 x 5120: 10.0 -> 9.0 us, 33 x 2560 x 5120: 8.6 -> 7.6 us).
template <typename T, int BN, int BM, int KS, int NS>
__global__ __launch_bounds__(64 * KS) void k_linear_q8_split(LinearQ8Args a, int32_t nt, int32_t mt) {
  constexpr int BK = 128, TN = BN / 32, TM = BM / 32, LOADS = (BN + BM) / 8;
  constexpr int STAGE = (BN + BM) * BK, RING = KS * NS * STAGE;
  constexpr int OUT = KS * TN * TM * 4096;
  static_assert((NS - 1) * LOADS < 64 && 4 * TN * TM % KS == 0);
  __shared__ __align__(1024) int8_t sm[RING > OUT ? RING : OUT];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const TileOf at(nt, mt, blockIdx.x);
  const int64_t m0 = (int64_t)at.m * BM, n0 = (int64_t)at.n * BN;
  const int nlast = (int)(a.N - n0 < BN ? a.N - n0 : BN) - 1;
  const int mlast = (int)(a.M - m0 < BM ? a.M - m0 : BM) - 1;
  uint32_t off[LOADS];
#pragma unroll
  for (int j = 0; j < LOADS; ++j) {
    const int r = j * 8 + lane / 8, chunk = (lane % 8) ^ (r / 2 % 8);
    const int row = j * 8 < BN ? min(r, nlast) : min(r - BN, mlast);
    off[j] = (uint32_t)row * (uint32_t)a.K + chunk * 16;
  }
  const int8_t* wp = a.wq + n0 * a.K;
  const int8_t* xp = a.q + m0 * a.K;
  const int steps = a.K / BK, s0 = steps * wave / KS, s1 = steps * (wave + 1) / KS;
  const int share = s1 - s0, turn = share > 0 ? (int)(blockIdx.x / 8 * 3 % share) : 0;
  int8_t* ring = sm + wave * NS * STAGE;
  auto stage = [&](int s, int buf) {   // past the end: the last step again, read by no one
    const int at = s + turn < s1 ? s + turn : s + turn - share;
    const int64_t k = (int64_t)(s < s1 ? at : steps - 1) * BK;
#pragma unroll
    for (int j = 0; j < LOADS; ++j)
      __builtin_amdgcn_global_load_lds(
          (const __attribute__((address_space(1))) void*)((j * 8 < BN ? wp : xp) + k + off[j]),
          (__attribute__((address_space(3))) void*)(ring + buf * STAGE + j * 1024), 16, 0, 0);
  };
  const int r32 = lane & 31, half = lane >> 5;
  i32x16 acc[TN][TM] = {};
#pragma unroll
  for (int p = 0; p < NS - 1; ++p) stage(s0 + p, p);
  int cur = 0;
  for (int s = s0; s < s1; ++s) {
    // step s has landed, and the reads of step s - 1 are done
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_waitcnt lgkmcnt(0)" ::"n"((NS - 2) * LOADS) : "memory");
    __builtin_amdgcn_sched_barrier(0);
    const int8_t* b = ring + cur * STAGE;
    i32x4 wf[4][TN], xf[4][TM];
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      const int pos = ((2 * kk + half) ^ (r32 / 2 % 8)) << 4;
#pragma unroll
      for (int t = 0; t < TN; ++t) wf[kk][t] = load16(b + (32 * t + r32) * BK + pos);
#pragma unroll
      for (int t = 0; t < TM; ++t) xf[kk][t] = load16(b + (BN + 32 * t + r32) * BK + pos);
    }
    stage(s + NS - 1, cur == 0 ? NS - 1 : cur - 1);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int tn = 0; tn < TN; ++tn)
#pragma unroll
        for (int tm = 0; tm < TM; ++tm)
          acc[tn][tm] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[kk][tn], xf[kk][tm], acc[tn][tm], 0, 0, 0);
    cur = cur + 1 == NS ? 0 : cur + 1;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // no load may reach LDS after this
  __syncthreads();
  // registers 4 p .. 4 p + 3 of all the sums meet in one wavefront, p % KS; a
  // lane holds four outputs of a token there and stores them as they are (by
  // way of LDS as whole lines, and by one wavefront, 64 x 768 x 1536: 5.6
  // against 4.2 us)
  i32x4* sums = reinterpret_cast<i32x4*>(sm);
#pragma unroll
  for (int t = 0; t < TN * TM; ++t)
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const i32x16& v = acc[t / TM][t % TM];
      sums[((t * 4 + p) * KS + wave) * 64 + lane] = i32x4{v[4 * p], v[4 * p + 1], v[4 * p + 2], v[4 * p + 3]};
    }
  __syncthreads();
#pragma unroll
  for (int o = 0; o < 4 * TN * TM / KS; ++o) {
    const int q = o * KS + wave, t = q / 4, p = q % 4;
    i32x4 sum = sums[q * KS * 64 + lane];
#pragma unroll
    for (int k = 1; k < KS; ++k) sum += sums[(q * KS + k) * 64 + lane];
    const int64_t n = n0 + t / TM * 32 + 8 * p + 4 * half, m = m0 + t % TM * 32 + r32;
    if (m < a.M && n < a.N)
      store_quad(reinterpret_cast<T*>(a.out) + m * a.N + n, sum, a.wscale + n, a.qscale[m],
                 (int)(a.N - n < 4 ? a.N - n : 4));
  }
}

template <typename T, int BN, int BM, int KS, int NS>
hipError_t split(const LinearQ8Args& a, hipStream_t s) {
  const int32_t nt = (int32_t)((a.N + BN - 1) / BN), mt = (int32_t)((a.M + BM - 1) / BM);
  hipLaunchKernelGGL((k_linear_q8_split<T, BN, BM, KS, NS>), dim3((unsigned)(nt * mt)), dim3(64 * KS), 0, s, a, nt, mt);
  return hipGetLastError();
}

// Many tiles: 32 TN outputs x 256 tokens, two groups of four wavefronts, one of
// each group on every SIMD.  The groups take turns: while one multiplies, the
// other fetches its operands of the next 128 columns from LDS into registers
// and requests the columns after those.  A load's issue holds its wavefront
// until the memory pipe takes it, which in the plain kernel above kept the
// matrix cores waiting for about as long as they worked.  Phase 2g: group 0
// reads step g from LDS, group 1 multiplies step g-1; phase 2g+1: group 0
// multiplies step g, group 1 reads it.  A buffer is free for step g+2 once group
// 1 has read step g, in the middle of phase 2g+1 (the second barrier there).
//
// A workgroup stays for several tiles: the loads run on into the next tile, so
// that its first columns arrive while this one is stored, and the waits for
// them leave the stores in flight.
constexpr int64_t kTurnsMaxOuts = 1 << 24;
constexpr int kTurnsOut = 16 * 256;   // bytes of LDS a wavefront's outputs pass through

template <typename T, int TN>
__global__ __launch_bounds__(512) void k_linear_q8_turns(LinearQ8Args a, int32_t nt, int32_t mt) {
  constexpr int TM = 4, BK = 128, BN = 32 * TN, BM = 256, NW = 8;
  constexpr int PIECES = (BN + BM) / 8, WPIECES = BN / 8, STAGE = (BN + BM) * BK;
  constexpr int LOADS = (PIECES + NW - 1) / NW;
  static_assert(WPIECES % 4 == 0 && PIECES % 4 == 0);   // a group's four loads share an operand
  constexpr int SW = kTurnsOut / 16 / (int)sizeof(T), ST = SW / 16, CH = SW / 4;
  // stores of a wavefront's whole tile, at least: every 64 columns and 4 tokens
  constexpr int STORES = TM * 4 * ((16 * TN + 63) / 64);
  static_assert(STORES < 64);
  __shared__ __align__(1024) int8_t sm[2 * STAGE + NW * kTurnsOut];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave & 1, wm = wave >> 1, l16 = lane & 15, q4 = lane >> 4;
  const int32_t tiles = nt * mt;
  const int steps = a.K / BK;
  const int mine = (tiles - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
  const int total = steps * mine;

  // loader: runs ahead of the products, into the next tile
  int32_t ltile = blockIdx.x;
  int lstep = 0;
  const int8_t *lw, *lx;
  uint32_t off[LOADS];
  auto aim = [&]() {
    // (an opaque lane index here and in finish: what they derive from it is then
    // formed there instead of being held in registers through the products)
    const int lane = opaque_tid() & 63;
    const TileOf at(nt, mt, ltile);
    lw = a.wq + (int64_t)at.n * BN * a.K;
    lx = a.q + (int64_t)at.m * BM * a.K;
    const int64_t nl = a.N - (int64_t)at.n * BN, ml = a.M - (int64_t)at.m * BM;
    const int nlast = (int)(nl < BN ? nl : BN) - 1, mlast = (int)(ml < BM ? ml : BM) - 1;
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      const int piece = j * NW + wave, r = piece * 8 + lane / 8;
      const int row = piece < WPIECES ? min(r, nlast) : min(r - BN, mlast);
      off[j] = (uint32_t)row * (uint32_t)a.K + (((lane % 8) ^ (r / 2 % 8)) << 4);
    }
  };
  // requests this wavefront's part of the loader's step into buffer g % 2
  auto stage = [&](auto group, int g) {
    constexpr int first = 4 * decltype(group)::value;
    int8_t* dst = sm + (g & 1) * STAGE + wave * 1024;
#pragma unroll
    for (int j = 0; j < LOADS; ++j)
      if (j * NW + first < PIECES)
        __builtin_amdgcn_global_load_lds(
            (const __attribute__((address_space(1))) void*)(
                (j * NW + first < WPIECES ? lw : lx) + off[j]),
            (__attribute__((address_space(3))) void*)(dst + j * NW * 1024), 16, 0, 0);
  };
  // past the last tile the loader repeats the last step, into a buffer no one
  // reads any more
  auto advance = [&]() {
    if (lstep + 1 < steps) {
      ++lstep;
      lw += BK;
      lx += BK;
    } else if (ltile + (int)gridDim.x < tiles) {
      ltile += gridDim.x;
      lstep = 0;
      aim();
    }
  };

  i32x4 acc[TN][TM] = {};
  i32x4 wf[2][TN], xf[2][TM];
  const int rw = wn * (BN / 2) + l16, rx = BN + wm * (BM / 4) + l16;
  auto frags = [&](int g) {
    const int8_t* b = sm + (g & 1) * STAGE;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      // (rows 16 apart share the swizzle of their first)
      const int pos = ((4 * kk + q4) ^ (l16 / 2 % 8)) << 4;
#pragma unroll
      for (int t = 0; t < TN; ++t) wf[kk][t] = load16(b + (rw + 16 * t) * BK + pos);
#pragma unroll
      for (int t = 0; t < TM; ++t) xf[kk][t] = load16(b + (rx + 16 * t) * BK + pos);
    }
  };
  auto product = [&](int kk) {
#pragma unroll
    for (int tn = 0; tn < TN; ++tn)
#pragma unroll
      for (int tm = 0; tm < TM; ++tm)
        acc[tn][tm] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[kk][tn], xf[kk][tm], acc[tn][tm], 0, 0, 0);
  };

  int32_t tile = blockIdx.x;
  // Stores the finished tile and clears the sums; true for a whole tile, which
  // issues at least STORES stores.  16 tokens x SW columns at a time pass
  // through LDS in the output type (four columns of a token at chunk c ^ 2
  // token), to leave as 64 adjacent columns of four tokens per instruction.
  // Where every such piece is whole lines of memory they go out non-temporal
  // (4096 x 10752 outputs: 133 -> 108 us); elsewhere the cache has to join the
  // pieces (10576 outputs non-temporal: no gain, at 128 columns 37 -> 57 us).
  // Shifting a token's pieces to its lines took longer (three instead of two
  // instructions; 115 -> 120 us).
  auto finish = [&]() {
    const int lane = opaque_tid() & 63, l16 = lane & 15, q4 = lane >> 4;
    typedef typename Pack<T, 4>::V V4;
    const TileOf at(nt, mt, tile);
    tile += gridDim.x;
    const int64_t n0 = (int64_t)at.n * BN + wn * (BN / 2), m0 = (int64_t)at.m * BM + wm * (BM / 4);
    const bool whole = (int64_t)(at.n + 1) * BN <= a.N && (int64_t)(at.m + 1) * BM <= a.M;
    const bool lines = ((a.N | n0 | (int64_t)(reinterpret_cast<uintptr_t>(a.out) / sizeof(T))) & 63) == 0;
    int8_t* lds = sm + 2 * STAGE + wave * kTurnsOut;
    float xs[TM];
#pragma unroll
    for (int tm = 0; tm < TM; ++tm) {
      const int64_t m = m0 + 16 * tm + l16;
      xs[tm] = a.qscale[m < a.M ? m : a.M - 1];
    }
#pragma unroll
    for (int t0 = 0; t0 < TN; t0 += ST) {
      constexpr int kFull = 16 * ST;
      const int W = 16 * (TN - t0) < kFull ? 16 * (TN - t0) : kFull;
      fvec<4> ws[ST];
#pragma unroll
      for (int t = 0; t < ST; ++t)
        if (t0 + t < TN) {
          const int64_t n = n0 + 16 * (t0 + t) + 4 * q4;
#pragma unroll
          for (int e = 0; e < 4; ++e) ws[t][e] = a.wscale[n + e < a.N ? n + e : a.N - 1];
        }
#pragma unroll
      for (int tm = 0; tm < TM; ++tm) {
#pragma unroll
        for (int t = 0; t < ST; ++t)
          if (t0 + t < TN) {
            fvec<4> v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = (float)acc[t0 + t][tm][e] * xs[tm] * ws[t][e];
            *reinterpret_cast<V4*>(lds + (l16 * CH + ((4 * t + q4) ^ (2 * l16 & (CH - 1)))) * sizeof(V4)) =
                convert_pack<T, 4>(v);
          }
        // (LDS operations of one wavefront complete in order)
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
          const int row = r + q4;
          const int64_t m = m0 + 16 * tm + row;
          // a uniform base and 32 bits per lane (15 rows of at most kTurnsMaxOuts)
          T* base = reinterpret_cast<T*>(a.out) + (m0 + 16 * tm) * a.N + n0 + 16 * t0;
          const uint32_t ro = (uint32_t)row * (uint32_t)a.N;
#pragma unroll
          for (int i = 0; i < (W + 63) / 64; ++i) {
            const int e = 64 * i + 4 * l16;
            if (e >= W) continue;
            const V4 o = *reinterpret_cast<const V4*>(
                lds + (row * CH + ((e / 4) ^ (2 * row & (CH - 1)))) * sizeof(V4));
            T* out = off32(base, ro + e);
            if (lines && whole) {
              __builtin_nontemporal_store(o, reinterpret_cast<typename Pack<T, 4>::U*>(out));
            } else if (whole) {
              store_pack<4>(out, o);
            } else if (m < a.M) {
              const int64_t left = a.N - (n0 + 16 * t0 + e);
              if (left >= 4) {
                store_pack<4>(out, o);
              } else {
#pragma unroll
                for (int k = 0; k < 3; ++k)
                  if (k < left) out[k] = o[k];
              }
            }
          }
        }
      }
    }
#pragma unroll
    for (int tn = 0; tn < TN; ++tn)
#pragma unroll
      for (int tm = 0; tm < TM; ++tm) acc[tn][tm] = i32x4{0, 0, 0, 0};
    return whole;
  };

#define SSD_FENCE(text)                     \
  __builtin_amdgcn_sched_barrier(0);        \
  asm volatile(text ::: "memory");          \
  __builtin_amdgcn_sched_barrier(0)
// every load has landed; `stored`: behind them are a whole tile's stores, which may stay in flight
#define SSD_LANDED(stored)                                                        \
  __builtin_amdgcn_sched_barrier(0);                                              \
  if (stored) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(STORES) : "memory");       \
  else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");                           \
  __builtin_amdgcn_sched_barrier(0)

  std::integral_constant<int, 0> g0;
  std::integral_constant<int, 1> g1;
  aim();
  int in = 0;   // steps of the current tile multiplied
  if (wave < 4) {
    stage(g0, 0);
    advance();
    SSD_FENCE("s_waitcnt vmcnt(0)\n\ts_barrier");
    for (int g = 0; g < total; ++g) {
      stage(g0, g + 1);
      advance();
      bool stored = false;
      if (in == steps) {
        __builtin_amdgcn_sched_barrier(0);
        stored = finish();
        in = 0;
        __builtin_amdgcn_sched_barrier(0);
      }
      frags(g);
      SSD_FENCE("s_waitcnt lgkmcnt(0)\n\ts_barrier");
      product(0);
      SSD_FENCE("s_barrier");
      product(1);
      ++in;
      SSD_LANDED(stored);
      SSD_FENCE("s_barrier");
    }
  } else {
    stage(g1, 0);
    advance();
    SSD_FENCE("s_waitcnt vmcnt(0)\n\ts_barrier");
    stage(g1, 1);
    advance();
    SSD_FENCE("s_barrier");
    frags(0);
    SSD_FENCE("s_waitcnt vmcnt(0)\n\ts_waitcnt lgkmcnt(0)\n\ts_barrier");
    stage(g1, 2);
    SSD_FENCE("s_barrier");
    for (int g = 1; g < total; ++g) {
      product(0);
      product(1);
      bool stored = false;
      if (++in == steps) {
        stored = finish();
        in = 0;
      }
      advance();   // (while no operands are held)
      SSD_FENCE("s_barrier");
      frags(g);
      SSD_LANDED(stored);
      SSD_FENCE("s_waitcnt lgkmcnt(0)\n\ts_barrier");
      stage(g1, g + 2);
      SSD_FENCE("s_barrier");
    }
    product(0);
    product(1);
  }
  finish();
  SSD_FENCE("s_waitcnt vmcnt(0)");   // no load may reach LDS after the end
#undef SSD_LANDED
#undef SSD_FENCE
}

template <typename T, int TN>
hipError_t turns(const LinearQ8Args& a, hipStream_t s) {
  const int32_t nt = (int32_t)((a.N + 32 * TN - 1) / (32 * TN)), mt = (int32_t)((a.M + 255) / 256);
  const int32_t tiles = nt * mt;
  hipLaunchKernelGGL((k_linear_q8_turns<T, TN>), dim3((unsigned)(tiles < 256 ? tiles : 256)), dim3(512),
                     0, s, a, nt, mt);
  return hipGetLastError();
}

template <typename T>
hipError_t stream(const LinearQ8Args& a, hipStream_t s) {
  hipLaunchKernelGGL(k_linear_q8_stream<T>, dim3((unsigned)((a.N + 15) / 16)), dim3(512), 0, s, a);
  return hipGetLastError();
}

template <typename T, int BN, int BM, int WN, int WM, int NS>
hipError_t tile(const LinearQ8Args& a, hipStream_t s) {
  const int32_t nt = (int32_t)((a.N + BN - 1) / BN), mt = (int32_t)((a.M + BM - 1) / BM);
  hipLaunchKernelGGL((k_linear_q8_tile<T, BN, BM, WN, WM, NS>), dim3((unsigned)(nt * mt)),
                     dim3(64 * WN * WM), 0, s, a, nt, mt);
  return hipGetLastError();
}

// The kernel for M tokens, N outputs and K columns.  Up to 16 tokens, as many
// as one instruction of the stream holds, the weights stream.  Against the
// better of the two split tiles (us, in a HIP graph):
//   N x K         1 token      8 tokens     16 tokens     17 tokens
//   768 x 1536   3.2 / 3.7    3.5 / 3.8    3.8 / 4.1        - / 4.1
//   3352 x 768   3.2 / 3.8    3.4 / 3.9    3.6 / 3.9        - / 4.0
//   2048 x 4096  4.9 / 5.5    5.6 / 5.6    6.2 / 5.7        - / 5.7
//   2560 x 5120  6.3 / 7.8    6.8 / 8.4    7.7 / 9.0        - / 9.1
//   10576 x 2560 8.8 / 9.7    9.5 / 9.5   10.9 / 10.1       - / 10.2
// (16 tokens of two of these shapes would gain 7 to 8% on split tiles.)  Beyond, the tile with the least modelled time:
// rounds over the 256 compute units times (fixed + columns / 128 * step), in
// units of 0.01 us fitted to these measurements (us, kernel time):
//                          64 x 2560  128 x 2560  256 x 2560  1024 x 2560  4096 x 2560  4096 x 10576
//                           x 5120      x 5120      x 5120      x 5120       x 5120       x 2560
//   32 x 32, split columns    9.0        13.2        17.6
//   the same, two to a CU     9.6        11.4        18.3
//   64 x 64                  17.5                    16.3         36           108          237
//   128 x 128                28.5                    30.4         30            86          193
//   160 x 256 in turns                                                          61          144
//   192 x 256 in turns                                                          62          127
//   224 x 256 in turns                                                          61          106-115
//   256 x 256 in turns                                                          77          118-132
// (The model overstates the split tiles past their first round, 23 to 27 us for
// 256 x 2560 x 5120, where 64 x 64 tiles are the fastest and taken.)
// A larger tile moves fewer bytes per product but fills the last round worse;
// at 8192 x 8192 x 8192 the 256 x 256 tiles reach 2.7 Pop/s (405 us), where the
// same instructions on operands that never change reach 4.0-4.5 (the clock
// falls with the work: 1.8-2.0 GHz there).
enum Variant { kSplit, kSplitPair, kTile64, kTile128, kTurns160, kTurns192, kTurns224, kTurns256 };
Variant variant_of(int64_t M, int64_t N, int64_t K) {
  const int64_t steps = K / 128;
  auto tiles = [&](int64_t bn, int64_t bm) { return ((N + bn - 1) / bn) * ((M + bm - 1) / bm); };
  auto rounds = [&](int64_t n) { return (n + 255) / 256; };
  // two 64 x 64 tiles and more share a compute unit
  const int64_t t64 = tiles(64, 64);
  const int64_t cost[] = {
      rounds(tiles(32, 32)) * (210 + 17 * steps),
      rounds((tiles(32, 32) + 1) / 2) * (315 + 21 * steps),   // two to a compute unit
      t64 <= 256 ? 200 + 36 * steps : 200 + steps * (22 + 30 * t64 / 256),
      rounds(tiles(128, 128)) * (200 + 70 * steps),
      rounds(tiles(160, 256)) * (1000 + 113 * steps),
      rounds(tiles(192, 256)) * (1000 + 124 * steps),
      rounds(tiles(224, 256)) * (1000 + 140 * steps),
      rounds(tiles(256, 256)) * ((N % 64 == 0 ? 450 : 1000) + 158 * steps),   // (whole lines)
  };
  int best = 0;
  for (int v = 1; v < (N <= kTurnsMaxOuts ? 8 : 4); ++v)
    if (cost[v] < cost[best]) best = v;
  return (Variant)best;
}

template <typename T>
hipError_t linear_t(const LinearQ8Args& a, hipStream_t s) {
  if (a.M <= 16) return stream<T>(a, s);
  switch (variant_of(a.M, a.N, a.K)) {
    case kSplit: return split<T, 32, 32, 4, 3>(a, s);
    case kSplitPair: return split<T, 32, 32, 4, 2>(a, s);
    case kTile64: return tile<T, 64, 64, 2, 2, 4>(a, s);
    case kTile128: return tile<T, 128, 128, 4, 2, 4>(a, s);
    case kTurns160: return turns<T, 5>(a, s);
    case kTurns192: return turns<T, 6>(a, s);
    case kTurns224: return turns<T, 7>(a, s);
    case kTurns256: return turns<T, 8>(a, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_linear_q8(const LinearQ8Args& a, bool out_bf16, hipStream_t s) {
  return out_bf16 ? linear_t<bf16>(a, s) : linear_t<float>(a, s);
}

}  // namespace ssd
