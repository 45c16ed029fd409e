// The norms around a block's scan for gfx950, forward and backward, and the
// quantiser of 8-bit rows.
//
// Source: "Compiler-First State Space Duality and Portable O(1)
// Autoregressive Caching", Implementation choices, "precision management" (the
// residual stream and the norms in float32).
//
//   add norm    r' = r + s x;          y   = r' c w,  c = 1/sqrt(mean(r'^2) + eps)
//               (with dropout: s x / (1 - p) where the generator keeps x, else r)
//   gated norm  g  = y z / (1+e^-z);   out = g c w,   c per group of columns
//   8-bit rows  a = max|v|;  q = rint(v 127/a), scale a/127
//
// A kernel reads its row once, keeps it in registers through the reduction, and
// writes once (two kernels of 8-bit rows, for several groups and for the widest
// rows, read it twice): they are bound by memory.  A row (or one group
// of it) is shared by one wavefront or by a workgroup (RowTeam).  Measured on
// one MI355X (kernel time in a HIP graph, inputs rotated through HBM):
//   add norm   131072 x 2048 bfloat16   567 us  5.7 TB/s
//              4097 x 768 float32      10.5 us  4.8 TB/s
//   gated norm 4096 x 5120 bfloat16    24.1 us  5.2 TB/s
//   gradients: add norm 4096 x 2560    32.6 us  5.1 TB/s (the sum of the parts 4 us of it)
//              gated, 8 groups, 16384 x 4096   129 us  5.2 TB/s (145 us on another card)
//   8-bit rows 10576 x 2560 float32    25.0 us  5.4 TB/s
//              4096 x 2560 bfloat16     9.1 us  3.5 TB/s
// against 4.8 TB/s for a plain copy of 4 GiB.  Just past a change of variant,
// where 33 to 42 of 64 lanes have a vector, less of it is reached: 65536 rows of
// 264 and 333 bfloat16 columns, gradients of the gated norm 3.3 and 3.9 TB/s,
// its forward 4.3 and 4.4, 8-bit rows 3.0 and 3.6 (512 columns: 5.1, 5.8, 5.1).
// Tried and slower: non-temporal stores (555 -> 572 us, gradients 32.3 -> 38.6
// us: the next kernel's reads and the partial lines of two instructions meet in
// the cache), forward wavefronts that take rows in turn with the weight kept in
// registers (555 -> 605 us), the gradients' next row requested before the
// current one's reduction (32.3 -> 33.8 us).
#include <type_traits>

#include "ssd_launch.h"
#include "ssd_rows.h"

namespace ssd {
namespace {

constexpr int kThreads = 256;        // four wavefronts, a row each
constexpr int kBlockThreads = 512;   // at most, for a workgroup per row
constexpr int kCus = 256;

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
template <typename T, int VEC, int NV, bool BLOCK, bool Q8, bool DROP>
__global__ __launch_bounds__(BLOCK ? kBlockThreads : kThreads) void k_add_norm(AddNormArgs a) {
  __shared__ float sm[kMaxWaves], smq[kMaxWaves];
  const int team = BLOCK ? blockDim.x : 64;
  const int lane = BLOCK ? threadIdx.x : threadIdx.x & 63;
  const int64_t row = BLOCK ? blockIdx.x : (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  if (row >= a.R) return;   // a whole wavefront, and no workgroup-wide team
  const RowCols<VEC, NV> cols(a.D, team, lane);
  fvec<VEC> w[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) w[k] = load_pack<VEC>(a.weight + cols.base[k]);
  const int64_t o = row * a.D;
  const T* x = reinterpret_cast<const T*>(a.x) + o;
  typename Pack<T, VEC>::V xr[NV];
  fvec<VEC> r[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) xr[k] = load_pack<VEC>(x + cols.base[k]);
  if (a.residual) {
#pragma unroll
    for (int k = 0; k < NV; ++k) r[k] = load_pack<VEC>(a.residual + o + cols.base[k]);
  } else {
#pragma unroll
    for (int k = 0; k < NV; ++k) r[k] = fvec<VEC>(0.0f);
  }
  float ss = 0.0f;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const fvec<VEC> xf = convert_pack<float, VEC>(xr[k]);
    if constexpr (DROP) {
      const uint32_t keep = Philox(a.rng).kept_pack<VEC>(cols.base[k], cols.may_move(k), (uint32_t)(a.row0 + row), a.drop);
#pragma unroll
      for (int e = 0; e < VEC; ++e) r[k][e] = keep >> e & 1 ? __fmaf_rn(a.scale, xf[e], r[k][e]) : r[k][e];
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) r[k][e] = __fmaf_rn(a.scale, xf[e], r[k][e]);
    }
    ss += sum_of<VEC>(cols.own(k, r[k] * r[k]));
  }
  const float c = rsqrtf(team_sum<BLOCK>(ss, sm) / (float)a.D + a.eps);
  if (a.residual_out) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (cols.kept(k)) store_pack<VEC>(a.residual_out + o + cols.base[k], r[k]);
  }
  if constexpr (Q8) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      r[k] = r[k] * c * w[k];
#pragma unroll
      for (int e = 0; e < VEC; ++e) m = max(m, magnitude(r[k][e]));
    }
    const Q8Row q8(team_max<BLOCK>(m, smq));
    int8_t* q = a.q + row * a.Dp;
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (cols.kept(k)) store_q8<VEC>(q + cols.base[k], r[k], q8);
    for (int p = a.D + lane; p < a.Dp; p += team) q[p] = 0;
    if (lane == 0) a.qscale[row] = q8.scale;
  } else {
    T* y = reinterpret_cast<T*>(a.y) + o;
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (cols.kept(k)) store_pack<VEC>(y + cols.base[k], convert_pack<T, VEC>(r[k] * c * w[k]));
  }
}

// grid (.., G): block y -> group of columns; Q8 with one group only
template <typename T, int VEC, int NV, bool BLOCK, bool Q8>
__global__ __launch_bounds__(BLOCK ? kBlockThreads : kThreads) void k_gated_norm(GatedNormArgs a) {
  __shared__ float sm[kMaxWaves], smq[kMaxWaves];
  const int team = BLOCK ? blockDim.x : 64;
  const int lane = BLOCK ? threadIdx.x : threadIdx.x & 63;
  const int64_t row = BLOCK ? blockIdx.x : (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  if (row >= a.R) return;   // a whole wavefront, and no workgroup-wide team
  const RowCols<VEC, NV> cols(a.W, team, lane);
  const int64_t c0 = (int64_t)blockIdx.y * a.W;
  fvec<VEC> w[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) w[k] = load_pack<VEC>(a.weight + c0 + cols.base[k]);
  const T* y = reinterpret_cast<const T*>(a.y) + row * a.D + c0;
  const T* z = reinterpret_cast<const T*>(a.z) + row * a.z_stride + c0;
  typename Pack<T, VEC>::V yr[NV], zr[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    yr[k] = load_pack<VEC>(y + cols.base[k]);
    zr[k] = load_pack<VEC>(z + cols.base[k]);
  }
  fvec<VEC> g[NV];
  float ss = 0.0f;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const fvec<VEC> zf = convert_pack<float, VEC>(zr[k]);
    g[k] = convert_pack<float, VEC>(yr[k]) * zf;
#pragma unroll
    for (int e = 0; e < VEC; ++e) g[k][e] *= logistic(zf[e]);
    ss += sum_of<VEC>(cols.own(k, g[k] * g[k]));
  }
  const float c = rsqrtf(team_sum<BLOCK>(ss, sm) / (float)a.W + a.eps);
  if constexpr (Q8) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      g[k] = g[k] * c * w[k];
#pragma unroll
      for (int e = 0; e < VEC; ++e) m = max(m, magnitude(g[k][e]));
    }
    const Q8Row q8(team_max<BLOCK>(m, smq));
    int8_t* q = a.q + row * a.Dp;
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (cols.kept(k)) store_q8<VEC>(q + cols.base[k], g[k], q8);
    for (int p = a.W + lane; p < a.Dp; p += team) q[p] = 0;
    if (lane == 0) a.qscale[row] = q8.scale;
  } else {
    T* out = reinterpret_cast<T*>(a.out) + row * a.D + c0;
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (cols.kept(k)) store_pack<VEC>(out + cols.base[k], convert_pack<T, VEC>(g[k] * c * w[k]));
  }
}

// The gated norm of several groups as one 8-bit row: a workgroup per row.  The
// scale needs every group's norm first, so wavefronts take the groups in turn
// for the mean squares and the largest |g w|, and the second pass reads the
// row again (from the cache) and forms every gate again: 4096 x 5120 bfloat16
// in 4 groups 48 us, against 23.5 us for one group in registers.
template <typename T, int VEC>
__global__ __launch_bounds__(1024) void k_gated_norm_groups_q8(GatedNormArgs a) {
  __shared__ float rms[1024];      // 1/rms of each group (SSD_NORM_MAX_GROUPS_Q8)
  __shared__ float smq[kMaxWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int64_t row = blockIdx.x;
  const T* y = reinterpret_cast<const T*>(a.y) + row * a.D;
  const T* z = reinterpret_cast<const T*>(a.z) + row * a.z_stride;
  int8_t* q = a.q + row * a.Dp;
  auto gated = [&](int c) {
    const fvec<VEC> zf = convert_pack<float, VEC>(load_pack<VEC>(z + c));
    fvec<VEC> g = convert_pack<float, VEC>(load_pack<VEC>(y + c)) * zf;
#pragma unroll
    for (int e = 0; e < VEC; ++e) g[e] *= logistic(zf[e]);
    return g;
  };
  uint32_t m = 0;
  for (int grp = wave; grp < a.G; grp += waves) {
    float ss = 0.0f;
    uint32_t mg = 0;
    for (int c = VEC * lane; c < a.W; c += VEC * 64) {   // VEC divides W
      const fvec<VEC> g = gated(grp * a.W + c);
      const fvec<VEC> gw = g * load_pack<VEC>(a.weight + grp * a.W + c);
      ss += sum_of<VEC>(g * g);
#pragma unroll
      for (int e = 0; e < VEC; ++e) mg = max(mg, magnitude(gw[e]));
    }
    const float c = rsqrtf(wave_sum(ss) / (float)a.W + a.eps);
    // |g c w| <= c max|g w| up to one rounding, which the quantiser's clamp takes
    m = max(m, magnitude(c * __uint_as_float(wave_max(mg))));
    if (lane == 0) rms[grp] = c;
  }
  const Q8Row q8(team_max<true>(m, smq));   // its barrier also covers rms
  for (int c = VEC * threadIdx.x; c < a.Dp; c += VEC * blockDim.x) {
    fvec<VEC> v = fvec<VEC>(0.0f);
    if (c < a.D) v = gated(c) * rms[c / a.W] * load_pack<VEC>(a.weight + c);
    store_q8<VEC>(q + c, v, q8);
  }
  if (threadIdx.x == 0) a.qscale[row] = q8.scale;
}

template <typename T, int VEC, int NV, bool BLOCK>
__global__ __launch_bounds__(BLOCK ? kBlockThreads : kThreads) void k_quantize_q8(const T* v, int64_t R,
                                                                         int32_t K, int32_t Kp,
                                                                         int8_t* q, float* qscale) {
  __shared__ float smq[kMaxWaves];
  const int team = BLOCK ? blockDim.x : 64;
  const int lane = BLOCK ? threadIdx.x : threadIdx.x & 63;
  const int64_t row = BLOCK ? blockIdx.x : (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  if (row >= R) return;   // a whole wavefront, and no workgroup-wide team
  const RowCols<VEC, NV> cols(K, team, lane);
  typename Pack<T, VEC>::V vr[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) vr[k] = load_pack<VEC>(v + row * K + cols.base[k]);
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const fvec<VEC> f = convert_pack<float, VEC>(vr[k]);
#pragma unroll
    for (int e = 0; e < VEC; ++e) m = max(m, magnitude(f[e]));
  }
  const Q8Row q8(team_max<BLOCK>(m, smq));
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (cols.kept(k))
      store_q8<VEC>(q + row * Kp + cols.base[k], convert_pack<float, VEC>(vr[k]), q8);
  for (int p = K + lane; p < Kp; p += team) q[row * Kp + p] = 0;
  if (lane == 0) qscale[row] = q8.scale;
}

// rows wider than the register kernels hold: two passes over the row, a column
// per lane (64 x 130944 float32: 104 us, 0.4 TB/s; 256 x 20000 bfloat16: 12.5)
template <typename T>
__global__ __launch_bounds__(1024) void k_quantize_q8_wide(const T* v, int32_t K, int32_t Kp,
                                                           int8_t* q, float* qscale) {
  __shared__ float smq[kMaxWaves];
  v += (int64_t)blockIdx.x * K;
  q += (int64_t)blockIdx.x * Kp;
  uint32_t m = 0;
  for (int c = threadIdx.x; c < K; c += blockDim.x) m = max(m, magnitude(to_f32(v[c])));
  const Q8Row q8(team_max<true>(m, smq));
  for (int c = threadIdx.x; c < Kp; c += blockDim.x) q[c] = c < K ? q8(to_f32(v[c])) : (int8_t)0;
  if (threadIdx.x == 0) qscale[blockIdx.x] = q8.scale;
}

// ---------------------------------------------------------------------------
// backward: a workgroup takes rows in turn and keeps its columns' part of
// dweight in registers; the parts are summed by a second launch.  The slope is
// c (p - n mean(p n)) with the normalised row n formed first: the equal -c^3 r
// mean(p r) leaves float32 at rows of 10^14 and 10^-13, where c itself does not
// ---------------------------------------------------------------------------

// The partial sums of the wavefronts that shared no row, added in the order of
// the wavefronts, to row `part` of the workspace.
template <int VEC, int NV, bool BLOCK>
__device__ __forceinline__ void store_part(const RowCols<VEC, NV>& cols, fvec<VEC> (&acc)[NV],
                                           float* part) {
  if constexpr (BLOCK) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (cols.kept(k)) store_pack<VEC>(part + cols.base[k], acc[k]);
  } else {
    constexpr int kWaves = kThreads / 64;
    __shared__ fvec<VEC> sm[kWaves - 1][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      __syncthreads();
      if (wave > 0) sm[wave - 1][lane] = acc[k];
      __syncthreads();
      if (wave == 0) {
#pragma unroll
        for (int o = 0; o < kWaves - 1; ++o) acc[k] += sm[o][lane];
        if (cols.kept(k)) store_pack<VEC>(part + cols.base[k], acc[k]);
      }
    }
  }
}

template <typename T, int VEC, int NV, bool BLOCK, bool DROP>
__global__ __launch_bounds__(BLOCK ? kBlockThreads : kThreads) void k_add_norm_backward(AddNormArgs a) {
  __shared__ float sm[2][2 * kMaxWaves];
  const int team = BLOCK ? blockDim.x : 64;
  const int lane = BLOCK ? threadIdx.x : threadIdx.x & 63;
  const int64_t step = BLOCK ? gridDim.x : (int64_t)gridDim.x * (kThreads / 64);
  int64_t row = BLOCK ? blockIdx.x : (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  const RowCols<VEC, NV> cols(a.D, team, lane);
  fvec<VEC> w[NV], acc[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    w[k] = load_pack<VEC>(a.weight + cols.base[k]);
    acc[k] = fvec<VEC>(0.0f);
  }
  for (int par = 0; row < a.R; row += step, par ^= 1) {
    const int64_t o = row * a.D;
    const T* dy = reinterpret_cast<const T*>(a.dy) + o;
    fvec<VEC> r[NV], dr[NV];
    typename Pack<T, VEC>::V dyr[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      r[k] = load_pack<VEC>(a.residual_out + o + cols.base[k]);
      dyr[k] = load_pack<VEC>(dy + cols.base[k]);
    }
    if (a.dres_out) {
#pragma unroll
      for (int k = 0; k < NV; ++k) dr[k] = load_pack<VEC>(a.dres_out + o + cols.base[k]);
    } else {
#pragma unroll
      for (int k = 0; k < NV; ++k) dr[k] = fvec<VEC>(0.0f);
    }
    float ss = 0.0f, pr = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const fvec<VEC> own = cols.own(k, r[k]);
      ss += sum_of<VEC>(own * own);
      pr += sum_of<VEC>(own * (convert_pack<float, VEC>(dyr[k]) * w[k]));
    }
    team_sum2<BLOCK>(ss, pr, sm[par]);
    const float c = rsqrtf(ss / (float)a.D + a.eps);
    const float m = c * (pr / (float)a.D);   // mean(p r c)
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const fvec<VEC> d = convert_pack<float, VEC>(dyr[k]);
      const fvec<VEC> n = r[k] * c;
      acc[k] += d * n;
      dr[k] += c * (d * w[k] - n * m);
      if (cols.kept(k)) {
        if (a.dres) store_pack<VEC>(a.dres + o + cols.base[k], dr[k]);
        if (a.dx) {
          fvec<VEC> dx = a.scale * dr[k];
          if constexpr (DROP) {
            const uint32_t keep = Philox(a.rng).kept_pack<VEC>(cols.base[k], cols.may_move(k), (uint32_t)row, a.drop);
#pragma unroll
            for (int e = 0; e < VEC; ++e) dx[e] = keep >> e & 1 ? dx[e] : 0.0f;
          }
          store_pack<VEC>(reinterpret_cast<T*>(a.dx) + o + cols.base[k], convert_pack<T, VEC>(dx));
        }
      }
    }
  }
  store_part<VEC, NV, BLOCK>(cols, acc, a.part + (int64_t)blockIdx.x * a.D);
}

// grid (parts, G)
template <typename T, int VEC, int NV, bool BLOCK>
__global__ __launch_bounds__(BLOCK ? kBlockThreads : kThreads) void k_gated_norm_backward(GatedNormArgs a) {
  __shared__ float sm[2][2 * kMaxWaves];
  const int team = BLOCK ? blockDim.x : 64;
  const int lane = BLOCK ? threadIdx.x : threadIdx.x & 63;
  const int64_t step = BLOCK ? gridDim.x : (int64_t)gridDim.x * (kThreads / 64);
  int64_t row = BLOCK ? blockIdx.x : (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  const RowCols<VEC, NV> cols(a.W, team, lane);
  const int64_t c0 = (int64_t)blockIdx.y * a.W;
  fvec<VEC> w[NV], acc[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    w[k] = load_pack<VEC>(a.weight + c0 + cols.base[k]);
    acc[k] = fvec<VEC>(0.0f);
  }
  for (int par = 0; row < a.R; row += step, par ^= 1) {
    const int64_t o = row * a.D + c0;
    const T* y = reinterpret_cast<const T*>(a.y) + o;
    const T* z = reinterpret_cast<const T*>(a.z) + row * a.z_stride + c0;
    const T* dout = reinterpret_cast<const T*>(a.dout) + o;
    typename Pack<T, VEC>::V yr[NV], zr[NV], dr[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      yr[k] = load_pack<VEC>(y + cols.base[k]);
      zr[k] = load_pack<VEC>(z + cols.base[k]);
      dr[k] = load_pack<VEC>(dout + cols.base[k]);
    }
    fvec<VEC> s[NV];
    float ss = 0.0f, pg = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const fvec<VEC> zf = convert_pack<float, VEC>(zr[k]);
#pragma unroll
      for (int e = 0; e < VEC; ++e) s[k][e] = logistic(zf[e]);
      const fvec<VEC> g = cols.own(k, convert_pack<float, VEC>(yr[k]) * zf * s[k]);
      ss += sum_of<VEC>(g * g);
      pg += sum_of<VEC>(g * (convert_pack<float, VEC>(dr[k]) * w[k]));
    }
    team_sum2<BLOCK>(ss, pg, sm[par]);
    const float c = rsqrtf(ss / (float)a.W + a.eps);
    const float m = c * (pg / (float)a.W);   // mean(p g c)
    T* dy = reinterpret_cast<T*>(a.dy) + o;
    T* dz = reinterpret_cast<T*>(a.dz) + row * a.dz_stride + c0;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const fvec<VEC> yf = convert_pack<float, VEC>(yr[k]), zf = convert_pack<float, VEC>(zr[k]);
      const fvec<VEC> d = convert_pack<float, VEC>(dr[k]);
      const fvec<VEC> act = zf * s[k], g = yf * act;
      const fvec<VEC> n = g * c;
      acc[k] += d * n;
      const fvec<VEC> dg = c * (d * w[k] - n * m);
      if (cols.kept(k)) {
        store_pack<VEC>(dy + cols.base[k], convert_pack<T, VEC>(dg * act));
        // silu'(z) = s (1 + z (1 - s)) = s + act (1 - s)
        store_pack<VEC>(dz + cols.base[k],
                        convert_pack<T, VEC>(dg * yf * (s[k] + act * (1.0f - s[k]))));
      }
    }
  }
  store_part<VEC, NV, BLOCK>(cols, acc, a.part + (int64_t)blockIdx.x * a.D + c0);
}

// out[c] = sum over the parts, 32 columns per workgroup: 32 lanes' worth of
// parts each, then the 32 sums in order.  4.1 us for 512 x 2560, and as much
// with four columns per lane: the launch, and one trip to what other XCDs have
// just written.
constexpr int kSumCols = 32, kSumSplit = 32;
__global__ __launch_bounds__(kSumCols * kSumSplit) void k_sum_parts(const float* part, float* out,
                                                                    int32_t parts, int64_t D) {
  __shared__ float sm[kSumSplit][kSumCols + 1];
  const int col = threadIdx.x % kSumCols, split = threadIdx.x / kSumCols;
  const int64_t c = (int64_t)blockIdx.x * kSumCols + col;
  float s = 0.0f;
  if (c < D) {
#pragma unroll 16
    for (int p = split; p < parts; p += kSumSplit) s += part[p * D + c];
  }
  sm[split][col] = s;
  __syncthreads();
  if (split == 0 && c < D) {
    for (int o = 1; o < kSumSplit; ++o) s += sm[o][col];
    out[c] = s;
  }
}

hipError_t sum_parts(const float* part, float* out, int64_t parts, int64_t D, hipStream_t s) {
  if (parts == 1) return hipSuccess;   // the part was written to `out` itself
  hipLaunchKernelGGL(k_sum_parts, dim3((unsigned)((D + kSumCols - 1) / kSumCols)),
                     dim3(kSumCols * kSumSplit), 0, s, part, out, (int32_t)parts, D);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// dispatch
// ---------------------------------------------------------------------------
// How the columns of a row are shared: NV vectors per lane, one wavefront per
// row (four rows per workgroup) or a workgroup of `threads` lanes.  Up to
// three vectors per lane a wavefront alone is as fast or faster (768 float32
// columns: 10.7 us against 10.6-11.1; 512 bfloat16: a workgroup per row pays a
// barrier for each 1 KB); beyond, a workgroup with one vector per lane spreads
// a row's latency (2048 bfloat16 columns: 555 us against 578 us with four
// vectors in one wavefront).  A row wider than 512 vectors takes more per
// lane (5120 bfloat16 columns as 5 wavefronts of two vectors: 24.1 us, as 10 of
// one: 28.5 us, three workgroups to a compute unit instead of six).  The
// choice depends on the width alone, so a row's bits do not depend on the batch.
struct RowTeam {
  int nv;
  bool block;
  int threads;
};
RowTeam team_of(int64_t W, int vec) {
  const int64_t chunks = (W + vec - 1) / vec;
  if (chunks <= 3 * 64) return {(int)((chunks + 63) / 64), false, kThreads};
  int nv = 1;
  while (chunks > kBlockThreads * nv) nv *= 2;
  return {nv, true, (int)((chunks + 64 * nv - 1) / (64 * nv)) * 64};
}

// calls f with (vector, vectors per lane, workgroup) as constants
template <int V> using ic = std::integral_constant<int, V>;
template <typename T> constexpr int vec_of() { return sizeof(T) == 2 ? 8 : 4; }

// A row of at most 64 vectors is cut finer while that leaves no second vector
// to a lane: the instructions per row count there, not the bytes (131072 rows
// of 64 bfloat16: add norm 35.2 -> 21.6 us, gradients of the gated norm 83.5 ->
// 43.8 us; of 256: 72.5 -> 70.6 and 101 -> 85 us).
template <typename T, typename F>
hipError_t dispatch(int64_t W, F&& f) {
  constexpr int VEC = vec_of<T>();
  if (W <= 64) return f(ic<1>{}, ic<1>{}, std::false_type{});
  if (W <= 128) return f(ic<2>{}, ic<1>{}, std::false_type{});
  if constexpr (VEC == 8)
    if (W <= 256) return f(ic<4>{}, ic<1>{}, std::false_type{});
  const RowTeam t = team_of(W, VEC);
  if (t.block) {
    if (t.nv == 1) return f(ic<VEC>{}, ic<1>{}, std::true_type{});
    if (t.nv == 2) return f(ic<VEC>{}, ic<2>{}, std::true_type{});
    if (t.nv == 4) return f(ic<VEC>{}, ic<4>{}, std::true_type{});
    if constexpr (VEC == 4) return f(ic<VEC>{}, ic<8>{}, std::true_type{});
    return hipErrorInvalidValue;  // 16384 columns end at four vectors of eight
  }
  if (t.nv == 1) return f(ic<VEC>{}, ic<1>{}, std::false_type{});
  if (t.nv == 2) return f(ic<VEC>{}, ic<2>{}, std::false_type{});
  return f(ic<VEC>{}, ic<3>{}, std::false_type{});
}

// The forward launches one workgroup per row at most.  A grid's threads are
// counted in 32 bits, so rows beyond kRowSlice (1024 threads each) go in
// further launches; f(first row, rows).
constexpr int64_t kRowSlice = 1 << 21;
template <typename F>
hipError_t in_slices(int64_t R, F&& f) {
  for (int64_t r0 = 0; r0 < R; r0 += kRowSlice) {
    const hipError_t e = f(r0, R - r0 < kRowSlice ? R - r0 : kRowSlice);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}
template <typename P>
P* ahead(P* p, int64_t bytes) {
  using B = std::conditional_t<std::is_const_v<P>, const char, char>;
  return p ? reinterpret_cast<P*>(reinterpret_cast<B*>(p) + bytes) : p;
}

// workgroups for R rows
int64_t row_blocks(const RowTeam& t, int64_t R) {
  return t.block ? R : (R + kThreads / 64 - 1) / (kThreads / 64);
}

template <typename T>
hipError_t add_norm_t(const AddNormArgs& a, hipStream_t s) {
  const RowTeam t = team_of(a.D, vec_of<T>());
  const dim3 grid((unsigned)row_blocks(t, a.R)), block(t.threads);
  return dispatch<T>(a.D, [&](auto vec, auto nv, auto blk) {
    if (a.q)
      hipLaunchKernelGGL((k_add_norm<T, vec, nv, blk, true, false>), grid, block, 0, s, a);
    else if (a.rng)
      hipLaunchKernelGGL((k_add_norm<T, vec, nv, blk, false, true>), grid, block, 0, s, a);
    else
      hipLaunchKernelGGL((k_add_norm<T, vec, nv, blk, false, false>), grid, block, 0, s, a);
    return hipGetLastError();
  });
}

template <typename T>
hipError_t gated_norm_t(const GatedNormArgs& a, hipStream_t s) {
  constexpr int VEC = vec_of<T>();
  if (a.q && a.G > 1) {
    const dim3 grid((unsigned)a.R), block(a.D >= 4096 ? 1024 : 256);
    if (a.W % VEC == 0)
      hipLaunchKernelGGL((k_gated_norm_groups_q8<T, VEC>), grid, block, 0, s, a);
    else
      hipLaunchKernelGGL((k_gated_norm_groups_q8<T, 1>), grid, block, 0, s, a);
    return hipGetLastError();
  }
  const RowTeam t = team_of(a.W, VEC);
  const dim3 grid((unsigned)row_blocks(t, a.R), (unsigned)a.G), block(t.threads);
  return dispatch<T>(a.W, [&](auto vec, auto nv, auto blk) {
    if (a.q)
      hipLaunchKernelGGL((k_gated_norm<T, vec, nv, blk, true>), grid, block, 0, s, a);
    else
      hipLaunchKernelGGL((k_gated_norm<T, vec, nv, blk, false>), grid, block, 0, s, a);
    return hipGetLastError();
  });
}

template <typename T>
hipError_t quantize_t(const T* v, int64_t R, int32_t K, int32_t Kp, int8_t* q, float* qscale,
                      hipStream_t s) {
  constexpr int VEC = vec_of<T>();
  if (K > 16384) {
    hipLaunchKernelGGL(k_quantize_q8_wide<T>, dim3((unsigned)R), dim3(1024), 0, s, v, K, Kp, q, qscale);
    return hipGetLastError();
  }
  const RowTeam t = team_of(K, VEC);
  const dim3 grid((unsigned)row_blocks(t, R)), block(t.threads);
  return dispatch<T>(K, [&](auto vec, auto nv, auto blk) {
    hipLaunchKernelGGL((k_quantize_q8<T, vec, nv, blk>), grid, block, 0, s, v, R, K, Kp, q, qscale);
    return hipGetLastError();
  });
}

// Workgroups of the gradients, each leaving one row of dweight's parts: two
// per compute unit over all groups (one, three and four per unit measured 37.2,
// 34.5 and 37.6 us against 32.3 us at 4096 x 2560).
int64_t backward_parts(int64_t R, int64_t G, int64_t W, bool io_bf16) {
  const int64_t n = row_blocks(team_of(W, io_bf16 ? 8 : 4), R), cap = (2 * kCus + G - 1) / G;
  // a few rows: one workgroup takes them in turn and its part is the sum, which
  // saves the second launch
  return n <= 4 ? 1 : n < cap ? n : cap;
}

}  // namespace

int64_t add_norm_backward_parts(int64_t R, int64_t D, bool io_bf16) {
  return backward_parts(R, 1, D, io_bf16);
}
int64_t gated_norm_backward_parts(int64_t R, int64_t G, int64_t W, bool io_bf16) {
  return backward_parts(R, G, W, io_bf16);
}

hipError_t launch_add_norm(const AddNormArgs& all, bool io_bf16, hipStream_t s) {
  return in_slices(all.R, [&](int64_t r0, int64_t rows) {
    AddNormArgs a = all;
    const int64_t e = r0 * a.D;
    const size_t es = io_bf16 ? 2 : 4;
    a.x = ahead(a.x, e * es);
    a.residual = ahead(a.residual, e * 4);
    a.y = ahead(a.y, e * es);
    a.q = ahead(a.q, r0 * a.Dp);
    a.qscale = ahead(a.qscale, r0 * 4);
    a.residual_out = ahead(a.residual_out, e * 4);
    a.R = rows;
    a.row0 = r0;
    return io_bf16 ? add_norm_t<bf16>(a, s) : add_norm_t<float>(a, s);
  });
}
hipError_t launch_gated_norm(const GatedNormArgs& all, bool io_bf16, hipStream_t s) {
  return in_slices(all.R, [&](int64_t r0, int64_t rows) {
    GatedNormArgs a = all;
    const size_t es = io_bf16 ? 2 : 4;
    a.y = ahead(a.y, r0 * a.D * es);
    a.z = ahead(a.z, r0 * a.z_stride * es);
    a.out = ahead(a.out, r0 * a.D * es);
    a.q = ahead(a.q, r0 * a.Dp);
    a.qscale = ahead(a.qscale, r0 * 4);
    a.R = rows;
    return io_bf16 ? gated_norm_t<bf16>(a, s) : gated_norm_t<float>(a, s);
  });
}

hipError_t launch_add_norm_backward(const AddNormArgs& all, bool io_bf16, hipStream_t s) {
  AddNormArgs a = all;
  const int64_t parts = add_norm_backward_parts(a.R, a.D, io_bf16);
  if (parts == 1) a.part = a.dweight;
  auto go = [&](auto zero) {
    using T = decltype(zero);
    const RowTeam t = team_of(a.D, vec_of<T>());
    return dispatch<T>(a.D, [&](auto vec, auto nv, auto blk) {
      if (a.rng)
        hipLaunchKernelGGL((k_add_norm_backward<T, vec, nv, blk, true>), dim3((unsigned)parts),
                           dim3(t.threads), 0, s, a);
      else
        hipLaunchKernelGGL((k_add_norm_backward<T, vec, nv, blk, false>), dim3((unsigned)parts),
                           dim3(t.threads), 0, s, a);
      return hipGetLastError();
    });
  };
  const hipError_t e = io_bf16 ? go(bf16{}) : go(float{});
  return e != hipSuccess ? e : sum_parts(a.part, a.dweight, parts, a.D, s);
}

hipError_t launch_gated_norm_backward(const GatedNormArgs& all, bool io_bf16, hipStream_t s) {
  GatedNormArgs a = all;
  const int64_t parts = gated_norm_backward_parts(a.R, a.G, a.W, io_bf16);
  if (parts == 1) a.part = a.dweight;
  auto go = [&](auto zero) {
    using T = decltype(zero);
    const RowTeam t = team_of(a.W, vec_of<T>());
    return dispatch<T>(a.W, [&](auto vec, auto nv, auto blk) {
      hipLaunchKernelGGL((k_gated_norm_backward<T, vec, nv, blk>),
                         dim3((unsigned)parts, (unsigned)a.G), dim3(t.threads), 0, s, a);
      return hipGetLastError();
    });
  };
  const hipError_t e = io_bf16 ? go(bf16{}) : go(float{});
  return e != hipSuccess ? e : sum_parts(a.part, a.dweight, parts, a.D, s);
}

hipError_t launch_quantize_q8(const void* v, bool v_bf16, int64_t R, int32_t K, int32_t Kp,
                              int8_t* q, float* qscale, hipStream_t s) {
  return in_slices(R, [&](int64_t r0, int64_t rows) {
    int8_t* qr = q + r0 * Kp;
    return v_bf16 ? quantize_t(static_cast<const bf16*>(v) + r0 * K, rows, K, Kp, qr, qscale + r0, s)
                  : quantize_t(static_cast<const float*>(v) + r0 * K, rows, K, Kp, qr, qscale + r0, s);
  });
}

}  // namespace ssd
