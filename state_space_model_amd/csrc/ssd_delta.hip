// The gated delta rule for gfx950: the chunked scan and the one-token step.
//
// Per (b, h), with a_t = exp(Delta_t A), b_t = sigmoid(beta_t) and unit k, q:
//   S_t = a_t S_{t-1} + b_t (v_t - a_t S_{t-1} k_t) k_t^T,   y_t = scale S_t q_t
// In a chunk of C = 64 tokens that starts from S (cum_i the sum of the decay up
// to token i, gamma_i = e^cum_i, D_ij = e^(cum_i - cum_j)):
//   L_ij = b_i D_ij k_i.k_j  (i > j)     the writes that a write has to allow for
//   W    = (1 + L)^-1 diag(b) (V - diag(gamma) K S^T)     the writes [C, P]
//   Y    = scale (diag(gamma) Q S^T + (D o Q K^T)_(i >= j) W)
//   S'   = gamma_last S + W^T diag(e^(cum_last - cum)) K
// k_delta_prep forms (1 + L)^-1 and D o Q K^T of every chunk, which need no
// state, in parallel; k_delta_chain walks the chunks of one head and a slice of
// its value columns in order, the state in matrix-core accumulators.
#include "ssd_delta.h"

#include <type_traits>

namespace ssd {
namespace delta {
namespace {

// ---------------------------------------------------------------------------
// Chunk by chunk, before the states are known.
// ---------------------------------------------------------------------------
// sum of squares of the lane's row
template <int PI, int KS>
__device__ __forceinline__ float row_squares(const Frag<PI> (&f)[KS]) {
  float ss = 0.0f;
#pragma unroll
  for (int s = 0; s < KS; ++s)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float x = (float)f[s].p[PI - 1][e];
#pragma unroll
      for (int i = PI - 2; i >= 0; --i) x += (float)f[s].p[i][e];
      ss = fmaf(x, x, ss);
    }
  ss += __shfl_xor(ss, 16, 64);
  ss += __shfl_xor(ss, 32, 64);
  return ss;
}

// GRADS: for the gradients, whose chain from the last chunk needs both matrices
// transposed and no output.
template <typename IO, int KP, bool GRADS>
__global__ __launch_bounds__(kThreads) void k_delta_prep(DeltaArgs a) {
  constexpr int PI = Planes<IO>::in, PY = Planes<IO>::y;
  constexpr int KS = KP / 32, KST = KP + 8;
  __shared__ __align__(16) bf16 s_k[PI * C * KST];
  __shared__ __align__(16) float s_a[C * kPairStride], s_x[C * kPairStride];
  __shared__ float s_hi[C], s_lo[C], s_beta[C], s_rk[C], s_rq[C];

  const int64_t id = xcd_remap(blockIdx.x, gridDim.x);
  const int64_t h = id % a.H, c = id / a.H % a.Nc, b = id / a.H / a.Nc;
  const int64_t g = h / (a.H / a.G);
  const int64_t at = chunk_at(a, b * a.H + h, c);
  const int64_t t0 = c * C, row0 = b * a.T + t0, left = a.T - t0;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, j = lane & 15, q = lane >> 4;

  Frag<PI> kf[KS], qf[KS];
  load_rows<IO, KP>(kf, static_cast<const IO*>(a.k) + g * a.N, a.k_stride, row0, left, a.N, 16 * w + j, q);
  load_rows<IO, KP>(qf, static_cast<const IO*>(a.q) + g * a.N, a.q_stride, row0, left, a.N, 16 * w + j, q);

  // Decay sums in units of log 2, in float64: differences of them are
  // exponents, and float32 sums over a chunk of strong decays would be off by
  // more than the results may be.  -1e5 stands for every decay below it (2^-1e5
  // is 0) and keeps infinities out of the differences.
  if (w == 0) {
    const bool in = lane < left;
    const int64_t th = (row0 + (in ? lane : 0)) * a.H + h;
    const float bias = a.dt_bias ? a.dt_bias[h] : 0.0f;
    const float d = delta_of(a.dt[th] + bias, a.softplus, a.dt_min, a.dt_max);
    double sum = (double)d * (double)a.A[h] * 1.4426950408889634;
    sum = in ? (sum < -1e5 ? -1e5 : sum) : 0.0;
    for (int off = 1; off < 64; off <<= 1) {
      const double o = __shfl_up(sum, off, 64);
      if (lane >= off) sum += o;
    }
    const float hi = (float)sum;
    s_hi[lane] = hi;
    s_lo[lane] = (float)(sum - (double)hi);
    const float beta = a.beta[th];
    s_beta[lane] = in ? (a.sigmoid ? sigmoid_of(beta) : beta) : 0.0f;
  }
  const bool row_in = 16 * w + j < left;
  {
    const float kk = row_squares<PI, KS>(kf), qq = row_squares<PI, KS>(qf);
    if (q == 0) {
      s_rk[16 * w + j] = !row_in ? 0.0f : a.unit ? 1.0f / sqrtf(kk + a.norm_eps) : 1.0f;
      s_rq[16 * w + j] = !row_in ? 0.0f : a.scale * (a.unit ? 1.0f / sqrtf(qq + a.norm_eps) : 1.0f);
    }
  }
#pragma unroll
  for (int s = 0; s < KS; ++s)
#pragma unroll
    for (int i = 0; i < PI; ++i)
      *reinterpret_cast<bf16x8*>(&s_k[i * C * KST + (16 * w + j) * KST + 32 * s + 8 * q]) = kf[s].p[i];
  __syncthreads();

  // rows of wavefront w against key tokens up to them: L to LDS, D o Q K^T kept
  f32x4 p[4];
#pragma unroll
  for (int jt = 0; jt < 4; ++jt) {
    p[jt] = f32x4{0, 0, 0, 0};
    if (jt > w) continue;
    f32x4 kk = {0, 0, 0, 0}, qk = {0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const auto bf = load_planes<PI>(&s_k[(16 * jt + j) * KST + 32 * s + 8 * q], C * KST);
      kk = mma(kf[s], bf, kk);
      qk = mma(qf[s], bf, qk);
    }
    const int col = 16 * jt + j;
    const float chi = s_hi[col], clo = s_lo[col], rk = s_rk[col];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * w + 4 * q + r;
      const float dec = exp2_of((s_hi[row] - chi) + (s_lo[row] - clo)) * rk;
      s_a[row * kPairStride + col] = row > col ? s_beta[row] * s_rk[row] * dec * kk[r] : 0.0f;
      p[jt][r] = row >= col ? s_rq[row] * dec * qk[r] : 0.0f;
    }
  }

  // The inverse of the diagonal 16 x 16 block by forward substitution, lane
  // column j (each group of 16 lanes the same).  Only this wavefront wrote the block.
  __builtin_amdgcn_wave_barrier();
  f32x4 x[4];  // block (w + d, w) in the layout of a result
  {
    float col[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float acc = i == j ? 1.0f : 0.0f;
      const float* row = &s_a[(16 * w + i) * kPairStride + 16 * w];
#pragma unroll
      for (int m = 0; m < i; ++m) acc = fmaf(-row[m], col[m], acc);
      col[i] = acc;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      x[0][r] = q == 0 ? col[r] : q == 1 ? col[4 + r] : q == 2 ? col[8 + r] : col[12 + r];
      s_x[(16 * w + 4 * q + r) * kPairStride + 16 * w + j] = x[0][r];
    }
  }
  __syncthreads();
  // the blocks below it, X_iw = -X_ii sum_m L_im X_mw; zeros above it
#pragma unroll
  for (int d = 1; d < 4; ++d) {
    const int i = w + d;
    if (i < 4) {
      f32x4 acc = {0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < d; ++e)
        acc = mma16(*reinterpret_cast<const f32x4*>(&s_a[(16 * i + j) * kPairStride + 16 * (w + e) + 4 * q]),
                    x[e], acc);
      acc = mma16(*reinterpret_cast<const f32x4*>(&s_x[(16 * i + j) * kPairStride + 16 * i + 4 * q]), acc,
                  f32x4{0, 0, 0, 0});
      x[d] = -acc;
#pragma unroll
      for (int r = 0; r < 4; ++r) s_x[(16 * i + 4 * q + r) * kPairStride + 16 * w + j] = x[d][r];
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)  // block (i - 4, w): above the diagonal
        s_x[(16 * (i - 4) + 4 * q + r) * kPairStride + 16 * w + j] = 0.0f;
    }
  }
  __syncthreads();
#pragma unroll
  for (int jt = 0; jt < 4; ++jt)
#pragma unroll
    for (int r = 0; r < 4; ++r) s_a[(16 * w + 4 * q + r) * kPairStride + 16 * jt + j] = p[jt][r];
  __syncthreads();

  // fragments of row tile w: 32 columns for tiles 0 and 1, 64 for 2 and 3
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    if (s > (w >> 1)) continue;
    const int f = lower_frag(w, s);
    float vx[8], vp[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      vx[e] = s_x[(16 * w + j) * kPairStride + 32 * s + 8 * q + e];
      vp[e] = s_a[(16 * w + j) * kPairStride + 32 * s + 8 * q + e];
    }
    store_frag(a.inv, at, f, lane, split8<3>(vx));
    if constexpr (!GRADS) store_frag(a.qk, at, f, lane, split8<PY>(vp));
  }
  if constexpr (GRADS) {
    // transposed: row tiles 0 and 1 reach over all columns, 2 and 3 over the last 32
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (s < (w >> 1)) continue;
      float vx[8], vp[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        vx[e] = s_x[(32 * s + 8 * q + e) * kPairStride + 16 * w + j];
        vp[e] = s_a[(32 * s + 8 * q + e) * kPairStride + 16 * w + j];
      }
      store_frag(a.inv_t, at, upper_frag(w, s), lane, split8<3>(vx));
      store_frag(a.qk, at, upper_frag(w, s), lane, split8<3>(vp));
    }
  }

  // what multiplies a token's rows: v, K S^T, its write on the way to the end,
  // Q S^T
  if (tid < C) {
    const float gamma = exp2_of(s_hi[tid] + s_lo[tid]), beta = s_beta[tid];
    const float end = exp2_of((s_hi[C - 1] - s_hi[tid]) + (s_lo[C - 1] - s_lo[tid]));
    a.gate[at * C + tid] = make_float4(beta, beta * gamma * s_rk[tid], end * s_rk[tid],
                                       gamma * s_rq[tid]);
    if (tid == C - 1) a.whole[at] = gamma;
    if constexpr (GRADS) a.row[at * C + tid] = make_float4(s_rk[tid], s_rq[tid], s_hi[tid], s_lo[tid]);
  }
}

// ---------------------------------------------------------------------------
// The chunks of one (b, h) in order, 16 NT value columns.
//
// The state's slice S^T [key, value] stays in accumulators (wavefront w: keys
// KP / 4 w ..); its planes go to LDS value-major, key-contiguous, as the right
// operand of K S^T and Q S^T.  What follows from them (right sides, writes)
// goes to LDS value-major and token-contiguous, one 8-byte store per plane and
// four tokens, since a result's lane holds four consecutive rows of a column.
// ---------------------------------------------------------------------------
// KEEP: for the gradients, which need the state entering every chunk and its
// writes, and no output.
template <typename IO, int KP, int NT, bool KEEP>
__global__ __launch_bounds__(kThreads) void k_delta_chain(DeltaArgs a) {
  constexpr int PI = Planes<IO>::in, PY = Planes<IO>::y;
  constexpr int KS = KP / 32, KST = KP + 8, KT = KP / 64, W = 16 * NT;
  __shared__ __align__(16) bf16 s_k[2][PI * C * KST];
  __shared__ __align__(16) bf16 s_s[3 * W * KST];
  __shared__ __align__(16) bf16 s_r[3 * W * kTokStride];   // right sides
  __shared__ __align__(16) bf16 s_e[3 * W * kTokStride];   // writes, decayed to the chunk's end
  __shared__ __align__(16) bf16 s_w[PY * W * kTokStride];  // writes

  const int64_t slices = (a.P + W - 1) / W;
  const int64_t id = xcd_remap(blockIdx.x, gridDim.x);
  const int64_t bh = id / slices, b = bh / a.H, h = bh % a.H, g = h / (a.H / a.G);
  const int col0 = (int)(id % slices) * W;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, j = lane & 15, q = lane >> 4;
  const IO* kb = static_cast<const IO*>(a.k) + g * a.N;
  const IO* qb = static_cast<const IO*>(a.q) + g * a.N;
  const IO* vb = static_cast<const IO*>(a.v) + h * a.P;
  IO* yb = KEEP ? nullptr : static_cast<IO*>(a.y) + h * a.P;
  bool col_in[NT];
  int col[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    col_in[n] = col0 + 16 * n + j < a.P;
    col[n] = col_in[n] ? col0 + 16 * n + j : 0;
  }

  // state tiles (keys 16 (KT w + t) + 4 q .. + 3, value column j of tile n)
  f32x4 st[NT][KT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const int key = 16 * (KT * w + t) + 4 * q;
      st[n][t] = f32x4{0, 0, 0, 0};
      if (a.h0 && col_in[n] && key < a.N)
        st[n][t] = *reinterpret_cast<const f32x4*>(a.h0 + (bh * a.P + col[n]) * a.N + key);
      store_split4<3>(&s_s[(16 * n + j) * KST + key], W * KST, st[n][t]);
    }

  Frag<PI> kf[KS], qf[KS];
  Frag<3> xf[2];
  Frag<PY> pf[2];
  float4 gate[4];
  IO v[NT][4];
  float whole;
  auto load_chunk = [&](int64_t c) {
    const int64_t t0 = c * C, row0 = b * a.T + t0, left = a.T - t0, at = chunk_at(a, bh, c);
    load_rows<IO, KP>(kf, kb, a.k_stride, row0, left, a.N, 16 * w + j, q);
    if constexpr (!KEEP) load_rows<IO, KP>(qf, qb, a.q_stride, row0, left, a.N, 16 * w + j, q);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int tok = 16 * w + 4 * q + r;
      gate[r] = a.gate[at * C + tok];
      const IO* row = vb + (row0 + (tok < left ? tok : 0)) * a.v_stride;
#pragma unroll
      for (int n = 0; n < NT; ++n) v[n][r] = row[col[n]];
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (s > (w >> 1)) continue;
      xf[s] = load_frag<3>(a.inv, at, lower_frag(w, s), lane);
      if constexpr (!KEEP) pf[s] = load_frag<PY>(a.qk, at, lower_frag(w, s), lane);
    }
    whole = a.whole[at];
  };
  auto store_k = [&](bf16* to) {
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int i = 0; i < PI; ++i)
        *reinterpret_cast<bf16x8*>(&to[i * C * KST + (16 * w + j) * KST + 32 * s + 8 * q]) = kf[s].p[i];
  };
  load_chunk(0);
  store_k(s_k[0]);
  __syncthreads();

  for (int64_t c = 0; c < a.Nc; ++c) {
    const int64_t t0 = c * C, row0 = b * a.T + t0, left = a.T - t0;
    const bf16* sk = s_k[c & 1];
    if constexpr (KEEP) store_state<NT, KT>(a.enter + chunk_at(a, bh, c) * a.P * a.N, st, a.N, col, col_in, w, q);
    // K S^T and Q S^T of the wavefront's tokens; the right sides b (v - gamma K S^T)
    f32x4 y[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      f32x4 ks = {0, 0, 0, 0}, qs = {0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const auto sf = load_planes<3>(&s_s[(16 * n + j) * KST + 32 * s + 8 * q], W * KST);
        ks = mma(kf[s], sf, ks);
        if constexpr (!KEEP) {
          Frag<PY> sy;
#pragma unroll
          for (int i = 0; i < PY; ++i) sy.p[i] = sf.p[i];
          qs = mma(qf[s], sy, qs);
        }
      }
      f32x4 rs;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float vv = 16 * w + 4 * q + r < left && col_in[n] ? to_f32(v[n][r]) : 0.0f;
        rs[r] = gate[r].x * vv - gate[r].y * ks[r];
        y[n][r] = gate[r].w * qs[r];
      }
      store_split4<3>(&s_r[(16 * n + j) * kTokStride + 16 * w + 4 * q], W * kTokStride, rs);
    }
    __syncthreads();
    // the writes
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      f32x4 ws = {0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (s > (w >> 1)) continue;
        ws = mma(xf[s], load_planes<3>(&s_r[(16 * n + j) * kTokStride + 32 * s + 8 * q], W * kTokStride), ws);
      }
      f32x4 es;
#pragma unroll
      for (int r = 0; r < 4; ++r) es[r] = gate[r].z * ws[r];
      const int o = (16 * n + j) * kTokStride + 16 * w + 4 * q;
      store_split4<3>(&s_e[o], W * kTokStride, es);
      if constexpr (!KEEP) {
        store_split4<PY>(&s_w[o], W * kTokStride, ws);
      } else {
        if (col_in[n])
          *reinterpret_cast<f32x4*>(a.write + (chunk_at(a, bh, c) * a.P + col[n]) * C + 16 * w + 4 * q) = ws;
      }
    }
    __syncthreads();
    // outputs
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if constexpr (KEEP) break;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (s > (w >> 1)) continue;
        y[n] = mma(pf[s], load_planes<PY>(&s_w[(16 * n + j) * kTokStride + 32 * s + 8 * q], W * kTokStride),
                   y[n]);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int tok = 16 * w + 4 * q + r;
        if (tok < left && col_in[n])
          yb[(row0 + tok) * (a.H * a.P) + col[n]] = to_io<IO>(y[n][r]);
      }
    }
    // the state at the chunk's end
    const float decay = whole;
    if (c + 1 < a.Nc) load_chunk(c + 1);
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      Frag<PI> ka[2];
#pragma unroll
      for (int s = 0; s < 2; ++s)
        ka[s] = load_planes_tr<PI>(sk, C * KST, KST, 32 * s, 16 * (KT * w + t), lane);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        f32x4 acc = {0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < 2; ++s)
          acc = mma(ka[s], load_planes<3>(&s_e[(16 * n + j) * kTokStride + 32 * s + 8 * q], W * kTokStride),
                    acc);
#pragma unroll
        for (int r = 0; r < 4; ++r) st[n][t][r] = fmaf(decay, st[n][t][r], acc[r]);
        store_split4<3>(&s_s[(16 * n + j) * KST + 16 * (KT * w + t) + 4 * q], W * KST, st[n][t]);
      }
    }
    store_k(s_k[(c + 1) & 1]);
    __syncthreads();
  }
  if (!KEEP && a.state) store_state<NT, KT>(a.state + bh * a.P * a.N, st, a.N, col, col_in, w, q);
}

// ---------------------------------------------------------------------------
// One token.  A row p of the state needs two dot products, S k and S q; the
// token's own part of y is its write times k.q.
//   y = a S.q + u k.q,  S' = a S + u k,  u = b (v - a S.k)
// NL lanes of four keys share a row; N / 4 of them have keys.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float lanes_sum(float v, int nl) {
  for (int off = nl >> 1; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

template <typename IO, int NL, int ROWS>
__global__ __launch_bounds__(kThreads) void k_delta_step(DeltaArgs a) {
  constexpr int per_pass = kThreads / NL;
  const int runs = (a.P + per_pass * ROWS - 1) / (per_pass * ROWS);
  const int64_t bh = blockIdx.x / runs, b = bh / a.H, h = bh % a.H, g = h / (a.H / a.G);
  const int p0 = (int)(blockIdx.x % runs) * per_pass * ROWS + threadIdx.x / NL;
  const int key = 4 * (threadIdx.x % NL);
  const bool key_in = key < a.N;
  float4* state = reinterpret_cast<float4*>(a.state + bh * a.P * a.N) + (key_in ? key / 4 : 0);
  float4 s[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int p = min(p0 + i * per_pass, a.P - 1);
    const f32x4 t = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(state + (int64_t)p * (a.N / 4)));
    s[i] = make_float4(t[0], t[1], t[2], t[3]);
  }
  float kv[4], qv[4], kk = 0.0f, qq = 0.0f, kq = 0.0f;
  const IO* kr = static_cast<const IO*>(a.k) + b * a.k_stride + g * a.N + (key_in ? key : 0);
  const IO* qr = static_cast<const IO*>(a.q) + b * a.q_stride + g * a.N + (key_in ? key : 0);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    kv[e] = key_in ? to_f32(kr[e]) : 0.0f;
    qv[e] = key_in ? to_f32(qr[e]) : 0.0f;
    kk = fmaf(kv[e], kv[e], kk);
    qq = fmaf(qv[e], qv[e], qq);
    kq = fmaf(kv[e], qv[e], kq);
  }
  kk = lanes_sum(kk, NL);
  qq = lanes_sum(qq, NL);
  kq = lanes_sum(kq, NL);
  const float rk = a.unit ? 1.0f / sqrtf(kk + a.norm_eps) : 1.0f;
  const float rq = a.scale * (a.unit ? 1.0f / sqrtf(qq + a.norm_eps) : 1.0f);
  const float bias = a.dt_bias ? a.dt_bias[h] : 0.0f;
  const float d = delta_of(a.dt[bh] + bias, a.softplus, a.dt_min, a.dt_max);
  const float alpha = expf(d * a.A[h]);
  const float beta = a.sigmoid ? sigmoid_of(a.beta[bh]) : a.beta[bh];
  const IO* vr = static_cast<const IO*>(a.v) + b * a.v_stride + h * a.P;
  IO* yr = static_cast<IO*>(a.y) + bh * a.P;
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int p = p0 + i * per_pass;
    float sk = s[i].x * kv[0] + s[i].y * kv[1] + s[i].z * kv[2] + s[i].w * kv[3];
    float sq = s[i].x * qv[0] + s[i].y * qv[1] + s[i].z * qv[2] + s[i].w * qv[3];
    sk = lanes_sum(key_in ? sk : 0.0f, NL);
    sq = lanes_sum(key_in ? sq : 0.0f, NL);
    if (p < a.P) {
      const float u = beta * (to_f32(vr[p]) - alpha * rk * sk), uk = u * rk;
      if (key_in)
        __builtin_nontemporal_store(f32x4{fmaf(alpha, s[i].x, uk * kv[0]), fmaf(alpha, s[i].y, uk * kv[1]),
                                          fmaf(alpha, s[i].z, uk * kv[2]), fmaf(alpha, s[i].w, uk * kv[3])},
                                    reinterpret_cast<f32x4*>(state + (int64_t)p * (a.N / 4)));
      if (threadIdx.x % NL == 0) yr[p] = to_io<IO>(rq * (alpha * sq + uk * kq));
    }
  }
}

// GRADS: the forward part of the gradients, which keeps states and writes
template <typename IO, int KP, bool GRADS>
hipError_t launch_scan(const DeltaArgs& a, hipStream_t stream) {
  const int64_t chunks = a.Bt * a.H * a.Nc;
  hipLaunchKernelGGL((k_delta_prep<IO, KP, GRADS>), dim3((unsigned)chunks), dim3(kThreads), 0, stream, a);
  hipLaunchKernelGGL((k_delta_chain<IO, KP, 1, GRADS>), dim3((unsigned)(a.Bt * a.H * ((a.P + 15) / 16))),
                     dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

template <bool GRADS>
hipError_t launch_scan_of(const DeltaArgs& a, bool io_bf16, hipStream_t stream) {
  if (a.N <= 64)
    return io_bf16 ? launch_scan<bf16, 64, GRADS>(a, stream) : launch_scan<float, 64, GRADS>(a, stream);
  return io_bf16 ? launch_scan<bf16, 128, GRADS>(a, stream) : launch_scan<float, 128, GRADS>(a, stream);
}

template <typename IO>
hipError_t launch_step(const DeltaArgs& a, hipStream_t stream) {
  auto go = [&](auto nl) {
    constexpr int NL = decltype(nl)::value, per_pass = kThreads / NL;
    const int64_t runs = (a.P + 2 * per_pass - 1) / (2 * per_pass);
    hipLaunchKernelGGL((k_delta_step<IO, NL, 2>), dim3((unsigned)(a.Bt * a.H * runs)), dim3(kThreads), 0,
                       stream, a);
  };
  if (a.N <= 64) go(std::integral_constant<int, 16>{});
  else go(std::integral_constant<int, 32>{});
  return hipGetLastError();
}

}  // namespace
}  // namespace delta

size_t delta_workspace(DeltaArgs& a, bool io_bf16, bool grads, char* ws) {
  const size_t n = (size_t)(a.Bt * a.H * a.Nc), C = kDeltaChunk;
  const size_t frags = delta::kTriFrags * delta::kFrag * sizeof(bf16);
  size_t at = 0;
  auto take = [&](auto*& p, size_t bytes) {
    if (ws) p = reinterpret_cast<std::remove_reference_t<decltype(p)>>(ws + at);
    at += (bytes + 255) / 256 * 256;
  };
  take(a.gate, n * C * sizeof(float4));
  take(a.whole, n * sizeof(float));
  take(a.inv, n * 3 * frags);
  take(a.qk, n * (io_bf16 && !grads ? 2 : 3) * frags);
  if (grads) {
    const size_t state = (size_t)a.P * a.N * sizeof(float), cols = (size_t)a.P * C * sizeof(float);
    const size_t keys = (size_t)(a.Bt * a.T * a.H * a.N) * sizeof(float);
    take(a.row, n * C * sizeof(float4));
    take(a.inv_t, n * 3 * frags);
    take(a.enter, n * state);
    take(a.leave, n * state);
    take(a.write, n * cols);
    take(a.dright, n * cols);
    take(a.part_q, keys);
    take(a.part_k, keys);
    take(a.part_h, n * 2 * sizeof(float));
  }
  return at;
}

hipError_t launch_delta_scan(const DeltaArgs& a, bool io_bf16, hipStream_t stream) {
  return delta::launch_scan_of<false>(a, io_bf16, stream);
}

hipError_t launch_delta_states(const DeltaArgs& a, bool io_bf16, hipStream_t stream) {
  return delta::launch_scan_of<true>(a, io_bf16, stream);
}

hipError_t launch_delta_step(const DeltaArgs& a, bool io_bf16, hipStream_t stream) {
  return io_bf16 ? delta::launch_step<bf16>(a, stream) : delta::launch_step<float>(a, stream);
}

}  // namespace ssd
