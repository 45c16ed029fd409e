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

namespace ssd {
namespace delta {
namespace {

// ---------------------------------------------------------------------------
// Chunk by chunk, before the states are known.
// ---------------------------------------------------------------------------
// Wavefront w owns tokens 16 w .. + 15 as rows of both matrices, and forms them
// transposed: a result's lane then holds four consecutive columns of its row,
// and two tiles of columns are a fragment of the matrix as it is (ssd_delta.h).
//
// The inverse X of 1 + L: the diagonal 16 x 16 blocks by back substitution, a
// lane a row (X (1 + L) = 1: x_c = [c = row] - sum_{m > c} x_m L_mc); the blocks
// left of them, nearest first, from X_ij = -(sum_{j < m <= i} X_im L_mj) X_jj on
// the float32 matrix core, transposed.
//
// GRADS: for the gradients, whose chain from the last chunk needs both matrices
// transposed and no output.
template <typename IO, int KP, bool FULL, bool GRADS>
__global__ __launch_bounds__(kThreads, sizeof(IO) == 2 ? 4 : 2) void k_delta_prep(DeltaArgs a) {
  constexpr int PI = Planes<IO>::in, PY = Planes<IO>::y;
  constexpr int KS = KP / 32, KST = KP + 8, kDiag = 20;
  constexpr int k_bytes = PI * C * KST * 2, l_bytes = (GRADS ? 2 : 1) * C * kPairStride * 4;
  // the keys, then L transposed ([column][row]), then for GRADS both results: a
  // workgroup in 24 KB (bfloat16), and six of them to a compute unit hide one
  // another's chain of dependent steps
  __shared__ __align__(16) char lds[k_bytes > l_bytes ? k_bytes : l_bytes];
  __shared__ __align__(16) float s_d[4 * 16 * kDiag];     // inverse diagonal blocks, transposed
  __shared__ __align__(16) float s_hi[C], s_lo[C], s_rk[C];
  __shared__ float s_beta[C], s_rq[C];
  bf16* const s_k = reinterpret_cast<bf16*>(lds);
  float* const s_l = reinterpret_cast<float*>(lds);

  const auto [b, c, h, g] = chunk_head(a);
  const int64_t at = chunk_at(a, b * a.H + h, c);
  const int64_t t0 = c * C, row0 = b * a.T + t0, left = a.T - t0;
  const int tid = threadIdx.x, lane = tid & 63, w = wave_of(tid), j = lane & 15, q = lane >> 4;
  const int own = 16 * w + j;   // the lane's token

  Frag<PI> kf[KS], qf[KS];
  {
    const int64_t row = row0 + (own < left ? own : left - 1), at = g * a.N + 8 * q;
    KeyRow<IO, KP, FULL> kr, qr;
    kr.load(static_cast<const IO*>(a.k) + row * a.k_stride + at, a.N, q);
    qr.load(static_cast<const IO*>(a.q) + row * a.q_stride + at, a.N, q);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      kf[s] = kr.frag(s, a.N, q);
      qf[s] = qr.frag(s, a.N, q);
    }
  }

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
#pragma unroll
  for (int s = 0; s < KS; ++s)
#pragma unroll
    for (int i = 0; i < PI; ++i)
      *reinterpret_cast<bf16x8*>(&s_k[i * C * KST + own * KST + 32 * s + 8 * q]) = kf[s].p[i];
  __syncthreads();

  // The rows against key tokens up to them, transposed: lane (keys 16 jt + 4 q
  // .. + 3, own token).  The diagonal of K K^T and one tile of Q Q^T are the
  // squares of the lengths.
  f32x4 p[4], l[4];
#pragma unroll
  for (int jt = 0; jt < 4; ++jt) {
    p[jt] = l[jt] = f32x4{0, 0, 0, 0};
    if (jt > w) continue;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const auto ka = load_planes<PI>(&s_k[(16 * jt + j) * KST + 32 * s + 8 * q], C * KST);
      l[jt] = mma(ka, kf[s], l[jt]);
      p[jt] = mma(ka, qf[s], p[jt]);
    }
    if (jt == w) {
      f32x4 qq = {0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < KS; ++s) qq = mma(qf[s], qf[s], qq);
      if (q == j >> 2) {
        const int r = j & 3;
        const float k2 = r == 0 ? l[jt][0] : r == 1 ? l[jt][1] : r == 2 ? l[jt][2] : l[jt][3];
        const float q2 = r == 0 ? qq[0] : r == 1 ? qq[1] : r == 2 ? qq[2] : qq[3];
        const bool in = own < left;
        s_rk[own] = !in ? 0.0f : a.unit ? 1.0f / sqrtf(k2 + a.norm_eps) : 1.0f;
        s_rq[own] = !in ? 0.0f : a.scale * (a.unit ? 1.0f / sqrtf(q2 + a.norm_eps) : 1.0f);
      }
    }
  }
  __syncthreads();
  {
    const float hi_own = s_hi[own], lo_own = s_lo[own], l_own = s_beta[own] * s_rk[own], p_own = s_rq[own];
    by_wave(w, [&](auto W) {
#pragma unroll
    for (int jt = 0; jt <= W; ++jt) {
      const int key0 = 16 * jt + 4 * q;
      const f32x4 hi = *reinterpret_cast<const f32x4*>(&s_hi[key0]), lo = *reinterpret_cast<const f32x4*>(&s_lo[key0]);
      const f32x4 rk = *reinterpret_cast<const f32x4*>(&s_rk[key0]);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float dec = exp2_of((hi_own - hi[r]) + (lo_own - lo[r])) * rk[r];
        l[jt][r] *= l_own * dec;
        p[jt][r] *= p_own * dec;
        if (jt == W) {
          l[jt][r] = own > key0 + r ? l[jt][r] : 0.0f;
          p[jt][r] = own >= key0 + r ? p[jt][r] : 0.0f;
        }
      }
    }
    });
  }
  if constexpr (!GRADS) {
#pragma unroll
    for (int s = 0; s < 2; ++s)
      if (s <= (w >> 1)) store_frag(a.qk, at, lower_frag(w, s), lane, right_of<PY>(p[2 * s], p[2 * s + 1]));
  }

  __syncthreads();
#pragma unroll
  for (int jt = 0; jt < 4; ++jt)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (jt <= w) s_l[(16 * jt + 4 * q + r) * kPairStride + own] = l[jt][r];

  f32x4 x[4];   // block (w, w - d) of the inverse, transposed
  {
    // only this wavefront wrote the block
    __builtin_amdgcn_wave_barrier();
    // halves of 8 by substitution, lane j solving for its half's column of the
    // transposed inverse; then D - D U D for the block U between them
    const int half = j & 8;
    float col[8];
#pragma unroll
    for (int m = 7; m >= 0; --m) {
      const float* l = &s_l[(16 * w + half + m) * kPairStride + 16 * w + half];   // column m of L
      float acc = m == (j & 7) ? 1.0f : 0.0f;
#pragma unroll
      for (int i = 7; i > m; --i) acc = fmaf(-l[i], col[i], acc);
      col[m] = acc;
    }
    const bool same = (q >> 1) == (j >> 3);
    const f32x4 zero = {0, 0, 0, 0};
    f32x4 u = *reinterpret_cast<const f32x4*>(&s_l[(16 * w + j) * kPairStride + 16 * w + 4 * q]);
    if (j >= 8 || q < 2) u = zero;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      x[0][r] = !same ? 0.0f : q & 1 ? col[4 + r] : col[r];
      s_d[(16 * w + 4 * q + r) * kDiag + j] = x[0][r];
    }
    __builtin_amdgcn_wave_barrier();
    const f32x4 d = *reinterpret_cast<const f32x4*>(&s_d[(16 * w + j) * kDiag + 4 * q]);
    x[0] -= mma16(d, mma16(u, x[0], zero), zero);
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int r = 0; r < 4; ++r) s_d[(16 * w + 4 * q + r) * kDiag + j] = x[0][r];
  }
  __syncthreads();
  f32x4 row[4];   // by column tile: x[w - t], zeros right of the diagonal
  by_wave(w, [&](auto W) {
#pragma unroll
    for (int d = 1; d <= W; ++d) {
      const int jb = W - d;
      f32x4 acc = {0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < d; ++e)
        acc = mma16(*reinterpret_cast<const f32x4*>(&s_l[(16 * jb + j) * kPairStride + 16 * (W - e) + 4 * q]), x[e], acc);
      x[d] = -mma16(*reinterpret_cast<const f32x4*>(&s_d[(16 * jb + j) * kDiag + 4 * q]), acc, f32x4{0, 0, 0, 0});
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) row[t] = t <= W ? x[t <= W ? W - t : 0] : f32x4{0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s <= W / 2; ++s) store_frag(a.inv, at, lower_frag(W, s), lane, right_of<3>(row[2 * s], row[2 * s + 1]));
  });

  if constexpr (GRADS) {
    // both again, as rows in LDS and read by columns: row tiles 0 and 1 of the
    // transposed reach over all of them, 2 and 3 over the last 32
    float* const s_p = s_l + C * kPairStride;
    __syncthreads();
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      *reinterpret_cast<f32x4*>(&s_l[own * kPairStride + 16 * t + 4 * q]) = row[t];
      *reinterpret_cast<f32x4*>(&s_p[own * kPairStride + 16 * t + 4 * q]) = p[t];
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (s < (w >> 1)) continue;
      f32x4 vx[2], vp[2];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int o = (32 * s + 16 * t + 4 * q + r) * kPairStride + own;
          vx[t][r] = s_l[o];
          vp[t][r] = s_p[o];
        }
      store_frag(a.inv_t, at, upper_frag(w, s), lane, right_of<3>(vx[0], vx[1]));
      store_frag(a.qk, at, upper_frag(w, s), lane, right_of<3>(vp[0], vp[1]));
    }
  }

  // what multiplies a token's rows: v, K S^T, its write on the way to the end,
  // Q S^T
  if (tid < C) {
    const float gamma = exp2_of(s_hi[tid] + s_lo[tid]), beta = s_beta[tid];
    const float end = exp2_of((s_hi[C - 1] - s_hi[tid]) + (s_lo[C - 1] - s_lo[tid]));
    float* gate = a.gate + at * kGates + tid;
    gate[kBeta] = beta;
    gate[kRight] = beta * gamma * s_rk[tid];
    gate[kEnd] = end * s_rk[tid];
    gate[kOut] = gamma * s_rq[tid];
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
//
// A chunk's operands are requested as soon as the registers of the last one's
// are free: k, q, v behind the first products, the inverse behind the second,
// q k^T behind the third.  Every load and store of a step is issued on every
// path (past the last chunk its own operands again; y of tokens past the end to
// `park`; the workspace holds whole tiles), so that a wait covers what it is for
// and no later request.
template <typename IO, int KP, bool FULL, int NT, bool KEEP>
__global__ __launch_bounds__(kThreads) void k_delta_chain(DeltaArgs a) {
  constexpr int PI = Planes<IO>::in, PY = Planes<IO>::y;
  constexpr int KS = KP / 32, KST = KP + 8, KTR = KP + 16, KT = KP / 64, W = 16 * NT;
  __shared__ __align__(16) bf16 s_k[2 * PI * C * KTR];
  __shared__ __align__(16) bf16 s_s[3 * W * KST];
  __shared__ __align__(16) bf16 s_r[3 * W * kTokStride];   // right sides
  __shared__ __align__(16) bf16 s_e[3 * W * kTokStride];   // writes, decayed to the chunk's end
  __shared__ __align__(16) bf16 s_w[KEEP ? 8 : PY * W * kTokStride];  // writes

  const int slices = (a.P + W - 1) / W;
  const int64_t id = xcd_remap(blockIdx.x, gridDim.x);
  const int64_t bh = id / slices, b = bh / a.H, h = bh % a.H, g = h / (a.H / a.G);
  const int col0 = (int)(id % slices) * W;
  const int tid = threadIdx.x, lane = tid & 63, w = wave_of(tid), j = lane & 15, q = lane >> 4;
  bool col_in[NT];
  int col[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    col_in[n] = col0 + 16 * n + j < a.P;
    col[n] = col_in[n] ? col0 + 16 * n + j : 0;
  }

  // state tiles (keys 16 (KT w + t) + 4 q .. + 3, value column j of tile n)
  f32x4 st[NT][KT];
  const int key0 = 16 * KT * w + 4 * q;
  bf16* const put_s = &s_s[j * KST + key0];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      st[n][t] = f32x4{0, 0, 0, 0};
      if (a.h0 && col_in[n] && key0 + 16 * t < a.N)
        st[n][t] = *reinterpret_cast<const f32x4*>(a.h0 + (bh * a.P + col[n]) * a.N + key0 + 16 * t);
      store_split4<3>(put_s + 16 * n * KST + 16 * t, W * KST, st[n][t]);
    }

  // where the lane's rows are: row 16 w + j of k and q, rows 16 w + 4 q + r of v
  const IO *kp, *qp, *vp[4];
  auto rows_of = [&](int64_t c) {
    const int64_t row0 = b * a.T + c * C, left = a.T - c * C;
    const int64_t row = row0 + (16 * w + j < left ? 16 * w + j : left - 1), at = g * a.N + 8 * q;
    kp = static_cast<const IO*>(a.k) + row * a.k_stride + at;
    qp = static_cast<const IO*>(a.q) + row * a.q_stride + at;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int tok = 16 * w + 4 * q + r;
      vp[r] = static_cast<const IO*>(a.v) + (row0 + (tok < left ? tok : left - 1)) * a.v_stride + h * a.P;
    }
  };
  const int64_t at0 = chunk_at(a, bh, 0);
  const float* gp = a.gate + at0 * kGates + 16 * w + 4 * q;
  // the second fragment of wavefronts 0 and 1 is their first one again, unused
  const int second = w >= 2 ? 1 : 0;
  const bf16* xp = a.inv + (at0 * kTriFrags + lower_frag(w, 0)) * (3 * kFrag) + lane * 8;
  const bf16* pp = a.qk + (at0 * kTriFrags + lower_frag(w, 0)) * (PY * kFrag) + lane * 8;
  const float* ep = a.whole + at0;
  const int64_t y_row = a.H * a.P;
  IO* yp = KEEP ? nullptr : static_cast<IO*>(a.y) + (b * a.T + 16 * w + 4 * q) * y_row + h * a.P;
  IO* const park = static_cast<IO*>(a.park) + lane;
  const int64_t cols = padded_cols(a.P);
  float* state_at = KEEP ? a.enter + (at0 * cols + col0 + j) * KP + key0 : nullptr;
  float* write_at = KEEP ? a.write + (at0 * cols + col0 + j) * C + 16 * w + 4 * q : nullptr;

  KeyRow<IO, KP, FULL> kr, qr;
  Frag<3> xf[2];
  Frag<PY> pf[2];
  f32x4 g_beta, g_right, g_end, g_out;
  IO v[NT][4];
  float whole = *ep;
  auto load_rows = [&]() {
    kr.load(kp, a.N, q);
    if constexpr (!KEEP) qr.load(qp, a.N, q);
    g_beta = *reinterpret_cast<const f32x4*>(gp + kBeta);
    g_right = *reinterpret_cast<const f32x4*>(gp + kRight);
    g_end = *reinterpret_cast<const f32x4*>(gp + kEnd);
    if constexpr (!KEEP) g_out = *reinterpret_cast<const f32x4*>(gp + kOut);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int n = 0; n < NT; ++n) v[n][r] = vp[r][col[n]];
  };
  auto load_x = [&]() {
    xf[0] = load_planes<3>(xp, kFrag);
    xf[1] = load_planes<3>(xp + second * (3 * kFrag), kFrag);
  };
  auto load_p = [&]() {
    pf[0] = load_planes<PY>(pp, kFrag);
    pf[1] = load_planes<PY>(pp + second * (PY * kFrag), kFrag);
  };
  bf16* const put_k = &s_k[(16 * w + j) * KTR + 8 * q];
  int k_at = 0;   // which half of s_k holds the chunk
  auto store_k = [&](int at) {
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const auto f = kr.frag(s, a.N, q);
#pragma unroll
      for (int i = 0; i < PI; ++i) *reinterpret_cast<bf16x8*>(put_k + at + i * C * KTR + 32 * s) = f.p[i];
    }
  };
  rows_of(0);
  load_rows();
  load_x();
  if constexpr (!KEEP) load_p();
  store_k(0);
  __syncthreads();

  const bf16* const get_s = &s_s[j * KST + 8 * q];
  const int put_t = j * kTokStride + token_slot(w, q), get_t = j * kTokStride + 8 * q;
  const bf16* const get_k = &s_k[(4 * q + (j >> 2)) * KTR + 16 * KT * w + 4 * (j & 3)];
  for (int64_t c = 0; c < a.Nc; ++c) {
    const int64_t left = a.T - c * C;
    const int64_t next = c + 1 < a.Nc ? 1 : 0;
    if constexpr (KEEP) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int t = 0; t < KT; ++t)
          *reinterpret_cast<f32x4*>(state_at + 16 * n * KP + 16 * t) = st[n][t];
      state_at += cols * KP;
    }
    // K S^T and Q S^T of the wavefront's tokens; the right sides b (v - gamma K S^T)
    f32x4 y[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      f32x4 ks = {0, 0, 0, 0}, qs = {0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const auto sf = load_planes<3>(get_s + 16 * n * KST + 32 * s, W * KST);
        ks = mma(kr.frag(s, a.N, q), sf, ks);
        if constexpr (!KEEP) {
          Frag<PY> sy;
#pragma unroll
          for (int i = 0; i < PY; ++i) sy.p[i] = sf.p[i];
          qs = mma(qr.frag(s, a.N, q), sy, qs);
        }
      }
      f32x4 rs;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        rs[r] = fmaf(-g_right[r], ks[r], g_beta[r] * to_f32(v[n][r]));
        if constexpr (!KEEP) y[n][r] = g_out[r] * qs[r];
      }
      store_split4<3>(s_r + put_t + 16 * n * kTokStride, W * kTokStride, rs);
    }
    const f32x4 eta = g_end;
    if (next && left < 2 * C) {
      rows_of(c + 1);
    } else {
      kp += next * a.k_stride * C;
      qp += next * a.q_stride * C;
#pragma unroll
      for (int r = 0; r < 4; ++r) vp[r] += next * a.v_stride * C;
    }
    gp += next * kGates;
    load_rows();
    __syncthreads();
    // the writes
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      f32x4 ws = mma(xf[0], load_planes<3>(s_r + get_t + 16 * n * kTokStride, W * kTokStride), f32x4{0, 0, 0, 0});
      if (w >= 2) ws = mma(xf[1], load_planes<3>(s_r + get_t + 16 * n * kTokStride + 32, W * kTokStride), ws);
      f32x4 es;
#pragma unroll
      for (int r = 0; r < 4; ++r) es[r] = eta[r] * ws[r];
      store_split4<3>(s_e + put_t + 16 * n * kTokStride, W * kTokStride, es);
      if constexpr (!KEEP) store_split4<PY>(s_w + put_t + 16 * n * kTokStride, W * kTokStride, ws);
      else *reinterpret_cast<f32x4*>(write_at + 16 * n * C) = ws;
    }
    if constexpr (KEEP) write_at += cols * C;
    xp += next * (kTriFrags * 3 * kFrag);
    load_x();
    __syncthreads();
    // the state at the chunk's end
    const float decay = whole;
    ep += next;
    whole = *ep;
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      Frag<PI> ka[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) ka[s] = read_tr<PI>(get_k + k_at + 32 * s * KTR + 16 * t, C * KTR, 16 * KTR);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        f32x4 acc = {0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < 2; ++s)
          acc = mma(ka[s], load_planes<3>(s_e + get_t + 16 * n * kTokStride + 32 * s, W * kTokStride), acc);
#pragma unroll
        for (int r = 0; r < 4; ++r) st[n][t][r] = fmaf(decay, st[n][t][r], acc[r]);
        store_split4<3>(put_s + 16 * n * KST + 16 * t, W * KST, st[n][t]);
      }
    }
    k_at = PI * C * KTR - k_at;
    store_k(k_at);
    // outputs
    if constexpr (!KEEP) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        y[n] = mma(pf[0], load_planes<PY>(s_w + get_t + 16 * n * kTokStride, W * kTokStride), y[n]);
        if (w >= 2) y[n] = mma(pf[1], load_planes<PY>(s_w + get_t + 16 * n * kTokStride + 32, W * kTokStride), y[n]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          IO* const to = 16 * w + 4 * q + r < left && col_in[n] ? yp + r * y_row + col[n] : park;
          *to = to_io<IO>(y[n][r]);
        }
      }
      yp += C * y_row;
      pp += next * (kTriFrags * PY * kFrag);
      load_p();
    }
    __syncthreads();
  }
  if (!KEEP && a.state) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int t = 0; t < KT; ++t)
        if (col_in[n] && key0 + 16 * t < a.N)
          *reinterpret_cast<f32x4*>(a.state + (bh * a.P + col[n]) * a.N + key0 + 16 * t) = st[n][t];
  }
}

// ---------------------------------------------------------------------------
// The chunks of one (b, h) in order, bfloat16 io: every wavefront owns 16 value
// columns alone.  The state, the right sides and the writes stay in its
// registers (ssd_delta.h); what the wavefronts share, k, q and the two
// matrices of a chunk, lands in LDS, half of a compute unit's, so that one
// workgroup computes while another waits for its chunk (8 x 16384 x 64 heads of
// 64 x 128: 1780 us; one
// workgroup a unit that requests a chunk ahead 2270).  A
// chunk takes a wavefront 182 matrix instructions (keys of 128), 2912 cycles.
// ---------------------------------------------------------------------------
template <int KP, int NW, bool KEEP> struct ColumnsLds {
  using Keys = KeyTile<KP, NW>;
  static constexpr int k = 0, q = k + Keys::kElems, x = q + (KEEP ? 0 : Keys::kElems);
  static constexpr int p = x + 3 * kTriFrags * kFrag, v = p + (KEEP ? 0 : 2 * kTriFrags * kFrag);
  static constexpr int gate = v + C * 16 * NW, elems = gate + 2 * kGates;
};

template <int KP, bool FULL, bool KEEP>
__global__ __launch_bounds__(256, 2) void k_delta_columns(DeltaArgs a) {
  constexpr int NW = 4, KS = KP / 32, KT = KP / 16, W = 16 * NW;
  using L = ColumnsLds<KP, NW, KEEP>;
  using Keys = KeyTile<KP, NW>;
  using Cols = ColumnTile<NW>;
  __shared__ __align__(1024) bf16 lds[L::elems];

  const int slices = (a.P + W - 1) / W;
  const int64_t id = xcd_remap(blockIdx.x, gridDim.x);
  const int64_t bh = id / slices, b = bh / a.H, h = bh % a.H, g = h / (a.H / a.G);
  const int col0 = (int)(id % slices) * W;
  const int tid = threadIdx.x, lane = tid & 63, w = wave_of(tid), j = lane & 15, q = lane >> 4;
  const int col = col0 + 16 * w + j;
  const bool col_in = col < a.P;
  const int64_t at0 = chunk_at(a, bh, 0), cols = padded_cols(a.P);

  // columns that no request reaches stay zero
  for (int i = tid; i < L::elems / 8; i += 256) reinterpret_cast<uint4*>(lds)[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  // what the wavefront requests of a chunk: lane offsets, and where it starts
  typename Keys::Offsets k_off, q_off;
  typename Cols::Offsets v_off;
  auto offsets = [&](int64_t c) {
    const int last = (int)min((int64_t)C, a.T - c * C) - 1;
    Keys::offsets(k_off, (int)a.k_stride, last, a.N, w, lane);
    if constexpr (!KEEP) Keys::offsets(q_off, (int)a.q_stride, last, a.N, w, lane);
    Cols::offsets(v_off, (int)a.v_stride, last, a.P - col0, w, lane);
  };
  const uint32_t lds0 = lds_address(lds) + w * 1024;
  const bf16* kp = static_cast<const bf16*>(a.k) + b * a.T * a.k_stride + g * a.N;
  const bf16* qp = static_cast<const bf16*>(a.q) + b * a.T * a.q_stride + g * a.N;
  const bf16* vp = static_cast<const bf16*>(a.v) + b * a.T * a.v_stride + h * a.P + col0;
  const bf16* xp = a.inv + at0 * (3 * kTriFrags * kFrag) + w * 512;
  const bf16* pp = a.qk + at0 * (2 * kTriFrags * kFrag) + w * 512;
  const float* gp = a.gate + at0 * kGates + w * 256;
  const bool all_cols = a.P - col0 >= W;
  auto request = [&]() {
    Keys::template request<FULL>(kp, k_off, lds0 + 2 * L::k);
    if constexpr (!KEEP) Keys::template request<FULL>(qp, q_off, lds0 + 2 * L::q);
    request_linear<3 * kTriFrags, NW>(xp, lds0 + 2 * L::x, w, lane);
    if constexpr (!KEEP) request_linear<2 * kTriFrags, NW>(pp, lds0 + 2 * L::p, w, lane);
    if (all_cols) Cols::template request<true>(vp, v_off, lds0 + 2 * L::v);
    else Cols::template request<false>(vp, v_off, lds0 + 2 * L::v);
    request_linear<1, NW>(gp, lds0 + 2 * L::gate, w, lane);
  };
  offsets(0);
  request();

  // state tiles: keys key_of(t, 4 q + r) of value column j
  f32x4 st[KT];
#pragma unroll
  for (int t = 0; t < KT; ++t) {
    const int key = key_of(t, 4 * q);
    st[t] = f32x4{0, 0, 0, 0};
    if (a.h0 && col_in && key < a.N) st[t] = *reinterpret_cast<const f32x4*>(a.h0 + (bh * a.P + col) * a.N + key);
  }
  const bool idle = col0 + 16 * w >= a.P;   // no column of this wavefront exists
  float* state_at = KEEP ? a.enter + (at0 * cols + col) * KP + 8 * q : nullptr;
  float* write_at = KEEP ? a.write + (at0 * cols + col) * C + 4 * q : nullptr;

  int row_at[KS], col_at[KT / 2];
#pragma unroll
  for (int s = 0; s < KS; ++s) row_at[s] = Keys::row_at(s, j, q);
#pragma unroll
  for (int u = 0; u < KT / 2; ++u) col_at[u] = Keys::col_at(u, j, q);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
  for (int t = 0; t < KT; ++t) pin(st[t]);

  for (int64_t c = 0; c < a.Nc; ++c) {
    landed<0>();
    const float whole = load_uniform(a.whole + at0 + c);
    const float* const gate = reinterpret_cast<const float*>(lds + L::gate) + 4 * q;
    auto gates = [&](int which, int i) { return *reinterpret_cast<const f32x4*>(gate + which + 16 * i); };
    if (KEEP && !idle) {
#pragma unroll
      for (int t = 0; t < KT; ++t) *reinterpret_cast<f32x4*>(state_at + key_of(t, 0)) = st[t];
      state_at += cols * KP;
    }

    // K S^T and Q S^T
    f32x4 ks[4], qs[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) ks[i] = qs[i] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const auto sf = right_of<3>(st[2 * s], st[2 * s + 1]);
      Frag<1> rows[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) rows[i] = load_planes<1>(lds + L::k + row_at[s] + 16 * i * KP, 0);
      mma_tiles(rows, sf, ks);
      if constexpr (!KEEP) {
        const Frag<2> sy = {{sf.p[0], sf.p[1]}};
#pragma unroll
        for (int i = 0; i < 4; ++i) rows[i] = load_planes<1>(lds + L::q + row_at[s] + 16 * i * KP, 0);
        mma_tiles(rows, sy, qs);
      }
    }
    // the right sides, and the writes
    Frag<3> rf[2], ef[2];
    f32x4 ws[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bf16x4 v = lds_read_tr4(lds + L::v + (16 * i + 4 * q + (j >> 2)) * W + 16 * w + 4 * (j & 3));
      const f32x4 gb = gates(kBeta, i), gr = gates(kRight, i);
#pragma unroll
      for (int r = 0; r < 4; ++r) ks[i][r] = fmaf(-gr[r], ks[i][r], gb[r] * (float)v[r]);
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) rf[s] = right_of<3>(ks[2 * s], ks[2 * s + 1]);
#pragma unroll
    for (int i = 0; i < 4; ++i) ws[i] = f32x4{0, 0, 0, 0};
    mma_lower<3>(lds + L::x + lane * 8, rf, ws);
    if (KEEP && !idle) {
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<f32x4*>(write_at + 16 * i) = ws[i];
      write_at += cols * C;
    }
    // the state at the chunk's end
#pragma unroll
    for (int s = 0; s < 2; ++s) ef[s] = right_of<3>(gates(kEnd, 2 * s) * ws[2 * s], gates(kEnd, 2 * s + 1) * ws[2 * s + 1]);
#pragma unroll
    for (int t0 = 0; t0 < KT; t0 += 4) {
      f32x4 acc[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) acc[t] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        Frag<1> keys[4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
          keys[t] = Keys::columns(lds + L::k + col_at[(t0 + t) / 2] + 4 * (t & 1) + 32 * s * KP);
        mma_tiles(keys, ef[s], acc);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) st[t0 + t][r] = fmaf(whole, st[t0 + t][r], acc[t][r]);
    }
    // outputs, through the wavefront's own columns of v
    if constexpr (!KEEP) {
      Frag<2> wf[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) wf[s] = right_of<2>(ws[2 * s], ws[2 * s + 1]);
      bf16* const out = lds + L::v + 16 * w;
#pragma unroll
      for (int i = 0; i < 4; ++i) qs[i] *= gates(kOut, i);
      mma_lower<2>(lds + L::p + lane * 8, wf, qs);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) out[(16 * i + 4 * q + r) * W + j] = (bf16)qs[i][r];
      const int64_t left = a.T - c * C;
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int row = 32 * n + (lane >> 1), part = 8 * (lane & 1);
        const uint4 v = *reinterpret_cast<const uint4*>(out + row * W + part);
        const bool in = row < left && col0 + 16 * w + part < a.P;
        bf16* const to = static_cast<bf16*>(a.y) + (b * a.T + c * C + row) * (a.H * a.P) + h * a.P + col0 + 16 * w + part;
        *reinterpret_cast<uint4*>(in ? to : static_cast<bf16*>(a.park) + lane * 8) = v;
      }
    }
    lds_free();
    if (c + 1 < a.Nc) {
      kp += C * a.k_stride;
      qp += C * a.q_stride;
      vp += C * a.v_stride;
      xp += 3 * kTriFrags * kFrag;
      pp += 2 * kTriFrags * kFrag;
      gp += kGates;
      if (c + 2 == a.Nc) offsets(c + 1);
      request();
    }
  }
  if (!KEEP && a.state && col_in) {
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const int key = key_of(t, 4 * q);
      if (key < a.N) *reinterpret_cast<f32x4*>(a.state + (bh * a.P + col) * a.N + key) = st[t];
    }
  }
}

// ---------------------------------------------------------------------------
// The chunks of one (b, h) in order, bfloat16 io: four wavefronts share 16 value
// columns (NG such groups to a workgroup), wavefront w the rows of tokens 16 w
// .. + 15 and a quarter of the state's keys.  The state, the right sides and the
// writes go through LDS as in k_delta_chain; what comes from memory lands in LDS
// as in k_delta_columns, each operand requested when its last reader is done:
//   top        q k^T of this chunk; k, gates of the next (two places for each)
//   barrier 1  q, v of the next            (waits for the inverse)
//   barrier 2  the next inverse            (waits for q k^T)
//   barrier 3                              (waits for k, gates, q, v)
// Every wavefront makes the same requests, so that the counts that the waits
// leave outstanding are constants.
// ---------------------------------------------------------------------------
template <int KP, int NG, bool KEEP> struct TokensLds {
  using Keys = KeyTile<KP, 4 * NG>;
  static constexpr int W = 16 * NG;
  static constexpr int k = 0, q = k + 2 * Keys::kElems, x = q + (KEEP ? 0 : Keys::kElems);
  static constexpr int p = x + 3 * kTriFrags * kFrag, v = p + (KEEP ? 0 : 2 * kTriFrags * kFrag);
  static constexpr int gate = v + C * W, s = gate + 4 * kGates, r = s + 3 * W * KP;
  static constexpr int e = r + 3 * W * C, wr = e + 3 * W * C;
  static constexpr int y = wr + (KEEP ? 0 : 2 * W * C), elems = y + (KEEP ? 0 : C * W);
};

template <int KP, bool FULL, int NG, bool KEEP>
__global__ __launch_bounds__(256 * NG) void k_delta_tokens(DeltaArgs a) {
  using L = TokensLds<KP, NG, KEEP>;
  using Keys = typename L::Keys;
  constexpr int KS = KP / 32, KT = KP / 64, W = L::W, NW = 4 * NG;
  constexpr int kKeyLoads = Keys::kLoads, kXLoads = (3 * kTriFrags + NW - 1) / NW, kPLoads = (2 * kTriFrags + NW - 1) / NW;
  __shared__ __align__(1024) bf16 lds[L::elems];

  const int slices = (a.P + W - 1) / W;
  const int64_t id = xcd_remap(blockIdx.x, gridDim.x);
  const int64_t bh = id / slices, b = bh / a.H, h = bh % a.H, g = h / (a.H / a.G);
  const int col0 = (int)(id % slices) * W;
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_of(tid), j = lane & 15, q = lane >> 4;
  const int w = wave & 3, n = wave >> 2;   // row tile, column group
  const int row = 16 * n + j;              // the lane's value column among the workgroup's
  const int64_t at0 = chunk_at(a, bh, 0), cols = padded_cols(a.P);

  // columns that no request reaches stay zero
  for (int i = tid; i < L::elems / 8; i += 64 * NW) reinterpret_cast<uint4*>(lds)[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  typename Keys::Offsets k_off, q_off;
  uint32_t v_off;
  constexpr int v_vecs = 2 * NG, v_rows = 64 / v_vecs, v_kb = C / v_rows;   // 16-byte vectors of a row, KB in all
  const int v_t = wave % v_kb;
  const bool v_in = col0 + 8 * (lane % v_vecs) < a.P;
  auto offsets = [&](int64_t c) {
    const int last = (int)min((int64_t)C, a.T - c * C) - 1;
    Keys::offsets(k_off, (int)a.k_stride, last, a.N, wave, lane);
    if constexpr (!KEEP) Keys::offsets(q_off, (int)a.q_stride, last, a.N, wave, lane);
    v_off = (uint32_t)min(v_t * v_rows + lane / v_vecs, last) * (uint32_t)a.v_stride * 2u + 16u * (lane % v_vecs);
  };
  const uint32_t lds0 = lds_address(lds), mine = lds0 + wave * 1024;
  const bf16* kp = static_cast<const bf16*>(a.k) + b * a.T * a.k_stride + g * a.N;
  const bf16* qp = static_cast<const bf16*>(a.q) + b * a.T * a.q_stride + g * a.N;
  const bf16* vp = static_cast<const bf16*>(a.v) + b * a.T * a.v_stride + h * a.P + col0;
  const bf16* xp = a.inv + at0 * (3 * kTriFrags * kFrag) + wave * 512;
  const bf16* pp = a.qk + at0 * (2 * kTriFrags * kFrag) + wave * 512;
  const float* gp = a.gate + at0 * kGates;
  const bool all_cols = a.P - col0 >= W;
  auto request_k = [&](int half) {
    Keys::template request<FULL>(kp, k_off, mine + 2 * (L::k + half * Keys::kElems));
    request16(gp, 16 * lane, lds0 + 2 * (L::gate + half * 2 * kGates));
  };
  auto request_qv = [&]() {
    if constexpr (!KEEP) Keys::template request<FULL>(qp, q_off, mine + 2 * L::q);
    if (all_cols || v_in) request16(vp, v_off, lds0 + 2 * L::v + v_t * 1024);
  };
  auto request_x = [&]() { request_evenly<3 * kTriFrags, NW>(xp, mine + 2 * L::x, wave, lane); };
  offsets(0);
  request_k(0);
  request_qv();
  request_x();

  // state tiles: keys key_of(KT w + t, 4 q + r) of the lane's value column
  f32x4 st[KT];
  const int col = col0 + row;
  const bool col_in = col < a.P;
  int key[KT], put_s[KT];
#pragma unroll
  for (int t = 0; t < KT; ++t) {
    key[t] = key_of(KT * w + t, 4 * q);
    put_s[t] = L::s + row_vec<KP>(row, key[t] / 8) + key[t] % 8;
    st[t] = f32x4{0, 0, 0, 0};
    if (a.h0 && col_in && key[t] < a.N) st[t] = *reinterpret_cast<const f32x4*>(a.h0 + (bh * a.P + col) * a.N + key[t]);
  }
  auto store_s = [&]() {
#pragma unroll
    for (int t = 0; t < KT; ++t) store_split4<3>(lds + put_s[t], W * KP, st[t]);
  };
  store_s();
  // the workspace has whole tiles of columns; the last groups may lie past them
  const bool kept = KEEP && col0 + 16 * n < cols;
  float* const park = static_cast<float*>(a.park) + 4 * lane;
  float* state_at = kept ? a.enter + (at0 * cols + col) * KP : park;
  float* write_at = kept ? a.write + (at0 * cols + col) * C + 16 * w + 4 * q : park;

  const int put_t = row_vec<C>(row, 4 * (w >> 1) + q) + 4 * (w & 1);   // token_slot(w, q)
  int get_s[KS], get_t[2], row_at[KS], col_at[KT];
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    get_s[s] = L::s + row_vec<KP>(row, 4 * s + q);
    row_at[s] = Keys::row_at(s, j, q) + 16 * w * KP;
  }
#pragma unroll
  for (int s = 0; s < 2; ++s) get_t[s] = row_vec<C>(row, 4 * s + q);
#pragma unroll
  for (int t = 0; t < KT; ++t) col_at[t] = Keys::col_at((KT * w + t) >> 1, j, q) + 4 * ((KT * w + t) & 1);
  const int own_v = (16 * w + 4 * q + (j >> 2)) * W + 16 * n + 4 * (j & 3);
  landed<0>();
#pragma unroll
  for (int t = 0; t < KT; ++t) pin(st[t]);

  for (int64_t c = 0; c < a.Nc; ++c) {
    const int half = (int)c & 1;
    const int64_t left = a.T - c * C;
    const bf16* const lk = lds + L::k + half * Keys::kElems;
    const float* const gate = reinterpret_cast<const float*>(lds + L::gate + half * 2 * kGates) + 16 * w + 4 * q;
    auto gates = [&](int which) { return *reinterpret_cast<const f32x4*>(gate + which); };
    const float whole = load_uniform(a.whole + at0 + c);
    if constexpr (KEEP) {
#pragma unroll
      for (int t = 0; t < KT; ++t) *reinterpret_cast<f32x4*>(kept ? state_at + key[t] : park) = st[t];
      state_at += cols * KP;
    } else {
      request_evenly<2 * kTriFrags, NW>(pp, mine + 2 * L::p, wave, lane);
      pp += 2 * kTriFrags * kFrag;
    }
    // past the last chunk that one again, to where no one reads any more
    if (c + 1 < a.Nc) {
      kp += C * a.k_stride;
      qp += C * a.q_stride;
      vp += C * a.v_stride;
      xp += 3 * kTriFrags * kFrag;
      gp += kGates;
      if (c + 2 == a.Nc) offsets(c + 1);
    }
    request_k(half ^ 1);

    // K S^T and Q S^T of the wavefront's tokens, in two sums each; the right sides
    f32x4 y;
    {
      f32x4 ks[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}}, qs[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
      for (int s = 0; s < KS; s += 2) {
        bf16x8 kf[2], qf[2];
        Frag<3> sf[2];
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          kf[o] = ld8(lk + row_at[s + o]);
          if constexpr (!KEEP) qf[o] = ld8(lds + L::q + row_at[s + o]);
          sf[o] = load_planes<3>(lds + get_s[s + o], W * KP);
        }
#pragma unroll
        for (int i = 2; i >= 0; --i) {
#pragma unroll
          for (int o = 0; o < 2; ++o) ks[o] = mma(kf[o], sf[o].p[i], ks[o]);
          if constexpr (!KEEP)
            if (i < 2)
#pragma unroll
              for (int o = 0; o < 2; ++o) qs[o] = mma(qf[o], sf[o].p[i], qs[o]);
        }
      }
      const f32x4 gb = gates(kBeta), gr = gates(kRight);
      const bf16x4 v = lds_read_tr4(lds + L::v + own_v);
      f32x4 rs;
#pragma unroll
      for (int r = 0; r < 4; ++r) rs[r] = fmaf(-gr[r], ks[0][r] + ks[1][r], gb[r] * (float)v[r]);
      store_split4<3>(lds + L::r + put_t, W * C, rs);
      if constexpr (!KEEP) y = gates(kOut) * (qs[0] + qs[1]);
    }
    landed<KEEP ? KT + kKeyLoads + 1 : 1 + kPLoads + kKeyLoads + 1>();
    request_qv();
    // the writes
    {
      const f32x4 ge = gates(kEnd);
      const bf16* const lx = lds + L::x + lower_frag(w, 0) * (3 * kFrag) + lane * 8;
      f32x4 ws = {0, 0, 0, 0}, ws2 = {0, 0, 0, 0};
      ws = mma(load_planes<3>(lx, kFrag), load_planes<3>(lds + L::r + get_t[0], W * C), ws);
      if (w >= 2) ws2 = mma(load_planes<3>(lx + 3 * kFrag, kFrag), load_planes<3>(lds + L::r + get_t[1], W * C), ws2);
      ws += ws2;
      store_split4<3>(lds + L::e + put_t, W * C, ge * ws);
      if constexpr (!KEEP) {
        store_split4<2>(lds + L::wr + put_t, W * C, ws);
      } else {
        *reinterpret_cast<f32x4*>(write_at) = ws;
        if (kept) write_at += cols * C;
      }
    }
    landed<KEEP ? 63 : kKeyLoads + 1 + kKeyLoads + 1>();
    request_x();
    // the state at the chunk's end
    {
      f32x4 acc[2][KT];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const auto ef = load_planes<3>(lds + L::e + get_t[s], W * C);
        Frag<1> ka[KT];
#pragma unroll
        for (int t = 0; t < KT; ++t) {
          ka[t] = Keys::columns(lk + col_at[t] + 32 * s * KP);
          acc[s][t] = f32x4{0, 0, 0, 0};
        }
        mma_tiles(ka, ef, acc[s]);
      }
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) st[t][r] = fmaf(whole, st[t][r], acc[0][t][r] + acc[1][t][r]);
      store_s();
    }
    // outputs
    if constexpr (!KEEP) {
      const bf16* const lp = lds + L::p + lower_frag(w, 0) * (2 * kFrag) + lane * 8;
      f32x4 y2 = {0, 0, 0, 0};
      y = mma(load_planes<2>(lp, kFrag), load_planes<2>(lds + L::wr + get_t[0], W * C), y);
      if (w >= 2) y2 = mma(load_planes<2>(lp + 2 * kFrag, kFrag), load_planes<2>(lds + L::wr + get_t[1], W * C), y2);
      // to rows of the output through LDS; only this wavefront touches these
      bf16* const out = lds + L::y + wave * 256;
#pragma unroll
      for (int r = 0; r < 4; ++r) out[(4 * q + r) * 16 + j] = (bf16)(y[r] + y2[r]);
      __builtin_amdgcn_wave_barrier();
      const int tok = lane >> 1 & 15, part = 8 * (lane & 1);
      const bool in = lane < 32 && 16 * w + tok < left && col0 + 16 * n + part < a.P;
      const uint4 val = *reinterpret_cast<const uint4*>(out + tok * 16 + part);
      bf16* const to = static_cast<bf16*>(a.y) + (b * a.T + c * C + 16 * w + tok) * (a.H * a.P) + h * a.P + col0 + 16 * n + part;
      *reinterpret_cast<uint4*>(in ? to : reinterpret_cast<bf16*>(park)) = val;
    }
    landed<KEEP ? 1 + kXLoads : kXLoads + 1>();
  }
  if (!KEEP && a.state && col_in) {
#pragma unroll
    for (int t = 0; t < KT; ++t)
      if (key[t] < a.N) *reinterpret_cast<f32x4*>(a.state + (bh * a.P + col) * a.N + key[t]) = st[t];
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // no request may reach LDS after this
}

// ---------------------------------------------------------------------------
// One token.  A row p of the state needs two dot products, S k and S q; the
// token's own part of y is its write times k.q.
//   y = a S.q + u k.q,  S' = a S + u k,  u = b (v - a S.k)
// NL lanes of four keys share a row; N / 4 of them have keys.
// ---------------------------------------------------------------------------
template <int CTRL> __device__ __forceinline__ float dpp_add(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
// sum over aligned groups of NL lanes, 16 or 32: within 16 by lanes' neighbours
// (quads, halves of 8, of 16) without a trip through LDS
template <int NL> __device__ __forceinline__ float lanes_sum(float v) {
  v = dpp_add<0xb1>(v);    // lane ^ 1
  v = dpp_add<0x4e>(v);    // lane ^ 2
  v = dpp_add<0x141>(v);   // mirrored within 8
  v = dpp_add<0x140>(v);   // mirrored within 16
  return NL == 16 ? v : v + __shfl_xor(v, 16, 64);
}

template <typename IO, int NL, int ROWS>
__global__ __launch_bounds__(kThreads) void k_delta_step(DeltaArgs a) {
  constexpr int per_pass = kThreads / NL;
  const uint32_t runs = (uint32_t)(a.P + per_pass * ROWS - 1) / (per_pass * ROWS), H = (uint32_t)a.H;
  const uint32_t slice = blockIdx.x / runs;
  const int64_t bh = slice, b = slice / H, h = slice % H, g = (uint32_t)h / (H / (uint32_t)a.G);
  const int p0 = (int)(blockIdx.x % runs) * per_pass * ROWS + threadIdx.x / NL;
  const int key = 4 * (threadIdx.x % NL);
  const bool key_in = key < a.N;
  float4* state = reinterpret_cast<float4*>(a.state + bh * a.P * a.N) + (key_in ? key / 4 : 0);
  // all loads on every path, the token's before the state's: a wait for a row of
  // the state then covers that row and no store
  IO kraw[4], qraw[4], vraw[ROWS];
  const IO* kr = static_cast<const IO*>(a.k) + b * a.k_stride + g * a.N + (key_in ? key : 0);
  const IO* qr = static_cast<const IO*>(a.q) + b * a.q_stride + g * a.N + (key_in ? key : 0);
  const IO* vr = static_cast<const IO*>(a.v) + b * a.v_stride + h * a.P;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    kraw[e] = kr[e];
    qraw[e] = qr[e];
  }
#pragma unroll
  for (int i = 0; i < ROWS; ++i) vraw[i] = vr[min(p0 + i * per_pass, a.P - 1)];
  f32x4 s[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i)
    s[i] = __builtin_nontemporal_load(
        reinterpret_cast<const f32x4*>(state + (int64_t)min(p0 + i * per_pass, a.P - 1) * (a.N / 4)));
  __builtin_amdgcn_sched_barrier(0);
  float kv[4], qv[4], kk = 0.0f, qq = 0.0f, kq = 0.0f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    kv[e] = key_in ? to_f32(kraw[e]) : 0.0f;
    qv[e] = key_in ? to_f32(qraw[e]) : 0.0f;
    kk = fmaf(kv[e], kv[e], kk);
    qq = fmaf(qv[e], qv[e], qq);
    kq = fmaf(kv[e], qv[e], kq);
  }
  kk = lanes_sum<NL>(kk);
  qq = lanes_sum<NL>(qq);
  kq = lanes_sum<NL>(kq);
  const float rk = a.unit ? 1.0f / sqrtf(kk + a.norm_eps) : 1.0f;
  const float rq = a.scale * (a.unit ? 1.0f / sqrtf(qq + a.norm_eps) : 1.0f);
  const float bias = a.dt_bias ? a.dt_bias[h] : 0.0f;
  const float d = delta_of(a.dt[bh] + bias, a.softplus, a.dt_min, a.dt_max);
  const float alpha = expf(d * a.A[h]);
  const float beta = a.sigmoid ? sigmoid_of(a.beta[bh]) : a.beta[bh];
  IO* yr = static_cast<IO*>(a.y) + bh * a.P;
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int p = p0 + i * per_pass;
    float sk = s[i][0] * kv[0] + s[i][1] * kv[1] + s[i][2] * kv[2] + s[i][3] * kv[3];
    float sq = s[i][0] * qv[0] + s[i][1] * qv[1] + s[i][2] * qv[2] + s[i][3] * qv[3];
    sk = lanes_sum<NL>(key_in ? sk : 0.0f);
    sq = lanes_sum<NL>(key_in ? sq : 0.0f);
    if (p < a.P) {
      const float u = beta * (to_f32(vraw[i]) - alpha * rk * sk), uk = u * rk;
      if (key_in) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[i][e] = fmaf(alpha, s[i][e], uk * kv[e]);
        __builtin_nontemporal_store(s[i], reinterpret_cast<f32x4*>(state + (int64_t)p * (a.N / 4)));
      }
      if (threadIdx.x % NL == 0) yr[p] = to_io<IO>(rq * (alpha * sq + uk * kq));
    }
  }
}

// GRADS: the forward part of the gradients, which keeps states and writes
template <bool GRADS>
hipError_t launch_scan(const DeltaArgs& a, bool io_bf16, hipStream_t stream) {
  return with_keys(a.N, io_bf16, [&](auto io, auto kp, auto full) {
    using IO = decltype(io);
    constexpr int KP = decltype(kp)::value;
    constexpr bool FULL = decltype(full)::value;
    const unsigned chunks = (unsigned)(a.Bt * a.H * a.Nc);
    const int64_t heads = a.Bt * a.H;
    hipLaunchKernelGGL((k_delta_prep<IO, KP, FULL, GRADS>), dim3(chunks), dim3(kThreads), 0, stream, a);
    if constexpr (sizeof(IO) == 2) {
      return chain_of(
          a,
          [&](auto ng, unsigned groups) {
            hipLaunchKernelGGL((k_delta_tokens<KP, FULL, ng.value, GRADS>), dim3(groups), dim3(256 * ng.value), 0,
                               stream, a);
          },
          [&](unsigned groups) {
            hipLaunchKernelGGL((k_delta_columns<KP, FULL, GRADS>), dim3(groups), dim3(256), 0, stream, a);
          });
    } else {
      hipLaunchKernelGGL((k_delta_chain<IO, KP, FULL, 1, GRADS>), dim3((unsigned)(heads * ((a.P + 15) / 16))),
                         dim3(kThreads), 0, stream, a);
    }
    return hipGetLastError();
  });
}

template <typename IO>
hipError_t launch_step(const DeltaArgs& a, hipStream_t stream) {
  auto go = [&](auto nl) {
    constexpr int NL = decltype(nl)::value, per_pass = kThreads / NL, ROWS = 2;
    const int64_t runs = (a.P + ROWS * per_pass - 1) / (ROWS * per_pass);
    hipLaunchKernelGGL((k_delta_step<IO, NL, ROWS>), dim3((unsigned)(a.Bt * a.H * runs)), dim3(kThreads), 0,
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
  take(a.gate, n * 4 * C * sizeof(float));
  take(a.whole, n * sizeof(float));
  take(a.inv, n * 3 * frags);
  take(a.qk, n * (io_bf16 && !grads ? 2 : 3) * frags);
  take(a.park, 64 * 16);
  if (grads) {
    const size_t P16 = (a.P + 15) / 16 * 16, KP = a.N > 64 ? 128 : 64;
    const size_t state = P16 * KP * sizeof(float), cols = P16 * C * sizeof(float);
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
  return delta::launch_scan<false>(a, io_bf16, stream);
}

hipError_t launch_delta_states(const DeltaArgs& a, bool io_bf16, hipStream_t stream) {
  return delta::launch_scan<true>(a, io_bf16, stream);
}

hipError_t launch_delta_step(const DeltaArgs& a, bool io_bf16, hipStream_t stream) {
  return io_bf16 ? delta::launch_step<bf16>(a, stream) : delta::launch_step<float>(a, stream);
}

}  // namespace ssd
