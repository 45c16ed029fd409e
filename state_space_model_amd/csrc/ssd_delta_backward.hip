// Gradients of the gated delta rule's scan for gfx950.
//
// With the chunk's notation of ssd_delta.hip (K, Q the unit keys and scaled
// unit queries, W the writes, R the right sides, D the decay between tokens,
// gamma from the chunk's start, eta to its end) and E the gradient of the state
// [P, N] that leaves the chunk:
//   dW  = (D o Q K^T)^T dY + diag(eta) K E^T;    dR = (1 + L)^-T dW
//   E'  = gamma_last E + dY^T diag(gamma) Q - dR^T diag(b gamma) K   (entering it)
// chunk by chunk from the last (k_delta_back_chain), after a forward pass that
// keeps the states and the writes.  Then, all chunks at once (k_delta_grads):
//   dP = D o dY W^T (i >= j),  dL = D o dR W^T (i > j)
//   dQ = diag(gamma) dY S + dP K;        Z = diag(gamma) dR S + dL K
//   X  = diag(eta) W E + dP^T Q - dL^T diag(b) K;    dK = X - diag(b) Z
//   dV = diag(b) dR;     db_i = dR_i.V_i - K_i.Z_i
// A decay factor e^(cum_i - cum_j) gives its gradient to cum_i and takes it
// from cum_j, and where these factors stand in the terms above sums to
//   dcum_i = Q_i.dQ_i - b_i K_i.Z_i - K_i.X_i   (+ <E, S_next> at the chunk's end)
// with <E, S_next> = gamma_last <E, S> + sum_i K_i.(eta_i W_i E); the gradient
// of a token's own decay is the sum of dcum from it to the chunk's end.  Last,
// the gradients of unit keys and queries are summed over the heads that share
// them and taken through the normalisation: du = r (dU - U (U.dU)), r = 1/|u|.
#include "ssd_delta.h"

#include <type_traits>

namespace ssd {
namespace delta {
namespace {

template <typename IO, int KP, int NT>
__global__ __launch_bounds__(kThreads) void k_delta_back_chain(DeltaArgs a) {
  constexpr int PI = Planes<IO>::in;
  constexpr int KS = KP / 32, KST = KP + 8, KT = KP / 64, W = 16 * NT;
  __shared__ __align__(16) bf16 s_k[PI * C * KST], s_q[PI * C * KST];
  __shared__ __align__(16) bf16 s_s[3 * W * KST];           // E, value-major
  __shared__ __align__(16) bf16 s_y[PI * W * kTokStride];   // dY
  __shared__ __align__(16) bf16 s_g[3 * W * kTokStride];    // diag(gamma / |q|) dY
  __shared__ __align__(16) bf16 s_r[3 * W * kTokStride];    // dW
  __shared__ __align__(16) bf16 s_e[3 * W * kTokStride];    // -diag(b gamma / |k|) dR

  const int64_t slices = (a.P + W - 1) / W;
  const int64_t id = xcd_remap(blockIdx.x, gridDim.x);
  const int64_t bh = id / slices, b = bh / a.H, h = bh % a.H, g = h / (a.H / a.G);
  const int col0 = (int)(id % slices) * W;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, j = lane & 15, q = lane >> 4;
  const IO* kb = static_cast<const IO*>(a.k) + g * a.N;
  const IO* qb = static_cast<const IO*>(a.q) + g * a.N;
  const IO* yb = static_cast<const IO*>(a.dy) + h * a.P;
  bool col_in[NT];
  int col[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    col_in[n] = col0 + 16 * n + j < a.P;
    col[n] = col_in[n] ? col0 + 16 * n + j : 0;
  }

  f32x4 st[NT][KT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const int key = 16 * (KT * w + t) + 4 * q;
      st[n][t] = f32x4{0, 0, 0, 0};
      if (a.dfinal && col_in[n] && key < a.N)
        st[n][t] = *reinterpret_cast<const f32x4*>(a.dfinal + (bh * a.P + col[n]) * a.N + key);
      store_split4<3>(&s_s[(16 * n + j) * KST + key], W * KST, st[n][t]);
    }

  Frag<PI> kf[KS], qf[KS];
  Frag<3> xf[2], pf[2];
  float4 gate[4];
  IO dy[NT][4];
  float whole;
  auto load_chunk = [&](int64_t c) {
    const int64_t t0 = c * C, row0 = b * a.T + t0, left = a.T - t0, at = chunk_at(a, bh, c);
    load_rows<IO, KP>(kf, kb, a.k_stride, row0, left, a.N, 16 * w + j, q);
    load_rows<IO, KP>(qf, qb, a.q_stride, row0, left, a.N, 16 * w + j, q);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int tok = 16 * w + 4 * q + r;
      gate[r] = a.gate[at * C + tok];
      const IO* row = yb + (row0 + (tok < left ? tok : 0)) * (a.H * a.P);
#pragma unroll
      for (int n = 0; n < NT; ++n) dy[n][r] = row[col[n]];
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (s < (w >> 1)) continue;
      xf[s] = load_frag<3>(a.inv_t, at, upper_frag(w, s), lane);
      pf[s] = load_frag<3>(a.qk, at, upper_frag(w, s), lane);
    }
    whole = a.whole[at];
  };
  auto store_chunk = [&](int64_t left) {
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int i = 0; i < PI; ++i) {
        const int o = i * C * KST + (16 * w + j) * KST + 32 * s + 8 * q;
        *reinterpret_cast<bf16x8*>(&s_k[o]) = kf[s].p[i];
        *reinterpret_cast<bf16x8*>(&s_q[o]) = qf[s].p[i];
      }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int o = (16 * n + j) * kTokStride + 16 * w + 4 * q;
      f32x4 v;
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = 16 * w + 4 * q + r < left && col_in[n] ? to_f32(dy[n][r]) : 0.0f;
      store_split4<PI>(&s_y[o], W * kTokStride, v);
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] *= gate[r].w;
      store_split4<3>(&s_g[o], W * kTokStride, v);
    }
  };
  load_chunk(a.Nc - 1);
  store_chunk(a.T - (a.Nc - 1) * C);
  __syncthreads();

  for (int64_t c = a.Nc - 1; c >= 0; --c) {
    const int64_t at = chunk_at(a, bh, c);
    store_state<NT, KT>(a.leave + at * a.P * a.N, st, a.N, col, col_in, w, q);
    // dW
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      f32x4 ke = {0, 0, 0, 0}, dw = {0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < KS; ++s)
        ke = mma(kf[s], load_planes<3>(&s_s[(16 * n + j) * KST + 32 * s + 8 * q], W * KST), ke);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (s < (w >> 1)) continue;
        dw = mma(pf[s], load_planes<PI>(&s_y[(16 * n + j) * kTokStride + 32 * s + 8 * q], W * kTokStride), dw);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) dw[r] = fmaf(gate[r].z, ke[r], dw[r]);
      store_split4<3>(&s_r[(16 * n + j) * kTokStride + 16 * w + 4 * q], W * kTokStride, dw);
    }
    __syncthreads();
    // dR
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      f32x4 dr = {0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (s < (w >> 1)) continue;
        dr = mma(xf[s], load_planes<3>(&s_r[(16 * n + j) * kTokStride + 32 * s + 8 * q], W * kTokStride), dr);
      }
      if (col_in[n])
        *reinterpret_cast<f32x4*>(a.dright + (at * a.P + col[n]) * C + 16 * w + 4 * q) = dr;
#pragma unroll
      for (int r = 0; r < 4; ++r) dr[r] *= -gate[r].y;
      store_split4<3>(&s_e[(16 * n + j) * kTokStride + 16 * w + 4 * q], W * kTokStride, dr);
    }
    __syncthreads();
    // the gradient of the state that enters the chunk
    const float decay = whole;
    if (c > 0) load_chunk(c - 1);
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      Frag<PI> ka[2], qa[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        ka[s] = load_planes_tr<PI>(s_k, C * KST, KST, 32 * s, 16 * (KT * w + t), lane);
        qa[s] = load_planes_tr<PI>(s_q, C * KST, KST, 32 * s, 16 * (KT * w + t), lane);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        f32x4 acc = {0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int o = (16 * n + j) * kTokStride + 32 * s + 8 * q;
          acc = mma(qa[s], load_planes<3>(&s_g[o], W * kTokStride), acc);
          acc = mma(ka[s], load_planes<3>(&s_e[o], W * kTokStride), acc);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) st[n][t][r] = fmaf(decay, st[n][t][r], acc[r]);
        store_split4<3>(&s_s[(16 * n + j) * KST + 16 * (KT * w + t) + 4 * q], W * KST, st[n][t]);
      }
    }
    __syncthreads();
    if (c > 0) store_chunk(C);
    __syncthreads();
  }
  if (a.dh0) store_state<NT, KT>(a.dh0 + bh * a.P * a.N, st, a.N, col, col_in, w, q);
}

// ---------------------------------------------------------------------------
// The gradients of one chunk of one head.  Wavefront w owns tokens 16 w .. + 15
// of every result.  The contractions over the values run over slices of 32
// value columns, whose operands are staged as planes and read transposed.
// ---------------------------------------------------------------------------
constexpr int kSlice = 32;

template <typename IO, int KP> struct GradsLds {
  static constexpr int PI = Planes<IO>::in, KST = KP + 8;
  static constexpr int tok = 3 * kSlice * kTokStride, key = 3 * kSlice * KST;  // staged slices
  static constexpr int rows = PI * C * KST, pairs = 3 * C * kTokStride;        // k, q and the pairs
  static constexpr int first = 2 * tok + 2 * key, second = 2 * rows + 2 * pairs;
  static constexpr int elems = first > second ? first : second;
};

// value (row, key) of an LDS tile of planes
template <int NP>
__device__ __forceinline__ float plane_sum(const bf16* p, int plane) {
  float x = (float)p[(NP - 1) * plane];
#pragma unroll
  for (int i = NP - 2; i >= 0; --i) x += (float)p[i * plane];
  return x;
}
__device__ __forceinline__ float sum16(float v) {
  for (int off = 8; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

template <typename IO, int KP>
__global__ __launch_bounds__(kThreads) void k_delta_grads(DeltaArgs a) {
  using L = GradsLds<IO, KP>;
  constexpr int PI = L::PI, KST = L::KST, KT = KP / 16;
  __shared__ __align__(16) bf16 lds[L::elems];
  __shared__ float4 s_gate[C], s_row[C];
  __shared__ float s_cum[C], s_beta[C], s_sum[2 * kThreads / 64];
  bf16 *s_w = lds, *s_d = lds + L::tok, *s_s = lds + 2 * L::tok, *s_e = s_s + L::key;
  bf16 *s_k = lds, *s_q = lds + L::rows, *s_p = lds + 2 * L::rows, *s_l = s_p + L::pairs;

  const int64_t id = xcd_remap(blockIdx.x, gridDim.x);
  const int64_t h = id % a.H, c = id / a.H % a.Nc, b = id / a.H / a.Nc;
  const int64_t g = h / (a.H / a.G), bh = b * a.H + h, at = chunk_at(a, bh, c);
  const int64_t t0 = c * C, row0 = b * a.T + t0, left = a.T - t0;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, j = lane & 15, q = lane >> 4;
  if (tid < C) {
    s_gate[tid] = a.gate[at * C + tid];
    s_row[tid] = a.row[at * C + tid];
  }

  f32x4 dp[4], dl[4], dq[KT], z[KT], x[KT];
#pragma unroll
  for (int i = 0; i < 4; ++i) dp[i] = dl[i] = f32x4{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < KT; ++i) dq[i] = z[i] = x[i] = f32x4{0, 0, 0, 0};
  const bool row_in = 16 * w + j < left;
  const int64_t my_row = row0 + (row_in ? 16 * w + j : 0);
  float es = 0.0f, dr_v = 0.0f;

  for (int p0 = 0; p0 < a.P; p0 += kSlice) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSlice * C / 4 / kThreads; ++i) {
      const int at4 = tid + i * kThreads, p = at4 / (C / 4), t = at4 % (C / 4) * 4;
      const bool in = p0 + p < a.P;
      const int64_t o = (at * a.P + (in ? p0 + p : 0)) * C + t;
      f32x4 vw = *reinterpret_cast<const f32x4*>(a.write + o), vd = *reinterpret_cast<const f32x4*>(a.dright + o);
      if (!in) vw = vd = f32x4{0, 0, 0, 0};
      store_split4<3>(&s_w[p * kTokStride + t], kSlice * kTokStride, vw);
      store_split4<3>(&s_d[p * kTokStride + t], kSlice * kTokStride, vd);
    }
#pragma unroll
    for (int i = 0; i < kSlice * KP / 4 / kThreads; ++i) {
      const int at4 = tid + i * kThreads, p = at4 / (KP / 4), key = at4 % (KP / 4) * 4;
      const bool in = p0 + p < a.P && key < a.N;
      const int64_t o = (at * a.P + (in ? p0 + p : 0)) * a.N + (in ? key : 0);
      f32x4 vs = *reinterpret_cast<const f32x4*>(a.enter + o), ve = *reinterpret_cast<const f32x4*>(a.leave + o);
      if (!in) vs = ve = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < 4; ++e) es = fmaf(vs[e], ve[e], es);
      store_split4<3>(&s_s[p * KST + key], kSlice * KST, vs);
      store_split4<3>(&s_e[p * KST + key], kSlice * KST, ve);
    }
    const bool col_in = p0 + 8 * q < a.P;
    const int64_t pc = h * a.P + (col_in ? p0 + 8 * q : 0);
    const auto dyf = load_io8<IO>(static_cast<const IO*>(a.dy) + my_row * (a.H * a.P) + pc, row_in && col_in);
    const auto vf = load_io8<IO>(static_cast<const IO*>(a.v) + my_row * a.v_stride + pc, row_in && col_in);
    __syncthreads();
    const auto drf = load_planes_tr<3>(s_d, kSlice * kTokStride, kTokStride, 0, 16 * w, lane);
    const auto wf = load_planes_tr<3>(s_w, kSlice * kTokStride, kTokStride, 0, 16 * w, lane);
    {
      const float beta = s_gate[16 * w + j].x;
      IO out[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = ((float)drf.p[2][e] + (float)drf.p[1][e]) + (float)drf.p[0][e];
        float v = (float)vf.p[PI - 1][e];
#pragma unroll
        for (int i = PI - 2; i >= 0; --i) v += (float)vf.p[i][e];
        dr_v = fmaf(d, v, dr_v);
        out[e] = to_io<IO>(beta * d);
      }
      if (row_in && col_in) {
        IO* to = static_cast<IO*>(a.dv) + my_row * a.dv_stride + pc;
        if constexpr (sizeof(IO) == 2) {
          *reinterpret_cast<bf16x8*>(to) = bf16x8{out[0], out[1], out[2], out[3], out[4], out[5], out[6], out[7]};
        } else {
          *reinterpret_cast<float4*>(to) = make_float4(out[0], out[1], out[2], out[3]);
          *reinterpret_cast<float4*>(to + 4) = make_float4(out[4], out[5], out[6], out[7]);
        }
      }
    }
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) {
      if (jt > w) continue;
      const auto wb = load_planes_tr<3>(s_w, kSlice * kTokStride, kTokStride, 0, 16 * jt, lane);
      dp[jt] = mma(dyf, wb, dp[jt]);
      dl[jt] = mma(drf, wb, dl[jt]);
    }
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      const auto sb = load_planes_tr<3>(s_s, kSlice * KST, KST, 0, 16 * kt, lane);
      dq[kt] = mma(dyf, sb, dq[kt]);
      z[kt] = mma(drf, sb, z[kt]);
      x[kt] = mma(wf, load_planes_tr<3>(s_e, kSlice * KST, KST, 0, 16 * kt, lane), x[kt]);
    }
  }
  __syncthreads();

  {
    Frag<PI> kf[KP / 32], qf[KP / 32];
    load_rows<IO, KP>(kf, static_cast<const IO*>(a.k) + g * a.N, a.k_stride, row0, left, a.N, 16 * w + j, q);
    load_rows<IO, KP>(qf, static_cast<const IO*>(a.q) + g * a.N, a.q_stride, row0, left, a.N, 16 * w + j, q);
#pragma unroll
    for (int s = 0; s < KP / 32; ++s)
#pragma unroll
      for (int i = 0; i < PI; ++i) {
        const int o = i * C * KST + (16 * w + j) * KST + 32 * s + 8 * q;
        *reinterpret_cast<bf16x8*>(&s_k[o]) = kf[s].p[i];
        *reinterpret_cast<bf16x8*>(&s_q[o]) = qf[s].p[i];
      }
  }
  // the pairs (i, j) of this wavefront's tokens i, over their decay, stored
  // [j][i]; times 1/|k_j| for the sums over j
  float4 rec[4];
  float gamma[4], eta[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    rec[r] = s_row[16 * w + 4 * q + r];
    gamma[r] = exp2_of(rec[r].z + rec[r].w);
    eta[r] = exp2_of((s_row[C - 1].z - rec[r].z) + (s_row[C - 1].w - rec[r].w));
  }
#pragma unroll
  for (int jt = 0; jt < 4; ++jt) {
    const int cj = 16 * jt + j;
    const float4 rj = s_row[cj];
    f32x4 vp, vl;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int ri = 16 * w + 4 * q + r;
      const float dec = exp2_of((rec[r].z - rj.z) + (rec[r].w - rj.w));
      dp[jt][r] = ri >= cj ? dec * dp[jt][r] : 0.0f;
      dl[jt][r] = ri > cj ? dec * dl[jt][r] : 0.0f;
      vp[r] = dp[jt][r] * rj.x;
      vl[r] = dl[jt][r] * rj.x;
    }
    store_split4<3>(&s_p[cj * kTokStride + 16 * w + 4 * q], C * kTokStride, vp);
    store_split4<3>(&s_l[cj * kTokStride + 16 * w + 4 * q], C * kTokStride, vl);
  }
  __syncthreads();
  // K . (eta W E) for the gradient at the chunk's end
  float end_sum = 0.0f;
#pragma unroll
  for (int kt = 0; kt < KT; ++kt)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      dq[kt][r] *= gamma[r];
      z[kt][r] *= gamma[r];
      x[kt][r] *= eta[r];
      const float k = rec[r].x * plane_sum<PI>(&s_k[(16 * w + 4 * q + r) * KST + 16 * kt + j], C * KST);
      end_sum = fmaf(k, x[kt][r], end_sum);
    }
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    if (s > (w >> 1)) continue;
    const auto pa = load_planes_tr<3>(s_p, C * kTokStride, kTokStride, 32 * s, 16 * w, lane);
    const auto la = load_planes_tr<3>(s_l, C * kTokStride, kTokStride, 32 * s, 16 * w, lane);
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      const auto kb = load_planes_tr<PI>(s_k, C * KST, KST, 32 * s, 16 * kt, lane);
      dq[kt] = mma(pa, kb, dq[kt]);
      z[kt] = mma(la, kb, z[kt]);
    }
  }
  __syncthreads();
  // the same pairs for the sums over i
#pragma unroll
  for (int jt = 0; jt < 4; ++jt) {
    const int cj = 16 * jt + j;
    f32x4 vp, vl;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      vp[r] = dp[jt][r] * rec[r].y;
      vl[r] = -dl[jt][r] * s_gate[16 * w + 4 * q + r].x * rec[r].x;
    }
    store_split4<3>(&s_p[cj * kTokStride + 16 * w + 4 * q], C * kTokStride, vp);
    store_split4<3>(&s_l[cj * kTokStride + 16 * w + 4 * q], C * kTokStride, vl);
  }
  __syncthreads();
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    if (s < (w >> 1)) continue;
    const int o = (16 * w + j) * kTokStride + 32 * s + 8 * q;
    const auto pa = load_planes<3>(&s_p[o], C * kTokStride);
    const auto la = load_planes<3>(&s_l[o], C * kTokStride);
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      x[kt] = mma(pa, load_planes_tr<PI>(s_q, C * KST, KST, 32 * s, 16 * kt, lane), x[kt]);
      x[kt] = mma(la, load_planes_tr<PI>(s_k, C * KST, KST, 32 * s, 16 * kt, lane), x[kt]);
    }
  }

  // row sums, and the gradients of unit keys and scaled unit queries
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int ri = 16 * w + 4 * q + r;
    const float beta = s_gate[ri].x;
    float kz = 0.0f, kx = 0.0f, qd = 0.0f;
    float* pq = a.part_q + ((row0 + ri) * a.H + h) * a.N;
    float* pk = a.part_k + ((row0 + ri) * a.H + h) * a.N;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      const int o = ri * KST + 16 * kt + j;
      const float k = plane_sum<PI>(&s_k[o], C * KST), u = plane_sum<PI>(&s_q[o], C * KST);
      kz = fmaf(k, z[kt][r], kz);
      kx = fmaf(k, x[kt][r], kx);
      qd = fmaf(u, dq[kt][r], qd);
      if (ri < left && 16 * kt + j < a.N) {
        pq[16 * kt + j] = dq[kt][r];
        pk[16 * kt + j] = x[kt][r] - beta * z[kt][r];
      }
    }
    kz = rec[r].x * sum16(kz);
    kx = rec[r].x * sum16(kx);
    qd = rec[r].y * sum16(qd);
    if (j == 0) {
      s_cum[ri] = qd - beta * kz - kx;
      s_beta[ri] = -kz;
    }
  }
  es = wave_sum64(es);
  end_sum = wave_sum64(end_sum);
  dr_v += __shfl_xor(dr_v, 16, 64);
  dr_v += __shfl_xor(dr_v, 32, 64);
  if (lane == 0) {
    s_sum[w] = es;
    s_sum[4 + w] = end_sum;
  }
  __builtin_amdgcn_wave_barrier();
  if (q == 0) s_beta[16 * w + j] += dr_v;   // rows of this wavefront
  __syncthreads();
  if (w != 0) return;

  // token `lane`: its decay and write strength
  const float all = a.whole[at] * ((s_sum[0] + s_sum[1]) + (s_sum[2] + s_sum[3])) +
                    ((s_sum[4] + s_sum[5]) + (s_sum[6] + s_sum[7]));
  float dg = s_cum[lane] + (lane == C - 1 ? all : 0.0f);
  for (int off = 1; off < 64; off <<= 1) {
    const float o = __shfl_down(dg, off, 64);
    if (lane + off < 64) dg += o;
  }
  const bool in = lane < left;
  const int64_t th = (row0 + (in ? lane : 0)) * a.H + h;
  const float zt = a.dt[th] + (a.dt_bias ? a.dt_bias[h] : 0.0f);
  const float pre = a.softplus ? softplus_of(zt) : zt;   // as in delta_of: the same clip decision
  const float rate = fminf(fmaxf(pre, a.dt_min), a.dt_max);
  float slope = pre >= a.dt_min && pre <= a.dt_max ? a.A[h] : 0.0f;
  if (a.softplus) slope *= sigmoid_of(zt);
  const float ddt = in ? dg * slope : 0.0f;
  const float sum_a = wave_sum64(in ? dg * rate : 0.0f), sum_b = wave_sum64(ddt);
  if (in) {
    const float beta = s_gate[lane].x;
    a.ddt[th] = ddt;
    a.dbeta[th] = s_beta[lane] * (a.sigmoid ? beta * (1.0f - beta) : 1.0f);
  }
  if (lane == 0) {
    a.part_h[2 * at] = sum_a;
    a.part_h[2 * at + 1] = sum_b;
  }
}

// Gradients of a token's keys or queries of one group from those of the unit
// vectors of its heads: NL lanes of four keys a row.
template <typename IO, int NL>
__global__ __launch_bounds__(kThreads) void k_delta_unit_grads(DeltaArgs a) {
  const int64_t id = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / NL;
  const int64_t rows = a.Bt * a.T * a.G;
  const bool in = id < 2 * rows;
  const bool is_q = id < rows;
  const int64_t row = in ? (is_q ? id : id - rows) : 0;
  const int64_t tok = row / a.G, g = row % a.G, per = a.H / a.G;
  const int key = 4 * (threadIdx.x % NL);
  const bool key_in = in && key < a.N;
  const int at = key_in ? key : 0;
  const float* part = (is_q ? a.part_q : a.part_k) + (tok * a.H + g * per) * a.N + at;
  f32x4 d = {0, 0, 0, 0};
  for (int64_t i = 0; i < per; ++i) d += *reinterpret_cast<const f32x4*>(part + i * a.N);
  const IO* xr = static_cast<const IO*>(is_q ? a.q : a.k) + tok * (is_q ? a.q_stride : a.k_stride) + g * a.N + at;
  f32x4 x;
  float ss = 0.0f, dot = 0.0f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[e] = key_in ? to_f32(xr[e]) : 0.0f;
    d[e] = key_in ? d[e] : 0.0f;
    ss = fmaf(x[e], x[e], ss);
    dot = fmaf(x[e], d[e], dot);
  }
  for (int off = NL >> 1; off > 0; off >>= 1) {
    ss += __shfl_xor(ss, off, 64);
    dot += __shfl_xor(dot, off, 64);
  }
  const float scale = is_q ? a.scale : 1.0f;
  if (a.unit) {
    const float r = 1.0f / sqrtf(ss + a.norm_eps), t = r * dot * r;
#pragma unroll
    for (int e = 0; e < 4; ++e) d[e] = scale * r * fmaf(-x[e], t, d[e]);
  } else {
    d *= scale;
  }
  if (key_in) {
    IO* to = static_cast<IO*>(is_q ? a.dq : a.dk) + tok * (is_q ? a.dq_stride : a.dk_stride) + g * a.N + key;
    if constexpr (sizeof(IO) == 2)
      *reinterpret_cast<bf16x4*>(to) = bf16x4{(bf16)d[0], (bf16)d[1], (bf16)d[2], (bf16)d[3]};
    else
      *reinterpret_cast<f32x4*>(to) = d;
  }
}

// dA and ddt_bias of a head: the chunks' parts in a fixed order
__global__ __launch_bounds__(kThreads) void k_delta_head_grads(DeltaArgs a) {
  __shared__ double s[2][kThreads];
  const int64_t h = blockIdx.x, n = a.Bt * a.Nc;
  double sa = 0.0, sb = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += kThreads) {
    const int64_t at = (i / a.Nc * a.H + h) * a.Nc + i % a.Nc;
    sa += a.part_h[2 * at];
    sb += a.part_h[2 * at + 1];
  }
  s[0][threadIdx.x] = sa;
  s[1][threadIdx.x] = sb;
  __syncthreads();
  for (int half = kThreads / 2; half > 0; half >>= 1) {
    if ((int)threadIdx.x < half) {
      s[0][threadIdx.x] += s[0][threadIdx.x + half];
      s[1][threadIdx.x] += s[1][threadIdx.x + half];
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    a.dA[h] = (float)s[0][0];
    if (a.ddt_bias) a.ddt_bias[h] = (float)s[1][0];
  }
}

template <typename IO, int KP>
hipError_t launch_grads(const DeltaArgs& a, hipStream_t stream) {
  const unsigned chunks = (unsigned)(a.Bt * a.H * a.Nc), chains = (unsigned)(a.Bt * a.H * ((a.P + 15) / 16));
  hipLaunchKernelGGL((k_delta_back_chain<IO, KP, 1>), dim3(chains), dim3(kThreads), 0, stream, a);
  hipLaunchKernelGGL((k_delta_grads<IO, KP>), dim3(chunks), dim3(kThreads), 0, stream, a);
  constexpr int per = kThreads / (KP / 4);
  const int64_t rows = 2 * a.Bt * a.T * a.G;
  hipLaunchKernelGGL((k_delta_unit_grads<IO, KP / 4>), dim3((unsigned)((rows + per - 1) / per)), dim3(kThreads), 0,
                     stream, a);
  hipLaunchKernelGGL(k_delta_head_grads, dim3((unsigned)a.H), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace
}  // namespace delta

hipError_t launch_delta_scan_backward(const DeltaArgs& a, bool io_bf16, hipStream_t stream) {
  const hipError_t e = launch_delta_states(a, io_bf16, stream);
  if (e != hipSuccess) return e;
  using namespace delta;
  if (a.N <= 64)
    return io_bf16 ? launch_grads<bf16, 64>(a, stream) : launch_grads<float, 64>(a, stream);
  return io_bf16 ? launch_grads<bf16, 128>(a, stream) : launch_grads<float, 128>(a, stream);
}

}  // namespace ssd
