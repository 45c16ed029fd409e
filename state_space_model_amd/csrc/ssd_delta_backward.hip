// Gradients of the gated delta rule's scan for gfx950.
//
// With the chunk's notation of ssd_delta.hip (K, Q the unit keys and scaled
// unit queries, W the writes, R the right sides, D the decay between tokens,
// gamma from the chunk's start, eta to its end) and E the gradient of the state
// [P, N] that leaves the chunk:
//   dW  = (D o Q K^T)^T dY + diag(eta) K E^T;    dR = (1 + L)^-T dW
//   E'  = gamma_last E + dY^T diag(gamma) Q - dR^T diag(b gamma) K   (entering it)
// chunk by chunk from the last (back_*), next to a forward pass that keeps the
// states and the writes.  Then, all chunks at once (k_delta_grads):
//   dP = D o dY W^T (i >= j),  dL = D o dR W^T (i > j)
//   dQ = diag(gamma) dY S + dP K;        Z = diag(gamma) dR S + dL K
//   X  = diag(eta) W E + dP^T Q - dL^T diag(b) K;    dK = X - diag(b) Z
//   dV = diag(b) dR;     db_i = dR_i.V_i - K_i.Z_i
// The decay of token t stands in every factor that spans it, so its gradient is
//   sum_{i >= t > j} (dP_ij Q_i.K_j - b_i dL_ij K_i.K_j)            pairs across t
//   + sum_{i >= t} gamma_i (Q_i.(dY S)_i - b_i K_i.(dR S)_i)     reads of the entering state
//   + sum_{j < t} eta_j K_j.(W E)_j + gamma_last <E, S>           what reaches the end
// Last, the gradients of unit keys and queries are summed over the heads that share
// them and taken through the normalisation: du = r (dU - U (U.dU)), r = 1/|u|.
#include "ssd_delta_chains.h"

namespace ssd {
namespace delta {
namespace {

// The matrix cores do not round their sums to nearest: a sum comes out a little low
// on the average, whatever its sign.  Through a sum of products with states, keys
// and queries, whose elements have a mean, that shows in the decays' gradients,
// and in those of A, a sum over all tokens, most.  So odd value columns of the
// chains from the last chunk (what they leave in the workspace included) and odd
// tokens of k_delta_grads are computed with the opposite sign: the bias of one half
// takes that of the other back (dA of 4096 tokens of 32 heads: 1.3e-6 -> 2e-7).
__device__ __forceinline__ float odd_sign(int i) { return i & 1 ? -1.0f : 1.0f; }
__device__ __forceinline__ uint32_t odd_flip(int i) { return i & 1 ? 0x80008000u : 0u; }
// the operand, negated where `flip` has the signs of two elements set
template <int NP> __device__ __forceinline__ Frag<NP> with_sign(Frag<NP> f, uint32_t flip) {
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const uint4 v = __builtin_bit_cast(uint4, f.p[i]);
    f.p[i] = __builtin_bit_cast(bf16x8, make_uint4(v.x ^ flip, v.y ^ flip, v.z ^ flip, v.w ^ flip));
  }
  return f;
}

// As chain, from the last chunk to the first.
template <typename IO, int KP, int NT> struct BackChainLds {
  static constexpr int PI = Planes<IO>::in, W = 16 * NT, tok = W * kTokStride;
  static constexpr int k = 0, q = k + PI * C * (KP + 16), s = q + PI * C * (KP + 16), y = s + 3 * W * (KP + 8);
  static constexpr int g = y + PI * tok, r = g + 3 * tok, e = r + 3 * tok, elems = e + 3 * tok;
};

template <typename IO, int KP, bool FULL, int NT>
__device__ __forceinline__ void back_chain(const DeltaArgs& a, bf16* lds, int64_t id) {
  using L = BackChainLds<IO, KP, NT>;
  constexpr int PI = Planes<IO>::in;
  constexpr int KS = KP / 32, KST = KP + 8, KTR = KP + 16, KT = KP / 64, W = 16 * NT;
  bf16 *const s_k = lds + L::k, *const s_q = lds + L::q;
  bf16* const s_s = lds + L::s;   // E, value-major
  bf16* const s_y = lds + L::y;   // dY
  bf16* const s_g = lds + L::g;   // diag(gamma / |q|) dY
  bf16* const s_r = lds + L::r;   // dW
  bf16* const s_e = lds + L::e;   // -diag(b gamma / |k|) dR

  const int slices = (a.P + W - 1) / W;
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

  const float sign = odd_sign(j);
  f32x4 st[NT][KT];
  const int key0 = 16 * KT * w + 4 * q;
  bf16* const put_s = &s_s[j * KST + key0];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      st[n][t] = f32x4{0, 0, 0, 0};
      if (a.dfinal && col_in[n] && key0 + 16 * t < a.N)
        st[n][t] = sign * *reinterpret_cast<const f32x4*>(a.dfinal + (bh * a.P + col[n]) * a.N + key0 + 16 * t);
      store_split4<3>(put_s + 16 * n * KST + 16 * t, W * KST, st[n][t]);
    }

  // where the lane's rows are: row 16 w + j of k and q, rows 16 w + 4 q + r of dy
  const IO *kp, *qp, *yp[4];
  const int64_t y_row = a.H * a.P;
  auto rows_of = [&](int64_t c) {
    const int64_t row0 = b * a.T + c * C, left = a.T - c * C;
    const int64_t row = row0 + (16 * w + j < left ? 16 * w + j : left - 1), at = g * a.N + 8 * q;
    kp = static_cast<const IO*>(a.k) + row * a.k_stride + at;
    qp = static_cast<const IO*>(a.q) + row * a.q_stride + at;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int tok = 16 * w + 4 * q + r;
      yp[r] = static_cast<const IO*>(a.dy) + (row0 + (tok < left ? tok : left - 1)) * y_row + h * a.P;
    }
  };
  const int64_t at_last = chunk_at(a, bh, a.Nc - 1);
  const float* gp = a.gate + at_last * kGates + 16 * w + 4 * q;
  const bf16* xp = a.inv_t + (at_last * kTriFrags + upper_frag(w, w >> 1)) * (3 * kFrag) + lane * 8;
  const bf16* pp = a.qk + (at_last * kTriFrags + upper_frag(w, w >> 1)) * (3 * kFrag) + lane * 8;
  const float* ep = a.whole + at_last;
  const int second = w < 2 ? 1 : 0;   // wavefronts 2 and 3: the first fragment again, unused
  const int64_t cols = padded_cols(a.P);
  float* state_at = a.leave + (at_last * cols + col0 + j) * KP + key0;
  float* right_at = a.dright + (at_last * cols + col0 + j) * C + 16 * w + 4 * q;

  KeyRow<IO, KP, FULL> kr, qr;
  Frag<3> xf[2], pf[2];
  f32x4 g_right, g_end, g_out;
  IO dy[NT][4];
  auto load_rows = [&]() {
    kr.load(kp, a.N, q);
    qr.load(qp, a.N, q);
    g_right = *reinterpret_cast<const f32x4*>(gp + kRight);
    g_end = *reinterpret_cast<const f32x4*>(gp + kEnd);
    g_out = *reinterpret_cast<const f32x4*>(gp + kOut);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int n = 0; n < NT; ++n) dy[n][r] = yp[r][col[n]];
  };
  // row tiles 0 and 1 reach over all columns, 2 and 3 over the last 32
  auto load_upper = [&](Frag<3>(&f)[2], const bf16* from) {
    f[0] = load_planes<3>(from, kFrag);
    f[1] = load_planes<3>(from + second * (3 * kFrag), kFrag);
  };
  bf16 *const put_k = &s_k[(16 * w + j) * KTR + 8 * q], *const put_q = &s_q[(16 * w + j) * KTR + 8 * q];
  const int put_t = j * kTokStride + token_slot(w, q), get_t = j * kTokStride + 8 * q;
  auto store_chunk = [&]() {
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const auto kf = kr.frag(s, a.N, q);
      const auto qf = qr.frag(s, a.N, q);
#pragma unroll
      for (int i = 0; i < PI; ++i) {
        *reinterpret_cast<bf16x8*>(put_k + i * C * KTR + 32 * s) = kf.p[i];
        *reinterpret_cast<bf16x8*>(put_q + i * C * KTR + 32 * s) = qf.p[i];
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      f32x4 v;
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = sign * to_f32(dy[n][r]);
      store_split4<PI>(s_y + put_t + 16 * n * kTokStride, W * kTokStride, v);
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] *= g_out[r];
      store_split4<3>(s_g + put_t + 16 * n * kTokStride, W * kTokStride, v);
    }
  };
  rows_of(a.Nc - 1);
  load_rows();
  load_upper(xf, xp);
  load_upper(pf, pp);
  float whole = *ep;
  store_chunk();
  __syncthreads();

  const bf16* const get_s = &s_s[j * KST + 8 * q];
  const int get_k = (4 * q + (j >> 2)) * KTR + 16 * KT * w + 4 * (j & 3);
  const int t_first = w < 2 ? 0 : 32;
  for (int64_t c = a.Nc - 1; c >= 0; --c) {
    const int64_t next = c > 0 ? 1 : 0;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int t = 0; t < KT; ++t)
        *reinterpret_cast<f32x4*>(state_at + 16 * n * KP + 16 * t) = st[n][t];
    state_at -= cols * KP;
    // dW
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      f32x4 ke = {0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < KS; ++s)
        ke = mma(kr.frag(s, a.N, q), load_planes<3>(get_s + 16 * n * KST + 32 * s, W * KST), ke);
      f32x4 dw = mma(pf[0], load_planes<PI>(s_y + get_t + 16 * n * kTokStride + t_first, W * kTokStride),
                     f32x4{0, 0, 0, 0});
      if (w < 2) dw = mma(pf[1], load_planes<PI>(s_y + get_t + 16 * n * kTokStride + 32, W * kTokStride), dw);
#pragma unroll
      for (int r = 0; r < 4; ++r) dw[r] = fmaf(g_end[r], ke[r], dw[r]);
      store_split4<3>(s_r + put_t + 16 * n * kTokStride, W * kTokStride, dw);
    }
    const f32x4 gamma = -g_right;
    if (next && c == a.Nc - 1) {
      rows_of(c - 1);
    } else {
      kp -= next * a.k_stride * C;
      qp -= next * a.q_stride * C;
#pragma unroll
      for (int r = 0; r < 4; ++r) yp[r] -= next * y_row * C;
    }
    gp -= next * kGates;
    load_rows();
    pp -= next * (kTriFrags * 3 * kFrag);
    load_upper(pf, pp);
    __syncthreads();
    // dR
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      f32x4 dr = mma(xf[0], load_planes<3>(s_r + get_t + 16 * n * kTokStride + t_first, W * kTokStride),
                     f32x4{0, 0, 0, 0});
      if (w < 2) dr = mma(xf[1], load_planes<3>(s_r + get_t + 16 * n * kTokStride + 32, W * kTokStride), dr);
      *reinterpret_cast<f32x4*>(right_at + 16 * n * C) = dr;
#pragma unroll
      for (int r = 0; r < 4; ++r) dr[r] *= gamma[r];
      store_split4<3>(s_e + put_t + 16 * n * kTokStride, W * kTokStride, dr);
    }
    right_at -= cols * C;
    xp -= next * (kTriFrags * 3 * kFrag);
    load_upper(xf, xp);
    __syncthreads();
    // the gradient of the state that enters the chunk
    const float decay = whole;
    ep -= next;
    whole = *ep;
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      Frag<PI> ka[2], qa[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        ka[s] = read_tr<PI>(s_k + get_k + 32 * s * KTR + 16 * t, C * KTR, 16 * KTR);
        qa[s] = read_tr<PI>(s_q + get_k + 32 * s * KTR + 16 * t, C * KTR, 16 * KTR);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        f32x4 acc = {0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int o = get_t + 16 * n * kTokStride + 32 * s;
          acc = mma(qa[s], load_planes<3>(s_g + o, W * kTokStride), acc);
          acc = mma(ka[s], load_planes<3>(s_e + o, W * kTokStride), acc);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) st[n][t][r] = fmaf(decay, st[n][t][r], acc[r]);
        store_split4<3>(put_s + 16 * n * KST + 16 * t, W * KST, st[n][t]);
      }
    }
    __syncthreads();
    store_chunk();
    __syncthreads();
  }
  if (a.dh0) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int t = 0; t < KT; ++t)
        if (col_in[n] && key0 + 16 * t < a.N)
          *reinterpret_cast<f32x4*>(a.dh0 + (bh * a.P + col[n]) * a.N + key0 + 16 * t) = sign * st[n][t];
  }
}

// ---------------------------------------------------------------------------
// The same for bfloat16 io, as k_delta_columns: every wavefront owns 16 value
// columns alone.
// ---------------------------------------------------------------------------
template <int KP, int NW> struct BackLds {
  using Keys = KeyTile<KP, NW>;
  static constexpr int k = 0, q = k + Keys::kElems, x = q + Keys::kElems, p = x + 3 * kTriFrags * kFrag;
  static constexpr int y = p + 3 * kTriFrags * kFrag, gate = y + C * 16 * NW, elems = gate + 2 * kGates;
};

template <int KP, bool FULL>
__device__ __forceinline__ void back_columns(const DeltaArgs& a, bf16* lds, int64_t id) {
  constexpr int NW = 4, KS = KP / 32, KT = KP / 16, W = 16 * NW;
  using L = BackLds<KP, NW>;
  using Keys = KeyTile<KP, NW>;
  using Cols = ColumnTile<NW>;

  const int slices = (a.P + W - 1) / W;
  const int64_t bh = id / slices, b = bh / a.H, h = bh % a.H, g = h / (a.H / a.G);
  const int col0 = (int)(id % slices) * W;
  const int tid = threadIdx.x, lane = tid & 63, w = wave_of(tid), j = lane & 15, q = lane >> 4;
  const int col = col0 + 16 * w + j;
  const bool col_in = col < a.P, idle = col0 + 16 * w >= a.P;
  const int64_t c_last = a.Nc - 1, at = chunk_at(a, bh, c_last), cols = padded_cols(a.P);

  for (int i = tid; i < L::elems / 8; i += 256) reinterpret_cast<uint4*>(lds)[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  typename Keys::Offsets k_off, q_off;
  typename Cols::Offsets y_off;
  const int64_t y_row = a.H * a.P;
  auto offsets = [&](int last) {
    Keys::offsets(k_off, (int)a.k_stride, last, a.N, w, lane);
    Keys::offsets(q_off, (int)a.q_stride, last, a.N, w, lane);
    Cols::offsets(y_off, (int)y_row, last, a.P - col0, w, lane);
  };
  const uint32_t lds0 = lds_address(lds) + w * 1024;
  const int64_t row0 = b * a.T + c_last * C;
  const bf16* kp = static_cast<const bf16*>(a.k) + row0 * a.k_stride + g * a.N;
  const bf16* qp = static_cast<const bf16*>(a.q) + row0 * a.q_stride + g * a.N;
  const bf16* yp = static_cast<const bf16*>(a.dy) + row0 * y_row + h * a.P + col0;
  const bf16* xp = a.inv_t + at * (3 * kTriFrags * kFrag) + w * 512;
  const bf16* pp = a.qk + at * (3 * kTriFrags * kFrag) + w * 512;
  const float* gp = a.gate + at * kGates + w * 256;
  const bool all_cols = a.P - col0 >= W;
  auto request = [&]() {
    Keys::template request<FULL>(kp, k_off, lds0 + 2 * L::k);
    Keys::template request<FULL>(qp, q_off, lds0 + 2 * L::q);
    request_linear<3 * kTriFrags, NW>(xp, lds0 + 2 * L::x, w, lane);
    request_linear<3 * kTriFrags, NW>(pp, lds0 + 2 * L::p, w, lane);
    if (all_cols) Cols::template request<true>(yp, y_off, lds0 + 2 * L::y);
    else Cols::template request<false>(yp, y_off, lds0 + 2 * L::y);
    request_linear<1, NW>(gp, lds0 + 2 * L::gate, w, lane);
  };
  offsets((int)(a.T - c_last * C) - 1);
  request();

  const float sign = odd_sign(j);
  f32x4 st[KT];
#pragma unroll
  for (int t = 0; t < KT; ++t) {
    const int key = key_of(t, 4 * q);
    st[t] = f32x4{0, 0, 0, 0};
    if (a.dfinal && col_in && key < a.N)
      st[t] = sign * *reinterpret_cast<const f32x4*>(a.dfinal + (bh * a.P + col) * a.N + key);
  }
  float* state_at = a.leave + (at * cols + col) * KP + 8 * q;
  float* right_at = a.dright + (at * cols + col) * C + 4 * q;
  int row_at[KS], col_at[KT / 2];
#pragma unroll
  for (int s = 0; s < KS; ++s) row_at[s] = Keys::row_at(s, j, q);
#pragma unroll
  for (int u = 0; u < KT / 2; ++u) col_at[u] = Keys::col_at(u, j, q);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
  for (int t = 0; t < KT; ++t) pin(st[t]);
  offsets(C - 1);

  for (int64_t c = c_last; c >= 0; --c) {
    landed<0>();
    const float whole = load_uniform(a.whole + at - c_last + c);
    const float* const gate = reinterpret_cast<const float*>(lds + L::gate) + 4 * q;
    auto gates = [&](int which, int i) { return *reinterpret_cast<const f32x4*>(gate + which + 16 * i); };
    if (!idle) {
#pragma unroll
      for (int t = 0; t < KT; ++t) *reinterpret_cast<f32x4*>(state_at + key_of(t, 0)) = st[t];
      state_at -= cols * KP;
    }
    // dW
    f32x4 ke[4], dw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) ke[i] = dw[i] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      Frag<1> rows[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) rows[i] = load_planes<1>(lds + L::k + row_at[s] + 16 * i * KP, 0);
      mma_tiles(rows, right_of<3>(st[2 * s], st[2 * s + 1]), ke);
    }
    Frag<1> dy[2];
    Frag<3> rf[2], gf[2];
#pragma unroll
    for (int s = 0; s < 2; ++s)
      dy[s] = with_sign(read_tr2(lds + L::y + (32 * s + 4 * q + (j >> 2)) * W + 16 * w + 4 * (j & 3), 16 * W), odd_flip(j));
    mma_upper<3>(lds + L::p + lane * 8, dy, dw);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4 ge = gates(kEnd, i);
#pragma unroll
      for (int r = 0; r < 4; ++r) dw[i][r] = fmaf(ge[r], ke[i][r], dw[i][r]);
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) rf[s] = right_of<3>(dw[2 * s], dw[2 * s + 1]);
    // dR
    f32x4 dr[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) dr[i] = f32x4{0, 0, 0, 0};
    mma_upper<3>(lds + L::x + lane * 8, rf, dr);
    if (!idle) {
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<f32x4*>(right_at + 16 * i) = dr[i];
      right_at -= cols * C;
    }
    // the gradient of the state that enters the chunk
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      rf[s] = right_of<3>(-gates(kRight, 2 * s) * dr[2 * s], -gates(kRight, 2 * s + 1) * dr[2 * s + 1]);
      f32x4 lo = gates(kOut, 2 * s), hi = gates(kOut, 2 * s + 1);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        lo[r] *= (float)dy[s].p[0][r];
        hi[r] *= (float)dy[s].p[0][4 + r];
      }
      gf[s] = right_of<3>(lo, hi);
    }
#pragma unroll
    for (int t0 = 0; t0 < KT; t0 += 4) {
      f32x4 acc[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) acc[t] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        Frag<1> cols4[4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
          cols4[t] = Keys::columns(lds + L::q + col_at[(t0 + t) / 2] + 4 * (t & 1) + 32 * s * KP);
        mma_tiles(cols4, gf[s], acc);
#pragma unroll
        for (int t = 0; t < 4; ++t)
          cols4[t] = Keys::columns(lds + L::k + col_at[(t0 + t) / 2] + 4 * (t & 1) + 32 * s * KP);
        mma_tiles(cols4, rf[s], acc);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) st[t0 + t][r] = fmaf(whole, st[t0 + t][r], acc[t][r]);
    }
    lds_free();
    if (c > 0) {
      kp -= C * a.k_stride;
      qp -= C * a.q_stride;
      yp -= C * y_row;
      xp -= 3 * kTriFrags * kFrag;
      pp -= 3 * kTriFrags * kFrag;
      gp -= kGates;
      request();
    }
  }
  if (a.dh0 && col_in) {
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const int key = key_of(t, 4 * q);
      if (key < a.N) *reinterpret_cast<f32x4*>(a.dh0 + (bh * a.P + col) * a.N + key) = sign * st[t];
    }
  }
}

// ---------------------------------------------------------------------------
// The same for bfloat16 io, as k_delta_tokens: four wavefronts share 16 value
// columns.  Requests, and what they wait for:
//   top        q of this chunk; k, gates of the one before it (two places for each)
//   barrier 1  q k^T, dy of the one before   (waits for the inverse)
//   barrier 2  its inverse                   (waits for q)
//   barrier 3                                (waits for k, gates, q k^T, dy)
// ---------------------------------------------------------------------------
template <int KP, int NG> struct BackTokensLds {
  using Keys = KeyTile<KP, 4 * NG>;
  static constexpr int W = 16 * NG;
  static constexpr int k = 0, q = k + 2 * Keys::kElems, x = q + Keys::kElems, p = x + 3 * kTriFrags * kFrag;
  static constexpr int y = p + 3 * kTriFrags * kFrag, gate = y + C * W, s = gate + 4 * kGates;
  static constexpr int r = s + 3 * W * KP, e = r + 3 * W * C, g = e + 3 * W * C, elems = g + 3 * W * C;
};

template <int KP, bool FULL, int NG>
__device__ __forceinline__ void back_tokens(const DeltaArgs& a, bf16* lds, int64_t id) {
  using L = BackTokensLds<KP, NG>;
  using Keys = typename L::Keys;
  constexpr int KS = KP / 32, KT = KP / 64, W = L::W, NW = 4 * NG;
  constexpr int kKeyLoads = Keys::kLoads, kTriLoads = (3 * kTriFrags + NW - 1) / NW;

  const int slices = (a.P + W - 1) / W;
  const int64_t bh = id / slices, b = bh / a.H, h = bh % a.H, g = h / (a.H / a.G);
  const int col0 = (int)(id % slices) * W;
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_of(tid), j = lane & 15, q = lane >> 4;
  const int w = wave & 3, n = wave >> 2, row = 16 * n + j;
  const int64_t c_last = a.Nc - 1, at0 = chunk_at(a, bh, 0), at = at0 + c_last, cols = padded_cols(a.P);

  for (int i = tid; i < L::elems / 8; i += 64 * NW) reinterpret_cast<uint4*>(lds)[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  typename Keys::Offsets k_off, q_off;
  uint32_t y_off;
  constexpr int v_vecs = 2 * NG, v_rows = 64 / v_vecs, v_kb = C / v_rows;
  const int v_t = wave % v_kb;
  const bool v_in = col0 + 8 * (lane % v_vecs) < a.P;
  const int64_t y_row = a.H * a.P;
  auto offsets_q = [&](int last) { Keys::offsets(q_off, (int)a.q_stride, last, a.N, wave, lane); };
  auto offsets_ky = [&](int last) {
    Keys::offsets(k_off, (int)a.k_stride, last, a.N, wave, lane);
    y_off = (uint32_t)min(v_t * v_rows + lane / v_vecs, last) * (uint32_t)y_row * 2u + 16u * (lane % v_vecs);
  };
  const uint32_t lds0 = lds_address(lds), mine = lds0 + wave * 1024;
  const int64_t row0 = b * a.T + c_last * C;
  const bf16* kp = static_cast<const bf16*>(a.k) + row0 * a.k_stride + g * a.N;
  const bf16* qp = static_cast<const bf16*>(a.q) + row0 * a.q_stride + g * a.N;
  const bf16* yp = static_cast<const bf16*>(a.dy) + row0 * y_row + h * a.P + col0;
  const bf16* xp = a.inv_t + at * (3 * kTriFrags * kFrag) + wave * 512;
  const bf16* pp = a.qk + at * (3 * kTriFrags * kFrag) + wave * 512;
  const float* gp = a.gate + at * kGates;
  const bool all_cols = a.P - col0 >= W;
  auto request_k = [&](int half) {
    Keys::template request<FULL>(kp, k_off, mine + 2 * (L::k + half * Keys::kElems));
    request16(gp, 16 * lane, lds0 + 2 * (L::gate + half * 2 * kGates));
  };
  auto request_py = [&]() {
    request_evenly<3 * kTriFrags, NW>(pp, mine + 2 * L::p, wave, lane);
    if (all_cols || v_in) request16(yp, y_off, lds0 + 2 * L::y + v_t * 1024);
  };
  auto request_x = [&]() { request_evenly<3 * kTriFrags, NW>(xp, mine + 2 * L::x, wave, lane); };
  const int tail = (int)(a.T - c_last * C) - 1;   // last row of the last chunk
  offsets_q(tail);
  offsets_ky(tail);
  request_k(0);
  request_py();
  request_x();

  const float sign = odd_sign(j);
  const uint32_t flip = odd_flip(j);
  f32x4 st[KT];
  const int col = col0 + row;
  const bool col_in = col < a.P;
  int key[KT], put_s[KT];
#pragma unroll
  for (int t = 0; t < KT; ++t) {
    key[t] = key_of(KT * w + t, 4 * q);
    put_s[t] = L::s + row_vec<KP>(row, key[t] / 8) + key[t] % 8;
    st[t] = f32x4{0, 0, 0, 0};
    if (a.dfinal && col_in && key[t] < a.N)
      st[t] = sign * *reinterpret_cast<const f32x4*>(a.dfinal + (bh * a.P + col) * a.N + key[t]);
  }
  auto store_s = [&]() {
#pragma unroll
    for (int t = 0; t < KT; ++t) store_split4<3>(lds + put_s[t], W * KP, st[t]);
  };
  store_s();
  const bool kept = col0 + 16 * n < cols;
  float* const park = static_cast<float*>(a.park) + 4 * lane;
  float* state_at = kept ? a.leave + (at * cols + col) * KP : park;
  float* right_at = kept ? a.dright + (at * cols + col) * C + 16 * w + 4 * q : park;
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
  // dy as right operand from token `tok` on, and as a result tile
  const int dy_at = L::y + (4 * q + (j >> 2)) * W + 16 * n + 4 * (j & 3);
  // rows of tiles 0 and 1 of the triangles reach over all columns, 2 and 3 over the last 32
  const int first = w >> 1;
  landed<0>();
#pragma unroll
  for (int t = 0; t < KT; ++t) pin(st[t]);
  if (c_last > 0) offsets_ky(C - 1);

  for (int64_t c = c_last; c >= 0; --c) {
    const int half = (int)(c_last - c) & 1;
    const bf16* const lk = lds + L::k + half * Keys::kElems;
    const float* const gate = reinterpret_cast<const float*>(lds + L::gate + half * 2 * kGates) + 16 * w + 4 * q;
    auto gates = [&](int which) { return *reinterpret_cast<const f32x4*>(gate + which); };
    const float whole = load_uniform(a.whole + at0 + c);
#pragma unroll
    for (int t = 0; t < KT; ++t) *reinterpret_cast<f32x4*>(kept ? state_at + key[t] : park) = st[t];
    state_at -= cols * KP;
    Keys::template request<FULL>(qp, q_off, mine + 2 * L::q);
    if (c == c_last) offsets_q(C - 1);
    if (c > 0) {   // before the first chunk that one again, to where no one reads any more
      kp -= C * a.k_stride;
      qp -= C * a.q_stride;
      yp -= C * y_row;
      xp -= 3 * kTriFrags * kFrag;
      pp -= 3 * kTriFrags * kFrag;
      gp -= kGates;
    }
    request_k(half ^ 1);

    // dW
    {
      f32x4 ke[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}}, dw[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
      for (int s = 0; s < KS; s += 2) {
        bf16x8 kf[2];
        Frag<3> ef[2];
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          kf[o] = ld8(lk + row_at[s + o]);
          ef[o] = load_planes<3>(lds + get_s[s + o], W * KP);
        }
#pragma unroll
        for (int i = 2; i >= 0; --i)
#pragma unroll
          for (int o = 0; o < 2; ++o) ke[o] = mma(kf[o], ef[o].p[i], ke[o]);
      }
      const bf16* const lp = lds + L::p + upper_frag(w, first) * (3 * kFrag) + lane * 8;
      dw[0] = mma(load_planes<3>(lp, kFrag), with_sign(read_tr2(lds + dy_at + 32 * first * W, 16 * W), flip), dw[0]);
      if (w < 2) dw[1] = mma(load_planes<3>(lp + 3 * kFrag, kFrag), with_sign(read_tr2(lds + dy_at + 32 * W, 16 * W), flip), dw[1]);
      const f32x4 ge = gates(kEnd), go = sign * gates(kOut);
      const bf16x4 own = lds_read_tr4(lds + dy_at + 16 * w * W);
      f32x4 gy;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        dw[0][r] = fmaf(ge[r], ke[0][r] + ke[1][r], dw[0][r] + dw[1][r]);
        gy[r] = go[r] * (float)own[r];
      }
      store_split4<3>(lds + L::r + put_t, W * C, dw[0]);
      store_split4<3>(lds + L::g + put_t, W * C, gy);
    }
    landed<KT + 2 * kKeyLoads + 1>();
    request_py();
    // dR
    {
      const f32x4 gr = gates(kRight);
      const bf16* const lx = lds + L::x + upper_frag(w, first) * (3 * kFrag) + lane * 8;
      f32x4 dr = {0, 0, 0, 0}, dr2 = {0, 0, 0, 0};
      dr = mma(load_planes<3>(lx, kFrag), load_planes<3>(lds + L::r + (w < 2 ? get_t[0] : get_t[1]), W * C), dr);
      if (w < 2) dr2 = mma(load_planes<3>(lx + 3 * kFrag, kFrag), load_planes<3>(lds + L::r + get_t[1], W * C), dr2);
      dr += dr2;
      *reinterpret_cast<f32x4*>(right_at) = dr;
      if (kept) right_at -= cols * C;
      store_split4<3>(lds + L::e + put_t, W * C, -gr * dr);
    }
    landed<kKeyLoads + 1 + kTriLoads + 1 + 1>();
    request_x();
    // the gradient of the state that enters the chunk
    {
      f32x4 acc[2][KT];
#pragma unroll
      for (int of = 0; of < 2; ++of) {   // Q^T of the outputs' gradients, K^T of the right sides'
#pragma unroll
        for (int t = 0; t < KT; ++t) acc[of][t] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          Frag<1> ka[KT];
#pragma unroll
          for (int t = 0; t < KT; ++t) ka[t] = Keys::columns((of == 0 ? lds + L::q : lk) + col_at[t] + 32 * s * KP);
          mma_tiles(ka, load_planes<3>(lds + (of == 0 ? L::g : L::e) + get_t[s], W * C), acc[of]);
        }
      }
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) st[t][r] = fmaf(whole, st[t][r], acc[0][t][r] + acc[1][t][r]);
      store_s();
    }
    landed<1 + kTriLoads>();
  }
  if (a.dh0 && col_in) {
#pragma unroll
    for (int t = 0; t < KT; ++t)
      if (key[t] < a.N) *reinterpret_cast<f32x4*>(a.dh0 + (bh * a.P + col) * a.N + key[t]) = sign * st[t];
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // no request may reach LDS after this
}

// ---------------------------------------------------------------------------
// Both chains in one launch: neither needs the other, and each is a sequence of
// dependent steps that leaves a compute unit idle most of the time.  The first
// half of the workgroups takes the longer one, from the last chunk.  4096 tokens of
// 32 heads of 128 x 128: 265 us, one after the other 315.
// ---------------------------------------------------------------------------
template <typename F, typename G> __device__ __forceinline__ void both_ways(F&& back, G&& forth) {
  const unsigned half = gridDim.x / 2;
  if (blockIdx.x < half) back(xcd_remap(blockIdx.x, half));
  else forth(xcd_remap(blockIdx.x - half, half));
}
constexpr int larger(int a, int b) { return a > b ? a : b; }

template <typename IO, int KP, bool FULL>
__global__ __launch_bounds__(kThreads) void k_delta_both_chains(DeltaArgs a) {
  __shared__ __align__(16) bf16 lds[larger(BackChainLds<IO, KP, 1>::elems, ChainLds<IO, KP, 1, true>::elems)];
  both_ways([&](int64_t id) { back_chain<IO, KP, FULL, 1>(a, lds, id); },
            [&](int64_t id) { chain<IO, KP, FULL, 1, true>(a, lds, id); });
}
template <int KP, bool FULL, int NG>
__global__ __launch_bounds__(256 * NG) void k_delta_both_tokens(DeltaArgs a) {
  __shared__ __align__(1024) bf16 lds[larger(BackTokensLds<KP, NG>::elems, TokensLds<KP, NG, true>::elems)];
  both_ways([&](int64_t id) { back_tokens<KP, FULL, NG>(a, lds, id); },
            [&](int64_t id) { tokens_chain<KP, FULL, NG, true>(a, lds, id); });
}
template <int KP, bool FULL>
__global__ __launch_bounds__(256, 2) void k_delta_both_columns(DeltaArgs a) {
  __shared__ __align__(1024) bf16 lds[larger(BackLds<KP, 4>::elems, ColumnsLds<KP, 4, true>::elems)];
  both_ways([&](int64_t id) { back_columns<KP, FULL>(a, lds, id); },
            [&](int64_t id) { columns_chain<KP, FULL, true>(a, lds, id); });
}

// ---------------------------------------------------------------------------
// The gradients of one chunk of one head.  Wavefront w owns tokens 16 w .. + 15
// of every result, each formed transposed, lane (4 rows, own token): a pair's
// gradients are then the right operand of the sums over earlier tokens as they
// stand, and only those over later tokens go through LDS.  The contractions over
// the values run over slices of 32 value columns, whose operands are staged as
// planes and read transposed.  Contractions take their indices in the order
// 4 q .. + 3, 16 + 4 q .. + 3, so that eight consecutive rows are read together,
// which rows of 144 or 80 elements put into different banks.
//
// bfloat16 io: two workgroups to a compute unit (69 KB of LDS, the states that
// enter and the gradients that leave through one buffer in turn).  4096 tokens of
// 32 heads of 128 x 128: 195-215 us (one workgroup a unit, results not transposed,
// pairs through LDS both times: 323), of which vector instructions 60, matrix
// instructions 40, LDS 40 and the 426 MB it moves 90.  The gradients that leave are
// requested behind the first products' operands and not with them: those registers
// would spill (20 us).
// ---------------------------------------------------------------------------
constexpr int kSlice = 32, kPairRow = C + 16;

__device__ __forceinline__ void store4(float* to, f32x4 v) { *reinterpret_cast<f32x4*>(to) = v; }
__device__ __forceinline__ void store4(bf16* to, f32x4 v) {
  *reinterpret_cast<bf16x4*>(to) = bf16x4{(bf16)v[0], (bf16)v[1], (bf16)v[2], (bf16)v[3]};
}

template <typename IO, int KP> struct GradsLds {
  static constexpr int PI = Planes<IO>::in;
  static constexpr int KST = KP + (PI == 3 && KP == 128 ? 8 : 16);   // (float32 keys of 128: tiles would not fit)
  static constexpr int tok = 3 * kSlice * kPairRow, key = 3 * kSlice * KST;    // staged slices
  static constexpr int rows = PI * C * KST, pairs = 3 * C * kPairRow;          // k, q and the pairs
  static constexpr int first = 2 * tok + key, second = 2 * rows + pairs;
  static constexpr int elems = first > second ? first : second;
};

// rows r0 + 4 q .. + 3 and r0 + 16 + 4 q .. + 3 of column c0 + lane % 16
template <int NP, int STRIDE>
__device__ __forceinline__ Frag<NP> columns_of(const bf16* m, int plane, int r0, int c0, int lane) {
  const int j = lane & 15, q = lane >> 4;
  return read_tr<NP>(m + (r0 + 4 * q + (j >> 2)) * STRIDE + c0 + 4 * (j & 3), plane, 16 * STRIDE);
}

// four consecutive values of an LDS tile of planes
template <int NP>
__device__ __forceinline__ f32x4 plane_sum4(const bf16* p, int plane) {
  f32x4 x = {0, 0, 0, 0};
#pragma unroll
  for (int i = NP - 1; i >= 0; --i) {
    const bf16x4 v = *reinterpret_cast<const bf16x4*>(p + i * plane);
#pragma unroll
    for (int r = 0; r < 4; ++r) x[r] += (float)v[r];
  }
  return x;
}

// value columns 4 q .. + 3 and 16 + 4 q .. + 3 of a row's slice, zeros where there are none
template <typename IO> struct Values8 {
  float x[8];
  __device__ __forceinline__ void load(const IO* p, bool lo, bool hi) {
    using V = std::conditional_t<sizeof(IO) == 2, bf16x4, f32x4>;
    const V a = *reinterpret_cast<const V*>(p), b = *reinterpret_cast<const V*>(hi ? p + 16 : p);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      x[r] = lo ? (float)a[r] : 0.0f;
      x[4 + r] = hi ? (float)b[r] : 0.0f;
    }
  }
};

__device__ __forceinline__ float sum_q(float v) {   // over the lanes of a token
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

template <typename IO, int KP, bool FULL>
__global__ __launch_bounds__(kThreads, sizeof(IO) == 2 ? 2 : 1) void k_delta_grads(DeltaArgs a) {
  using L = GradsLds<IO, KP>;
  constexpr int PI = L::PI, KST = L::KST, KT = KP / 16;
  constexpr int kTokParts = kSlice * C / 4 / kThreads, kKeyParts = kSlice * KP / 4 / kThreads;
  __shared__ __align__(16) bf16 lds[L::elems];
  __shared__ float4 s_row[C];
  __shared__ float s_b[C], s_from[C], s_to[C], s_beta[C], s_sum[kThreads / 64];
  __shared__ __align__(16) float s_over[kThreads / 64][C];
  bf16 *const s_w = lds, *const s_d = lds + L::tok, *const s_s = lds + 2 * L::tok;
  bf16 *const s_k = lds, *const s_q = lds + L::rows, *const s_p = lds + 2 * L::rows;

  const auto [b, c, h, g] = chunk_head(a);
  const int64_t bh = b * a.H + h, at = chunk_at(a, bh, c);
  const int64_t t0 = c * C, row0 = b * a.T + t0, left = a.T - t0;
  const int tid = threadIdx.x, lane = tid & 63, w = wave_of(tid), j = lane & 15, q = lane >> 4;
  const int own = 16 * w + j;
  // odd tokens negated, until the decays are applied; odd value columns of what the
  // chains left back to their signs
  static_assert(kThreads / (C / 4) % 2 == 0 && kThreads / (KP / 4) % 2 == 0, "a thread's columns are all odd or all even");
  const float sign = odd_sign(own), sign_t = odd_sign(tid / (C / 4)), sign_k = odd_sign(tid / (KP / 4));
  if (tid < C) {
    s_b[tid] = a.gate[at * kGates + kBeta + tid];
    s_row[tid] = a.row[at * C + tid];
  }

  f32x4 dp[4], dl[4], dq[KT], z[KT], x[KT];
#pragma unroll
  for (int i = 0; i < 4; ++i) dp[i] = dl[i] = f32x4{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < KT; ++i) dq[i] = z[i] = x[i] = f32x4{0, 0, 0, 0};
  const bool row_in = own < left;
  const int64_t my_row = row0 + (row_in ? own : 0);
  const int64_t cols = padded_cols(a.P);
  float es = 0.0f, dr_v = 0.0f;

  for (int p0 = 0; p0 < a.P; p0 += kSlice) {
    f32x4 vw[kTokParts], vd[kTokParts], vs[kKeyParts];
#pragma unroll
    for (int i = 0; i < kTokParts; ++i) {
      const int at4 = tid + i * kThreads, p = at4 / (C / 4), t = at4 % (C / 4) * 4;
      const bool in = p0 + p < a.P;
      const int64_t o = (at * cols + (in ? p0 + p : 0)) * C + t;
      vw[i] = *reinterpret_cast<const f32x4*>(a.write + o) * f32x4{1.0f, -1.0f, 1.0f, -1.0f};
      vd[i] = *reinterpret_cast<const f32x4*>(a.dright + o) * f32x4{sign_t, -sign_t, sign_t, -sign_t};
      if (!in) vw[i] = vd[i] = f32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int i = 0; i < kKeyParts; ++i) {
      const int at4 = tid + i * kThreads, p = at4 / (KP / 4), key = at4 % (KP / 4) * 4;
      const bool in = p0 + p < a.P && key < a.N;
      const int64_t o = (at * cols + (in ? p0 + p : 0)) * KP + (in ? key : 0);
      vs[i] = *reinterpret_cast<const f32x4*>(a.enter + o);
      if (!in) vs[i] = f32x4{0, 0, 0, 0};
    }
    // P is a multiple of 8
    const bool lo_in = row_in && p0 + 4 * q < a.P, hi_in = row_in && p0 + 16 + 4 * q < a.P;
    const int64_t pc = h * a.P + (lo_in ? p0 + 4 * q : 0);
    Values8<IO> dy, v;
    dy.load(static_cast<const IO*>(a.dy) + my_row * (a.H * a.P) + pc, lo_in, hi_in);
    v.load(static_cast<const IO*>(a.v) + my_row * a.v_stride + pc, lo_in, hi_in);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kTokParts; ++i) {
      const int at4 = tid + i * kThreads, o = at4 / (C / 4) * kPairRow + at4 % (C / 4) * 4;
      store_split4<3>(&s_w[o], kSlice * kPairRow, vw[i]);
      store_split4<3>(&s_d[o], kSlice * kPairRow, vd[i]);
    }
#pragma unroll
    for (int i = 0; i < kKeyParts; ++i) {
      const int at4 = tid + i * kThreads, o = at4 / (KP / 4) * KST + at4 % (KP / 4) * 4;
      store_split4<3>(&s_s[o], kSlice * KST, vs[i]);
    }
    __syncthreads();
    f32x4 ve[kKeyParts];
#pragma unroll
    for (int i = 0; i < kKeyParts; ++i) {
      const int at4 = tid + i * kThreads, p = at4 / (KP / 4), key = at4 % (KP / 4) * 4;
      const bool in = p0 + p < a.P && key < a.N;
      const int64_t o = (at * cols + (in ? p0 + p : 0)) * KP + (in ? key : 0);
      ve[i] = *reinterpret_cast<const f32x4*>(a.leave + o);
      if (!in) ve[i] = f32x4{0, 0, 0, 0};
    }
    const auto dyf = with_sign(split8<PI>(dy.x), odd_flip(own));
    const auto drf = columns_of<3, kPairRow>(s_d, kSlice * kPairRow, 0, 16 * w, lane);
    const auto wf = columns_of<3, kPairRow>(s_w, kSlice * kPairRow, 0, 16 * w, lane);
    {
      const float beta = sign * s_b[own];
      float out[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = ((float)drf.p[2][e] + (float)drf.p[1][e]) + (float)drf.p[0][e];
        dr_v = fmaf(d, v.x[e], dr_v);
        out[e] = beta * d;
      }
      IO* const to = static_cast<IO*>(a.dv) + my_row * a.dv_stride + pc;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        if (!(n ? hi_in : lo_in)) continue;
        const float* o = out + 4 * n;
        store4(to + 16 * n, f32x4{o[0], o[1], o[2], o[3]});
      }
    }
#pragma unroll
    for (int j0 = 0; j0 < 4; j0 += 2) {
      if (j0 > w) continue;
      Frag<3> wb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) wb[i] = columns_of<3, kPairRow>(s_w, kSlice * kPairRow, 0, 16 * (j0 + i), lane);
      mma_tiles(wb, dyf, dp + j0);
      mma_tiles(wb, drf, dl + j0);
    }
#pragma unroll
    for (int k0 = 0; k0 < KT; k0 += 2) {
      Frag<3> sb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) sb[i] = columns_of<3, KST>(s_s, kSlice * KST, 0, 16 * (k0 + i), lane);
      mma_tiles(sb, dyf, dq + k0);
      mma_tiles(sb, drf, z + k0);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kKeyParts; ++i) {
      const int at4 = tid + i * kThreads, o = at4 / (KP / 4) * KST + at4 % (KP / 4) * 4;
      const f32x4 e = sign_k * ve[i], own_s = plane_sum4<3>(&s_s[o], kSlice * KST);   // what this thread put there
#pragma unroll
      for (int r = 0; r < 4; ++r) es = fmaf(own_s[r], e[r], es);
      store_split4<3>(&s_s[o], kSlice * KST, e);
    }
    __syncthreads();
#pragma unroll
    for (int k0 = 0; k0 < KT; k0 += 2) {
      Frag<3> eb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) eb[i] = columns_of<3, KST>(s_s, kSlice * KST, 0, 16 * (k0 + i), lane);
      mma_tiles(eb, wf, x + k0);
    }
  }
  {
    const int64_t row = row0 + (row_in ? own : left - 1), at = g * a.N + 8 * q;
    KeyRow<IO, KP, FULL> kr, qr;
    kr.load(static_cast<const IO*>(a.k) + row * a.k_stride + at, a.N, q);
    qr.load(static_cast<const IO*>(a.q) + row * a.q_stride + at, a.N, q);
    __syncthreads();
#pragma unroll
    for (int s = 0; s < KP / 32; ++s) {
      const auto kf = kr.frag(s, a.N, q);
      const auto qf = qr.frag(s, a.N, q);
#pragma unroll
      for (int i = 0; i < PI; ++i) {
        const int o = i * C * KST + own * KST + 32 * s + 8 * q;
        *reinterpret_cast<bf16x8*>(&s_k[o]) = kf.p[i];
        *reinterpret_cast<bf16x8*>(&s_q[o]) = qf.p[i];
      }
    }
  }
  __syncthreads();

  // the pairs (own token i, earlier token) over their decay; times 1/|k| of the
  // earlier one they are the right operands of the sums over it
  const float4 rec = s_row[own], last = s_row[C - 1];
  const float beta = s_b[own];
  const float gamma = sign * exp2_of(rec.z + rec.w), eta = sign * exp2_of((last.z - rec.z) + (last.w - rec.w));
  f32x4 rk[4];
#pragma unroll
  for (int jt = 0; jt < 4; ++jt)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int cj = 16 * jt + 4 * q + r;
      const float4 rj = s_row[cj];
      const float dec = sign * odd_sign(r) * exp2_of((rec.z - rj.z) + (rec.w - rj.w));   // W's rows are cj, odd as r
      dp[jt][r] = own >= cj ? dec * dp[jt][r] : 0.0f;
      dl[jt][r] = own > cj ? dec * dl[jt][r] : 0.0f;
      rk[jt][r] = rj.x;
    }
  // What a decay's gradient is a sum of, for token t: pairs with t between them
  // (below), what later tokens read of the entering state (from), what earlier
  // ones wrote that reaches the end (to), and the state that passes through.  No
  // term is in the sum and taken out again, which keeps float32's rounding at that
  // of the result (differences of row and column sums: five times as much).
  float from = 0.0f, to = 0.0f, kz = 0.0f;
#pragma unroll
  for (int kt = 0; kt < KT; ++kt) {
    dq[kt] *= gamma;
    z[kt] *= gamma;
    x[kt] *= eta;
    const int o = own * KST + 16 * kt + 4 * q;
    const f32x4 k = plane_sum4<PI>(&s_k[o], C * KST), u = plane_sum4<PI>(&s_q[o], C * KST);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      from = fmaf(u[r], dq[kt][r], from);
      kz = fmaf(k[r], z[kt][r], kz);
      to = fmaf(k[r], x[kt][r], to);
    }
  }
  kz = rec.x * sum_q(kz);
  from = rec.y * sum_q(from) - beta * kz;
  to = rec.x * sum_q(to);
  {
    float before = 0.0f, pair_kz = 0.0f;   // the pairs (own, j) with j in earlier tiles
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) {
      if (jt > w) continue;
      f32x4 kk = {0, 0, 0, 0}, qk = {0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < KP / 32; ++s) {
        const auto ka = load_planes<PI>(&s_k[(16 * jt + j) * KST + 32 * s + 8 * q], C * KST);
        kk = mma(ka, load_planes<PI>(&s_k[own * KST + 32 * s + 8 * q], C * KST), kk);
        qk = mma(ka, load_planes<PI>(&s_q[own * KST + 32 * s + 8 * q], C * KST), qk);
      }
      float sum = 0.0f, up[4];   // over the lane's pairs, up to each
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float lk = rec.x * dl[jt][r] * rk[jt][r] * kk[r];
        pair_kz += lk;
        up[r] = sum;
        sum += fmaf(rec.y * dp[jt][r] * rk[jt][r], qk[r], -beta * lk);
      }
      float upto = sum;          // over the lanes of the token, up to this one
      float o = __shfl_up(upto, 16, 64);
      upto += q >= 1 ? o : 0.0f;
      o = __shfl_up(upto, 32, 64);
      upto += q >= 2 ? o : 0.0f;
      o = __shfl_up(upto, 16, 64);
      const float base = before + (q >= 1 ? o : 0.0f);
      f32x4 over;
#pragma unroll
      for (int r = 0; r < 4; ++r) over[r] = sum_of_16(own >= 16 * jt + 4 * q + r ? base + up[r] : 0.0f);
      if (j == 0) *reinterpret_cast<f32x4*>(&s_over[w][16 * jt + 4 * q]) = over;
      before += __shfl(upto, 48 + j, 64);
    }
    dr_v = sign * sum_q(dr_v) - kz - sum_q(pair_kz);
    if (q == 0) {
      s_from[own] = from;
      s_to[own] = to;
      s_beta[own] = dr_v;
    }
  }
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    if (s > (w >> 1)) continue;
    const auto pf = right_of<3>(dp[2 * s] * rk[2 * s], dp[2 * s + 1] * rk[2 * s + 1]);
    const auto lf = right_of<3>(dl[2 * s] * rk[2 * s], dl[2 * s + 1] * rk[2 * s + 1]);
#pragma unroll
    for (int k0 = 0; k0 < KT; k0 += 2) {
      Frag<PI> kb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) kb[i] = columns_of<PI, KST>(s_k, C * KST, 32 * s, 16 * (k0 + i), lane);
      mma_tiles(kb, pf, dq + k0);
      mma_tiles(kb, lf, z + k0);
    }
  }
  // the sums over later tokens: pairs [i][j], tiles that a reader of 32 rows meets
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
    const float f = pass ? -beta * rec.x : rec.y;
    if (pass) __syncthreads();
#pragma unroll
    for (int jt = 0; jt < 4; ++jt)
      if (jt <= (w | 1)) store_split4<3>(&s_p[own * kPairRow + 16 * jt + 4 * q], C * kPairRow, (pass ? dl : dp)[jt] * f);
    __syncthreads();
    const bf16* const m = pass ? s_k : s_q;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (s < (w >> 1)) continue;
      const auto pf = columns_of<3, kPairRow>(s_p, C * kPairRow, 32 * s, 16 * w, lane);
#pragma unroll
      for (int k0 = 0; k0 < KT; k0 += 4) {
        Frag<PI> mb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) mb[i] = columns_of<PI, KST>(m, C * KST, 32 * s, 16 * (k0 + i), lane);
        mma_tiles(mb, pf, x + k0);
      }
    }
  }

  // the gradients of unit keys and scaled unit queries: of the only head of its
  // group through the normalisation here, else to be summed over the heads first
  // (k_delta_unit_grads: 2 x 515 tokens of 24 heads in float32 15 us more)
  if (a.H == a.G) {
    float uu = 0.0f, ud = 0.0f, kk = 0.0f, kd = 0.0f;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      const int o = own * KST + 16 * kt + 4 * q;
      const f32x4 k = plane_sum4<PI>(&s_k[o], C * KST), u = plane_sum4<PI>(&s_q[o], C * KST);
      x[kt] -= beta * z[kt];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        uu = fmaf(u[r], u[r], uu);
        ud = fmaf(u[r], dq[kt][r], ud);
        kk = fmaf(k[r], k[r], kk);
        kd = fmaf(k[r], x[kt][r], kd);
      }
    }
    const float ru = 1.0f / sqrtf(sum_q(uu) + a.norm_eps), rk2 = rec.x * rec.x;
    const float tu = a.unit ? ru * sum_q(ud) * ru : 0.0f, tk = a.unit ? rk2 * sum_q(kd) : 0.0f;
    int own_row = own;   // my_row formed again: kept over the slices it would spill
    asm("" : "+v"(own_row));
    const int64_t row = row0 + (own_row < left ? own_row : 0);
    IO* const to_q = static_cast<IO*>(a.dq) + row * a.dq_stride + g * a.N;
    IO* const to_k = static_cast<IO*>(a.dk) + row * a.dk_stride + g * a.N;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      const int key = 16 * kt + 4 * q, o = own * KST + key;
      const f32x4 k = plane_sum4<PI>(&s_k[o], C * KST), u = plane_sum4<PI>(&s_q[o], C * KST);
      f32x4 du, dk;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        du[r] = rec.y * fmaf(-u[r], tu, dq[kt][r]);
        dk[r] = rec.x * fmaf(-k[r], tk, x[kt][r]);
      }
      if (row_in && key < a.N) {
        store4(to_q + key, du);
        store4(to_k + key, dk);
      }
    }
  } else {
    const int64_t out = ((row0 + own) * a.H + h) * a.N;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      const int key = 16 * kt + 4 * q;
      if (row_in && key < a.N) {
        *reinterpret_cast<f32x4*>(a.part_q + out + key) = dq[kt];
        *reinterpret_cast<f32x4*>(a.part_k + out + key) = x[kt] - beta * z[kt];
      }
    }
  }
  es = wave_sum64(es);
  if (lane == 0) s_sum[w] = es;
  __syncthreads();
  if (w != 0) return;

  // token `lane`: its decay and write strength
  float from_on = s_from[lane], to_before = s_to[lane];
  for (int off = 1; off < 64; off <<= 1) {
    const float later = __shfl_down(from_on, off, 64), earlier = __shfl_up(to_before, off, 64);
    from_on += lane + off < 64 ? later : 0.0f;
    to_before += lane >= off ? earlier : 0.0f;
  }
  to_before = __shfl_up(to_before, 1, 64);
  float dg = lane > 0 ? to_before : 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) dg += i >= lane / 16 ? s_over[i][lane] : 0.0f;
  dg += from_on + a.whole[at] * ((s_sum[0] + s_sum[1]) + (s_sum[2] + s_sum[3]));
  const bool in = lane < left;
  const int64_t th = (row0 + (in ? lane : 0)) * a.H + h;
  const float zt = a.dt[th] + (a.dt_bias ? a.dt_bias[h] : 0.0f);
  const float pre = a.softplus ? softplus_of(zt) : zt;   // as in delta_of: the same clip decision
  const float rate = rate_of(a, zt);
  float slope = pre < a.dt_min || pre > a.dt_max ? 0.0f : a.A[h];   // a NaN is not clipped
  if (a.softplus) slope *= sigmoid_of(zt);
  const float ddt = in ? dg * slope : 0.0f;
  // an infinite rate forgets all: dg is 0, and so is what A's gradient has of it (x e^-x at infinity)
  const float sum_a = wave_sum64(in && dg != 0.0f ? dg * rate : 0.0f), sum_b = wave_sum64(ddt);
  if (in) {
    // the logistic's slope as a product: 1 - b would cancel where b is close to 1
    const float zb = a.beta[th];
    a.ddt[th] = ddt;
    a.dbeta[th] = s_beta[lane] * (a.sigmoid ? sigmoid_of(zb) * sigmoid_of(-zb) : 1.0f);
  }
  if (lane == 0) {
    a.part_h[2 * at] = sum_a;
    a.part_h[2 * at + 1] = sum_b;
  }
}

// Gradients of a token's keys or queries of one group from those of the unit
// vectors of its heads: NL lanes of four keys a row.  Bound by memory: 4096 tokens
// of 32 heads of 128 in pairs 46 us, 4.4 TB/s.
template <typename IO, int NL>
__global__ __launch_bounds__(kThreads) void k_delta_unit_grads(DeltaArgs a) {
  // rows up to 2^27 - 8 (checked by the caller: a grid's threads count in 32 bits):
  // divisions of 32 bits (64-bit ones cost a fifth)
  const uint32_t id = (uint32_t)(((int64_t)blockIdx.x * kThreads + threadIdx.x) / NL);
  const uint32_t rows = (uint32_t)(a.Bt * a.T * a.G);
  const bool in = id < 2 * rows;
  const bool is_q = id < rows;
  const uint32_t row = in ? (is_q ? id : id - rows) : 0, G = (uint32_t)a.G;
  const int64_t tok = row / G, g = row % G, per = (uint32_t)a.H / G;
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
    store4(to, d);
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

hipError_t launch_grads(const DeltaArgs& a, bool io_bf16, hipStream_t stream) {
  return with_keys(a.N, io_bf16, [&](auto io, auto kp, auto full) {
    using IO = decltype(io);
    constexpr int KP = decltype(kp)::value;
    constexpr bool FULL = decltype(full)::value;
    const unsigned chunks = (unsigned)(a.Bt * a.H * a.Nc);
    hipError_t e;   // nothing is launched behind a launch that failed
    if constexpr (sizeof(IO) == 2) {
      e = chain_of(
          a, 2,
          [&](auto ng, unsigned groups) {
            hipLaunchKernelGGL((k_delta_both_tokens<KP, FULL, ng.value>), dim3(groups), dim3(256 * ng.value), 0, stream,
                               a);
          },
          [&](unsigned groups) {
            hipLaunchKernelGGL((k_delta_both_columns<KP, FULL>), dim3(groups), dim3(256), 0, stream, a);
          });
    } else {
      hipLaunchKernelGGL((k_delta_both_chains<IO, KP, FULL>), dim3((unsigned)(2 * a.Bt * a.H * ((a.P + 15) / 16))),
                         dim3(kThreads), 0, stream, a);
      e = hipGetLastError();
    }
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_delta_grads<IO, KP, FULL>), dim3(chunks), dim3(kThreads), 0, stream, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (a.H != a.G) {
      constexpr int per = kThreads / (KP / 4);
      const int64_t rows = 2 * a.Bt * a.T * a.G;
      hipLaunchKernelGGL((k_delta_unit_grads<IO, KP / 4>), dim3((unsigned)((rows + per - 1) / per)), dim3(kThreads),
                         0, stream, a);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    hipLaunchKernelGGL(k_delta_head_grads, dim3((unsigned)a.H), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
  });
}

}  // namespace
}  // namespace delta

hipError_t launch_delta_scan_backward(const DeltaArgs& a, bool io_bf16, hipStream_t stream) {
  const hipError_t e = launch_delta_matrices(a, io_bf16, stream);
  return e != hipSuccess ? e : delta::launch_grads(a, io_bf16, stream);
}

}  // namespace ssd
