// The chains of the gated delta rule: what a workgroup does for value columns of
// one head, chunk after chunk.  The scan's kernels run them by themselves, the
// gradients' next to the chains from the other end (ssd_delta_backward.hip).
#pragma once

#include "ssd_delta.h"

namespace ssd {
namespace delta {
namespace {

// ---------------------------------------------------------------------------
// The chunks of one (b, h) in order, 16 NT value columns, float32 io (keys and
// queries are three planes there, and every product with them six).  Bound by a
// step's chain of LDS, matrix instructions and barriers: 3 x 1001 tokens of 24
// heads of 64 x 64, 288 workgroups, 73 us (two to a compute unit, as keys are
// written to LDS behind their first products and not a chunk ahead: 96 before).
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
template <typename IO, int KP, int NT, bool KEEP> struct ChainLds {
  static constexpr int PI = Planes<IO>::in, W = 16 * NT;
  static constexpr int k = 0, s = k + PI * C * (KP + 16), r = s + 3 * W * (KP + 8);
  static constexpr int e = r + 3 * W * kTokStride, w = e + 3 * W * kTokStride;
  static constexpr int elems = w + (KEEP ? 0 : 3 * W * kTokStride);
};

template <typename IO, int KP, bool FULL, int NT, bool KEEP>
__device__ __forceinline__ void chain(const DeltaArgs& a, bf16* lds, int64_t id) {
  using L = ChainLds<IO, KP, NT, KEEP>;
  constexpr int PI = Planes<IO>::in;
  constexpr int KS = KP / 32, KST = KP + 8, KTR = KP + 16, KT = KP / 64, W = 16 * NT;
  bf16 *const s_k = lds + L::k, *const s_s = lds + L::s;
  bf16* const s_r = lds + L::r;   // right sides
  bf16* const s_e = lds + L::e;   // writes, decayed to the chunk's end
  bf16* const s_w = lds + L::w;   // writes

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
  const bf16* pp = a.qk + (at0 * kTriFrags + lower_frag(w, 0)) * (3 * kFrag) + lane * 8;
  const float* ep = a.whole + at0;
  const int64_t y_row = a.H * a.P;
  IO* yp = KEEP ? nullptr : static_cast<IO*>(a.y) + (b * a.T + 16 * w + 4 * q) * y_row + h * a.P;
  IO* const park = static_cast<IO*>(a.park) + lane;
  const int64_t cols = padded_cols(a.P);
  float* state_at = KEEP ? a.enter + (at0 * cols + col0 + j) * KP + key0 : nullptr;
  float* write_at = KEEP ? a.write + (at0 * cols + col0 + j) * C + 16 * w + 4 * q : nullptr;

  KeyRow<IO, KP, FULL> kr, qr;
  Frag<3> xf[2], pf[2];
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
    pf[0] = load_planes<3>(pp, kFrag);
    pf[1] = load_planes<3>(pp + second * (3 * kFrag), kFrag);
  };
  bf16* const put_k = &s_k[(16 * w + j) * KTR + 8 * q];
  rows_of(0);
  load_rows();
  load_x();
  if constexpr (!KEEP) load_p();
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
    // K S^T and Q S^T of the wavefront's tokens; the right sides b (v - gamma K S^T);
    // the keys to LDS, where they are next read two barriers on
    f32x4 y[NT], ks[NT], qs[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) ks[n] = qs[n] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const auto kf = kr.frag(s, a.N, q);
#pragma unroll
      for (int i = 0; i < PI; ++i) *reinterpret_cast<bf16x8*>(put_k + i * C * KTR + 32 * s) = kf.p[i];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const auto sf = load_planes<3>(get_s + 16 * n * KST + 32 * s, W * KST);
        ks[n] = mma(kf, sf, ks[n]);
        if constexpr (!KEEP) qs[n] = mma(qr.frag(s, a.N, q), sf, qs[n]);
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      f32x4 rs;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        rs[r] = fmaf(-g_right[r], ks[n][r], g_beta[r] * to_f32(v[n][r]));
        if constexpr (!KEEP) y[n][r] = g_out[r] * qs[n][r];
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
      if constexpr (!KEEP) store_split4<3>(s_w + put_t + 16 * n * kTokStride, W * kTokStride, ws);
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
      for (int s = 0; s < 2; ++s) ka[s] = read_tr<PI>(get_k + 32 * s * KTR + 16 * t, C * KTR, 16 * KTR);
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
    // outputs
    if constexpr (!KEEP) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        y[n] = mma(pf[0], load_planes<3>(s_w + get_t + 16 * n * kTokStride, W * kTokStride), y[n]);
        if (w >= 2) y[n] = mma(pf[1], load_planes<3>(s_w + get_t + 16 * n * kTokStride + 32, W * kTokStride), y[n]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          IO* const to = 16 * w + 4 * q + r < left && col_in[n] ? yp + r * y_row + col[n] : park;
          *to = to_io<IO>(y[n][r]);
        }
      }
      yp += C * y_row;
      pp += next * (kTriFrags * 3 * kFrag);
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
// workgroup computes while another waits for its chunk (8 x 16384 tokens of 64
// heads of 64 x 128: 2100 us; one workgroup a unit that requests a chunk ahead
// takes a quarter more).  A chunk takes a wavefront 216 matrix instructions (keys of
// 128), 3456 cycles, and about as many cycles of its 800 vector instructions, most
// of them to split float32 into planes; that is what bounds it (the same chunk
// again and again, from the L2: an eighth less).
// ---------------------------------------------------------------------------
template <int KP, int NW, bool KEEP> struct ColumnsLds {
  using Keys = KeyTile<KP, NW>;
  static constexpr int k = 0, q = k + Keys::kElems, x = q + (KEEP ? 0 : Keys::kElems);
  static constexpr int p = x + 3 * kTriFrags * kFrag, v = p + (KEEP ? 0 : 3 * kTriFrags * kFrag);
  static constexpr int gate = v + C * 16 * NW, elems = gate + 2 * kGates;
};

template <int KP, bool FULL, bool KEEP>
__device__ __forceinline__ void columns_chain(const DeltaArgs& a, bf16* lds, int64_t id) {
  constexpr int NW = 4, KS = KP / 32, KT = KP / 16, W = 16 * NW;
  using L = ColumnsLds<KP, NW, KEEP>;
  using Keys = KeyTile<KP, NW>;
  using Cols = ColumnTile<NW>;

  const int slices = (a.P + W - 1) / W;
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
  const bf16* pp = a.qk + at0 * (3 * kTriFrags * kFrag) + w * 512;
  const float* gp = a.gate + at0 * kGates + w * 256;
  const bool all_cols = a.P - col0 >= W;
  auto request = [&]() {
    Keys::template request<FULL>(kp, k_off, lds0 + 2 * L::k);
    if constexpr (!KEEP) Keys::template request<FULL>(qp, q_off, lds0 + 2 * L::q);
    request_linear<3 * kTriFrags, NW>(xp, lds0 + 2 * L::x, w, lane);
    if constexpr (!KEEP) request_linear<3 * kTriFrags, NW>(pp, lds0 + 2 * L::p, w, lane);
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
#pragma unroll
        for (int i = 0; i < 4; ++i) rows[i] = load_planes<1>(lds + L::q + row_at[s] + 16 * i * KP, 0);
        mma_tiles(rows, sf, qs);
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
      Frag<3> wf[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) wf[s] = right_of<3>(ws[2 * s], ws[2 * s + 1]);
      bf16* const out = lds + L::v + 16 * w;
#pragma unroll
      for (int i = 0; i < 4; ++i) qs[i] *= gates(kOut, i);
      mma_lower<3>(lds + L::p + lane * 8, wf, qs);
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
      pp += 3 * kTriFrags * kFrag;
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
// writes go through LDS as in chain; what comes from memory lands in LDS
// as in columns_chain, each operand requested when its last reader is done:
//   top        q k^T of this chunk; k, gates of the next (two places for each)
//   barrier 1  q, v of the next            (waits for the inverse)
//   barrier 2  the next inverse            (waits for q k^T)
//   barrier 3                              (waits for k, gates, q, v)
// Every wavefront makes the same requests, so that the counts that the waits
// leave outstanding are constants.
//
// Bound by the step's length: 4096 tokens of 80 heads of 64 x 128 190 us, 3.0 us a
// chunk in pairs, of which the requests account for a fifth; the rest is three
// products that wait for each other through LDS.
// ---------------------------------------------------------------------------
template <int KP, int NG, bool KEEP> struct TokensLds {
  using Keys = KeyTile<KP, 4 * NG>;
  static constexpr int W = 16 * NG;
  static constexpr int k = 0, q = k + 2 * Keys::kElems, x = q + (KEEP ? 0 : Keys::kElems);
  static constexpr int p = x + 3 * kTriFrags * kFrag, v = p + (KEEP ? 0 : 3 * kTriFrags * kFrag);
  static constexpr int gate = v + C * W, s = gate + 4 * kGates, r = s + 3 * W * KP;
  static constexpr int e = r + 3 * W * C, wr = e + 3 * W * C;
  static constexpr int y = wr + (KEEP ? 0 : 3 * W * C), elems = y + (KEEP ? 0 : C * W);
};

template <int KP, bool FULL, int NG, bool KEEP>
__device__ __forceinline__ void tokens_chain(const DeltaArgs& a, bf16* lds, int64_t id) {
  using L = TokensLds<KP, NG, KEEP>;
  using Keys = typename L::Keys;
  constexpr int KS = KP / 32, KT = KP / 64, W = L::W, NW = 4 * NG;
  constexpr int kKeyLoads = Keys::kLoads, kTriLoads = (3 * kTriFrags + NW - 1) / NW;

  const int slices = (a.P + W - 1) / W;
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
  const bf16* pp = a.qk + at0 * (3 * kTriFrags * kFrag) + wave * 512;
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
      request_evenly<3 * kTriFrags, NW>(pp, mine + 2 * L::p, wave, lane);
      pp += 3 * kTriFrags * kFrag;
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
    landed<KEEP ? KT + kKeyLoads + 1 : 1 + kTriLoads + kKeyLoads + 1>();
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
        store_split4<3>(lds + L::wr + put_t, W * C, ws);
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
      const bf16* const lp = lds + L::p + lower_frag(w, 0) * (3 * kFrag) + lane * 8;
      f32x4 y2 = {0, 0, 0, 0};
      y = mma(load_planes<3>(lp, kFrag), load_planes<3>(lds + L::wr + get_t[0], W * C), y);
      if (w >= 2) y2 = mma(load_planes<3>(lp + 3 * kFrag, kFrag), load_planes<3>(lds + L::wr + get_t[1], W * C), y2);
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
    landed<KEEP ? 1 + kTriLoads : kTriLoads + 1>();
  }
  if (!KEEP && a.state && col_in) {
#pragma unroll
    for (int t = 0; t < KT; ++t)
      if (key[t] < a.N) *reinterpret_cast<f32x4*>(a.state + (bh * a.P + col) * a.N + key[t]) = st[t];
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // no request may reach LDS after this
}

}  // namespace
}  // namespace delta
}  // namespace ssd
