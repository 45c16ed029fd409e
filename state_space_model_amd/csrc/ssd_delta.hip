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
// state, in parallel; a chain (ssd_delta_chains.h) walks the chunks of one head
// and a slice of its value columns in order, the state in matrix-core
// accumulators.  64 tokens: the work on states falls with the chunk's length, that
// on pairs and the inverse grows with it, and a chunk of 128 would not leave its
// matrices room in LDS.
#include "ssd_delta_chains.h"

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
// The inverse X of 1 + L: the diagonal 8 x 8 blocks by back substitution, a
// lane a row (X (1 + L) = 1: x_c = [c = row] - sum_{m > c} x_m L_mc); what is
// left of them, first within blocks of 16, then by blocks of 16, nearest first,
// from X_ij = -(sum_{j < m <= i} X_im L_mj) X_jj on the float32 matrix core,
// transposed.  (16 x 16 blocks by substitution: a hundred dependent instructions
// more a wavefront.)
//
// GRADS: for the gradients, whose chain from the last chunk needs both matrices
// transposed and no output.
//
// Bound by its instructions and, with few heads to a key, by what it stores: 8 x
// 16384 tokens of 64 heads in bfloat16 1540 us (3.6 TB/s), 4096 tokens of 80 heads
// with keys of their own 68 us (5.3 TB/s).  bfloat16 takes 96 registers, five
// workgroups to a compute unit (held to the 80 of six it spills and takes a fifth
// more); float32's planes need more.
template <typename IO, int KP, bool FULL, bool GRADS>
__global__ __launch_bounds__(kThreads, sizeof(IO) == 2 ? 4 : 2) void k_delta_prep(DeltaArgs a) {
  constexpr int PI = Planes<IO>::in;
  constexpr int KS = KP / 32, KST = KP + 8, kDiag = 20;
  constexpr int k_bytes = PI * C * KST * 2, l_bytes = (GRADS ? 2 : 1) * C * kPairStride * 4;
  // the keys, then L transposed ([column][row]), then for GRADS both results: a
  // workgroup in 24 KB (bfloat16), and five of them to a compute unit hide one
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
    const float d = rate_of(a, a.dt[th] + bias);
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
      if (s <= (w >> 1)) store_frag(a.qk, at, lower_frag(w, s), lane, right_of<3>(p[2 * s], p[2 * s + 1]));
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
// One token.  A row p of the state needs two dot products, S k and S q; the
// token's own part of y is its write times k.q.
//   y = a S.q + u k.q,  S' = a S + u k,  u = b (v - a S.k)
// NL lanes of four keys share a row; N / 4 of them have keys.  Bound by memory:
// 64 sequences of 80 heads of 64 x 128 55 us, 6.1 TB/s of states read and written
// (the token's loads behind the state's, and lane sums through LDS: 79); one
// sequence 4.1 us, a launch.  Two rows a lane: four take 56 and 4.4, eight 56 and
// 5.0.
// ---------------------------------------------------------------------------
// sum over aligned groups of NL lanes, 16 or 32
template <int NL> __device__ __forceinline__ float lanes_sum(float v) {
  v = sum_of_16(v);
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
  const float d = rate_of(a, a.dt[bh] + bias);
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

template <typename IO, int KP, bool FULL>
__global__ __launch_bounds__(kThreads) void k_delta_chain(DeltaArgs a) {
  __shared__ __align__(16) bf16 lds[ChainLds<IO, KP, 1, false>::elems];
  chain<IO, KP, FULL, 1, false>(a, lds, xcd_remap(blockIdx.x, gridDim.x));
}
template <int KP, bool FULL, int NG>
__global__ __launch_bounds__(256 * NG) void k_delta_tokens(DeltaArgs a) {
  __shared__ __align__(1024) bf16 lds[TokensLds<KP, NG, false>::elems];
  tokens_chain<KP, FULL, NG, false>(a, lds, xcd_remap(blockIdx.x, gridDim.x));
}
template <int KP, bool FULL>
__global__ __launch_bounds__(256, 2) void k_delta_columns(DeltaArgs a) {
  __shared__ __align__(1024) bf16 lds[ColumnsLds<KP, 4, false>::elems];
  columns_chain<KP, FULL, false>(a, lds, xcd_remap(blockIdx.x, gridDim.x));
}

// GRADS: what the gradients' chains need of a chunk, and no chain.  Nothing is
// launched behind a launch that failed: it would read what that one did not write.
template <bool GRADS>
hipError_t launch_scan(const DeltaArgs& a, bool io_bf16, hipStream_t stream) {
  return with_keys(a.N, io_bf16, [&](auto io, auto kp, auto full) {
    using IO = decltype(io);
    constexpr int KP = decltype(kp)::value;
    constexpr bool FULL = decltype(full)::value;
    const unsigned chunks = (unsigned)(a.Bt * a.H * a.Nc);
    hipLaunchKernelGGL((k_delta_prep<IO, KP, FULL, GRADS>), dim3(chunks), dim3(kThreads), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (GRADS || e != hipSuccess) return e;
    if constexpr (sizeof(IO) == 2) {
      return chain_of(
          a, 1,
          [&](auto ng, unsigned groups) {
            hipLaunchKernelGGL((k_delta_tokens<KP, FULL, ng.value>), dim3(groups), dim3(256 * ng.value), 0, stream, a);
          },
          [&](unsigned groups) {
            hipLaunchKernelGGL((k_delta_columns<KP, FULL>), dim3(groups), dim3(256), 0, stream, a);
          });
    } else {
      hipLaunchKernelGGL((k_delta_chain<IO, KP, FULL>), dim3((unsigned)(a.Bt * a.H * ((a.P + 15) / 16))),
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

size_t delta_workspace(DeltaArgs& a, bool grads, char* ws) {
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
  take(a.qk, n * 3 * frags);
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
    if (a.H != a.G) {
      take(a.part_q, keys);
      take(a.part_k, keys);
    }
    take(a.part_h, n * 2 * sizeof(float));
  }
  return at;
}

hipError_t launch_delta_scan(const DeltaArgs& a, bool io_bf16, hipStream_t stream) {
  return delta::launch_scan<false>(a, io_bf16, stream);
}

hipError_t launch_delta_matrices(const DeltaArgs& a, bool io_bf16, hipStream_t stream) {
  return delta::launch_scan<true>(a, io_bf16, stream);
}

hipError_t launch_delta_step(const DeltaArgs& a, bool io_bf16, hipStream_t stream) {
  return io_bf16 ? delta::launch_step<bf16>(a, stream) : delta::launch_step<float>(a, stream);
}

}  // namespace ssd
