// C ABI of the gated delta rule: argument validation and dispatch to the gfx950
// kernels.  Declarations and the contract are in include/ssd.h.  As in
// ssd_api.cpp everything here runs on the host, validation is complete before
// the first launch, and nothing is allocated, synchronised or kept.
#include "ssd.h"

#include <math.h>
#include <stdint.h>

#include "ssd_check.h"
#include "ssd_launch.h"

namespace {

using namespace ssd;

inline bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }
inline ssd_status status_of(hipError_t e) { return e == hipSuccess ? SSD_OK : SSD_ERR_HIP; }

// workgroups of 256 threads: a grid's threads count in 32 bits
constexpr int64_t kMaxGroups = (1 << 24) - 1;

// of any length, also where a sum with it would overflow
int64_t chunks_of(int64_t tokens) { return tokens / kDeltaChunk + (tokens % kDeltaChunk != 0); }

// bytes that tensors and the spans of strided ones take
struct Sizes {
  int64_t q, k, v, y, gates, heads, state;
  int64_t dq = 0, dk = 0, dv = 0;
};

// elements from the first to the last of `rows` rows of `width`, `stride` apart
bool span_of(int64_t rows, int64_t width, int64_t stride, int64_t es, int64_t* bytes) {
  int64_t n = 0;
  if (rows == 0) { *bytes = 0; return true; }
  if (!mul_ok(rows, stride, &n) || n > INT64_MAX / 16) return false;
  *bytes = (n - stride + width) * es;
  return true;
}

ssd_status check(const ssd_delta_desc* d, bool step, bool grads, Sizes* s) {
  if (!d) return SSD_ERR_INVALID_ARG;
  if (d->io_dtype != SSD_F32 && d->io_dtype != SSD_BF16) return SSD_ERR_DTYPE;
  if (d->batch < 0 || (!step && d->seqlen < 0) || d->nheads <= 0 || d->headdim <= 0 ||
      d->dstate <= 0 || d->ngroups <= 0 || d->nheads % d->ngroups != 0)
    return SSD_ERR_SHAPE;
  if (!limits_ok(d->dt_min, d->dt_max) || !(d->norm_eps >= 0.0f) || !isfinite(d->norm_eps) ||
      !isfinite(d->scale))
    return SSD_ERR_INVALID_ARG;
  // the 64 rows of a chunk count in 32 bits of bytes
  constexpr int64_t kMaxStride = (1 << 25) - 512;
  if (d->q_stride > kMaxStride || d->k_stride > kMaxStride || d->v_stride > kMaxStride ||
      d->headdim % 8 != 0 || d->headdim > SSD_DELTA_MAX_P || d->dstate % 8 != 0 ||
      d->dstate > SSD_DELTA_MAX_N || d->nheads > kMaxGroups)
    return SSD_ERR_UNSUPPORTED;
  const int64_t es = (int64_t)io_size(d->io_dtype);
  const int64_t gn = d->ngroups * d->dstate, hp = d->nheads * d->headdim;
  if (d->q_stride < gn || d->k_stride < gn || d->v_stride < hp) return SSD_ERR_SHAPE;
  if (grads && (d->dq_stride < gn || d->dk_stride < gn || d->dv_stride < hp)) return SSD_ERR_SHAPE;
  const int64_t chunks = step ? 1 : chunks_of(d->seqlen);
  int64_t bh = 0, groups = 0, tokens = 0, state = 0, y = 0, gates = 0;
  if (!mul_ok(d->batch, d->nheads, &bh) || !mul_ok(bh, chunks, &groups) || groups > kMaxGroups ||
      !mul_ok(bh, (grads ? 2 : 1) * ((d->headdim + 15) / 16), &groups) || groups > kMaxGroups ||
      !mul_ok(d->batch, step ? 1 : d->seqlen, &tokens) ||
      !span_of(tokens, gn, d->q_stride, es, &s->q) || !span_of(tokens, gn, d->k_stride, es, &s->k) ||
      !span_of(tokens, hp, d->v_stride, es, &s->v) || !mul_ok(tokens, hp, &y) || y > INT64_MAX / 16 ||
      !mul_ok(tokens, d->nheads, &gates) || gates > INT64_MAX / 16)
    return SSD_ERR_UNSUPPORTED;
  if (grads && (!span_of(tokens, gn, d->dq_stride, es, &s->dq) ||
                !span_of(tokens, gn, d->dk_stride, es, &s->dk) ||
                !span_of(tokens, hp, d->dv_stride, es, &s->dv)))
    return SSD_ERR_UNSUPPORTED;
  // the gradients' workspace, in bytes (a bound), and 2 Bt T G rows, up to 32 threads for each
  int64_t rows = 0, ws = 0;
  if (grads && (!mul_ok(tokens, 2 * d->ngroups, &rows) || rows > (int64_t{1} << 27) - 8 ||
                !mul_ok(bh * chunks, 8 * ((d->headdim + 8) * 128 + 64 * (d->headdim + d->dstate + 80)), &ws) ||
                ws > INT64_MAX / 16))
    return SSD_ERR_UNSUPPORTED;
  state = bh * d->headdim * d->dstate;
  s->y = y * es;
  s->gates = gates * 4;
  s->heads = d->nheads * 4;
  s->state = state * 4;
  return SSD_OK;
}

// rows that are read or written 16 bytes at a time
bool rows_aligned(const void* p, int64_t stride, int32_t dtype) {
  return aligned16(p) && stride * (int64_t)io_size(dtype) % 16 == 0;
}

// every output against every input and every other output
template <size_t NO, size_t NI>
bool outputs_clear(const Range (&outs)[NO], const Range (&ins)[NI]) {
  for (size_t i = 0; i < NO; ++i) {
    for (const Range& r : ins)
      if (overlap(outs[i], r)) return false;
    for (size_t j = i + 1; j < NO; ++j)
      if (overlap(outs[i], outs[j])) return false;
  }
  return true;
}

// Rows of two outputs that lie in one another's spans: disjoint columns of one
// tensor are apart, everything else is not.
struct Rows {
  const void* p;
  int64_t bytes, width, stride;  // of all rows, of a row's columns, between rows
};
bool rows_clear(const Rows& x, const Rows& y) {
  const Range a = range_of(x.p, x.bytes), b = range_of(y.p, y.bytes);
  if (!overlap(a, b)) return true;
  if (a.lo > b.lo) return rows_clear(y, x);
  const int64_t off = (int64_t)(b.lo - a.lo) % x.stride;
  return x.stride == y.stride && off >= x.width && off + y.width <= x.stride;
}

DeltaArgs args_of(const ssd_delta_desc* d, const void* q, const void* k, const void* v,
                  const float* dt, const float* dt_bias, const float* A, const float* beta) {
  DeltaArgs a = {};
  a.q = q; a.k = k; a.v = v;
  a.q_stride = d->q_stride; a.k_stride = d->k_stride; a.v_stride = d->v_stride;
  a.dt = dt; a.dt_bias = dt_bias; a.A = A; a.beta = beta;
  a.Bt = d->batch; a.T = d->seqlen; a.H = d->nheads; a.G = d->ngroups;
  a.Nc = chunks_of(d->seqlen);
  a.P = (int32_t)d->headdim; a.N = (int32_t)d->dstate;
  a.softplus = d->dt_softplus ? 1 : 0; a.sigmoid = d->beta_sigmoid ? 1 : 0;
  a.unit = d->qk_norm ? 1 : 0;
  a.dt_min = d->dt_min; a.dt_max = d->dt_max; a.norm_eps = d->norm_eps; a.scale = d->scale;
  return a;
}

// dst = src, or zeros; a launch's threads, one for 4 floats, count in 32 bits
ssd_status copy_state(float* dst, const float* src, int64_t n, hipStream_t stream) {
  constexpr int64_t kPart = int64_t{1} << 30;
  for (int64_t at = 0; at < n; at += kPart) {
    const hipError_t e = launch_copy_or_zero(dst + at, src ? src + at : nullptr, n - at < kPart ? n - at : kPart,
                                             stream);
    if (e != hipSuccess) return SSD_ERR_HIP;
  }
  return SSD_OK;
}

}  // namespace

extern "C" {

size_t ssd_delta_scan_workspace_bytes(const ssd_delta_desc* d) {
  Sizes s;
  if (check(d, false, false, &s) != SSD_OK) return 0;
  DeltaArgs a = args_of(d, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr);
  return delta_workspace(a, false, nullptr);
}

ssd_status ssd_delta_scan(const ssd_delta_desc* d, const void* q, const void* k, const void* v,
                          const float* dt, const float* dt_bias, const float* A, const float* beta,
                          const float* initial_state, void* y, float* final_state, void* workspace,
                          size_t workspace_bytes, hipStream_t stream) {
  Sizes s;
  const ssd_status st = check(d, false, false, &s);
  if (st != SSD_OK) return st;
  const bool tokens = d->batch > 0 && d->seqlen > 0;
  if (tokens && (!q || !k || !v || !dt || !A || !beta || !y)) return SSD_ERR_INVALID_ARG;
  if (!rows_aligned(q, d->q_stride, d->io_dtype) || !rows_aligned(k, d->k_stride, d->io_dtype) ||
      !rows_aligned(v, d->v_stride, d->io_dtype) || !aligned16(y) || !aligned16(initial_state) ||
      !aligned16(final_state) || !aligned4(dt) || !aligned4(dt_bias) || !aligned4(A) ||
      !aligned4(beta) || !aligned256(workspace))
    return SSD_ERR_ALIGNMENT;
  const size_t need = ssd_delta_scan_workspace_bytes(d);
  if (tokens && (!workspace || workspace_bytes < need)) return SSD_ERR_WORKSPACE;
  const bool in_place = final_state && final_state == initial_state;
  const Range outs[] = {range_of(y, s.y), range_of(final_state, s.state),
                        range_of(workspace, tokens ? (int64_t)need : 0)};
  const Range ins[] = {range_of(q, s.q), range_of(k, s.k), range_of(v, s.v), range_of(dt, s.gates),
                       range_of(beta, s.gates), range_of(A, s.heads), range_of(dt_bias, s.heads),
                       in_place ? Range{0, 0} : range_of(initial_state, s.state)};
  if (!outputs_clear(outs, ins)) return SSD_ERR_INVALID_ARG;
  if (!tokens) {
    if (!final_state || in_place) return SSD_OK;
    return copy_state(final_state, initial_state, s.state / 4, stream);
  }
  const bool io_bf16 = d->io_dtype == SSD_BF16;
  DeltaArgs a = args_of(d, q, k, v, dt, dt_bias, A, beta);
  a.h0 = initial_state; a.y = y; a.state = final_state;
  delta_workspace(a, false, static_cast<char*>(workspace));
  return status_of(launch_delta_scan(a, io_bf16, stream));
}

size_t ssd_delta_scan_backward_workspace_bytes(const ssd_delta_desc* d) {
  Sizes s;
  if (check(d, false, true, &s) != SSD_OK) return 0;
  DeltaArgs a = args_of(d, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr);
  return delta_workspace(a, true, nullptr);
}

ssd_status ssd_delta_scan_backward(const ssd_delta_desc* d, const void* q, const void* k,
                                   const void* v, const float* dt, const float* dt_bias,
                                   const float* A, const float* beta, const float* initial_state,
                                   const void* dy, const float* dfinal_state, void* dq, void* dk,
                                   void* dv, float* ddt, float* dbeta, float* dA, float* ddt_bias,
                                   float* dinitial_state, void* workspace, size_t workspace_bytes,
                                   hipStream_t stream) {
  Sizes s;
  const ssd_status st = check(d, false, true, &s);
  if (st != SSD_OK) return st;
  const bool tokens = d->batch > 0 && d->seqlen > 0;
  if (!dA || (tokens && (!q || !k || !v || !dt || !A || !beta || !dy || !dq || !dk || !dv || !ddt || !dbeta)))
    return SSD_ERR_INVALID_ARG;
  const int32_t io = d->io_dtype;
  if (!rows_aligned(q, d->q_stride, io) || !rows_aligned(k, d->k_stride, io) ||
      !rows_aligned(v, d->v_stride, io) || !rows_aligned(dq, d->dq_stride, io) ||
      !rows_aligned(dk, d->dk_stride, io) || !rows_aligned(dv, d->dv_stride, io) || !aligned16(dy) ||
      !aligned16(initial_state) || !aligned16(dfinal_state) || !aligned16(dinitial_state) ||
      !aligned256(workspace))
    return SSD_ERR_ALIGNMENT;
  for (const float* p : {dt, dt_bias, A, beta, (const float*)ddt, (const float*)dbeta, (const float*)dA,
                         (const float*)ddt_bias})
    if (!aligned4(p)) return SSD_ERR_ALIGNMENT;
  const size_t need = ssd_delta_scan_backward_workspace_bytes(d);
  if (tokens && (!workspace || workspace_bytes < need)) return SSD_ERR_WORKSPACE;
  const Range outs[] = {range_of(ddt, s.gates), range_of(dbeta, s.gates), range_of(dA, s.heads),
                        range_of(ddt_bias, s.heads), range_of(dinitial_state, s.state),
                        range_of(workspace, tokens ? (int64_t)need : 0)};
  const Range ins[] = {range_of(q, s.q), range_of(k, s.k), range_of(v, s.v), range_of(dy, s.y),
                       range_of(dt, s.gates), range_of(beta, s.gates), range_of(A, s.heads),
                       range_of(dt_bias, s.heads), range_of(initial_state, s.state),
                       range_of(dfinal_state, s.state)};
  if (!outputs_clear(outs, ins)) return SSD_ERR_INVALID_ARG;
  const int64_t es = (int64_t)io_size(io), gn = d->ngroups * d->dstate * es, hp = d->nheads * d->headdim * es;
  const Rows rows[] = {{dq, s.dq, gn, d->dq_stride * es}, {dk, s.dk, gn, d->dk_stride * es},
                       {dv, s.dv, hp, d->dv_stride * es}};
  for (int i = 0; i < 3; ++i) {
    for (const Range& r : ins)
      if (overlap(range_of(rows[i].p, rows[i].bytes), r)) return SSD_ERR_INVALID_ARG;
    for (const Range& r : outs)
      if (overlap(range_of(rows[i].p, rows[i].bytes), r)) return SSD_ERR_INVALID_ARG;
    for (int j = i + 1; j < 3; ++j)
      if (!rows_clear(rows[i], rows[j])) return SSD_ERR_INVALID_ARG;
  }
  if (!tokens) {
    const hipError_t e = launch_backward_zero_heads(dA, ddt_bias, nullptr, d->nheads, stream);
    if (e != hipSuccess) return SSD_ERR_HIP;
    return dinitial_state ? copy_state(dinitial_state, dfinal_state, s.state / 4, stream) : SSD_OK;
  }
  const bool io_bf16 = io == SSD_BF16;
  DeltaArgs a = args_of(d, q, k, v, dt, dt_bias, A, beta);
  a.h0 = initial_state; a.dy = dy; a.dfinal = dfinal_state;
  a.dq = dq; a.dk = dk; a.dv = dv;
  a.dq_stride = d->dq_stride; a.dk_stride = d->dk_stride; a.dv_stride = d->dv_stride;
  a.ddt = ddt; a.dbeta = dbeta; a.dA = dA; a.ddt_bias = ddt_bias; a.dh0 = dinitial_state;
  delta_workspace(a, true, static_cast<char*>(workspace));
  return status_of(launch_delta_scan_backward(a, io_bf16, stream));
}

ssd_status ssd_delta_step(const ssd_delta_desc* d, float* state, const void* q, const void* k,
                          const void* v, const float* dt, const float* dt_bias, const float* A,
                          const float* beta, void* y, hipStream_t stream) {
  Sizes s;
  const ssd_status st = check(d, true, false, &s);
  if (st != SSD_OK) return st;
  if (d->batch == 0) return SSD_OK;
  if (!state || !q || !k || !v || !dt || !A || !beta || !y) return SSD_ERR_INVALID_ARG;
  if (!rows_aligned(q, d->q_stride, d->io_dtype) || !rows_aligned(k, d->k_stride, d->io_dtype) ||
      !rows_aligned(v, d->v_stride, d->io_dtype) || !aligned16(y) || !aligned16(state) ||
      !aligned4(dt) || !aligned4(dt_bias) || !aligned4(A) || !aligned4(beta))
    return SSD_ERR_ALIGNMENT;
  const Range outs[] = {range_of(y, s.y), range_of(state, s.state)};
  const Range ins[] = {range_of(q, s.q), range_of(k, s.k), range_of(v, s.v), range_of(dt, s.gates),
                       range_of(beta, s.gates), range_of(A, s.heads), range_of(dt_bias, s.heads)};
  if (!outputs_clear(outs, ins)) return SSD_ERR_INVALID_ARG;
  DeltaArgs a = args_of(d, q, k, v, dt, dt_bias, A, beta);
  a.y = y; a.state = state;
  return status_of(launch_delta_step(a, d->io_dtype == SSD_BF16, stream));
}

}  // extern "C"
