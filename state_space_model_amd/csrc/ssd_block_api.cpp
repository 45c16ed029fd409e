// C ABI of the operators between two scans (norms, 8-bit projections, the
// convolution's gradients): argument validation and dispatch to the gfx950
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

inline bool io_dtype_ok(int32_t dt) { return dt == SSD_F32 || dt == SSD_BF16; }
inline bool eps_ok(float e) { return e >= 0.0f && isfinite(e); }
inline bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline int64_t pad_q8(int64_t cols) { return (cols + SSD_Q8_PAD - 1) / SSD_Q8_PAD * SSD_Q8_PAD; }
inline ssd_status status_of(hipError_t e) { return e == hipSuccess ? SSD_OK : SSD_ERR_HIP; }

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

// sizes whose byte counts must fit comfortably in 64 bits
bool elems_ok(int64_t rows, int64_t cols, int64_t* n) {
  return mul_ok(rows, cols, n) && *n <= INT64_MAX / 16;
}

ssd_status check_add_norm(const ssd_add_norm_desc* d, int64_t* n) {
  if (!d) return SSD_ERR_INVALID_ARG;
  if (!io_dtype_ok(d->io_dtype)) return SSD_ERR_DTYPE;
  if (d->rows < 0 || d->cols <= 0) return SSD_ERR_SHAPE;
  if (!eps_ok(d->eps) || !isfinite(d->scale)) return SSD_ERR_INVALID_ARG;
  // one workgroup per row at most: rows index a 32-bit grid dimension
  if (d->cols > SSD_NORM_MAX_COLS || d->rows > INT32_MAX || !elems_ok(d->rows, d->cols, n))
    return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

ssd_status check_gated_norm(const ssd_gated_norm_desc* d, bool backward, int64_t* n, int64_t* nz,
                            int64_t* ndz) {
  if (!d) return SSD_ERR_INVALID_ARG;
  if (!io_dtype_ok(d->io_dtype)) return SSD_ERR_DTYPE;
  if (d->rows < 0 || d->cols <= 0 || d->groups <= 0 || d->cols % d->groups != 0)
    return SSD_ERR_SHAPE;
  if (d->z_stride < d->cols || (backward && d->dz_stride < d->cols)) return SSD_ERR_SHAPE;
  if (!eps_ok(d->eps)) return SSD_ERR_INVALID_ARG;
  int64_t units = 0;
  if (d->cols / d->groups > SSD_NORM_MAX_COLS || !elems_ok(d->rows, d->cols, n) ||
      !elems_ok(d->rows, d->z_stride, nz) ||
      !elems_ok(d->rows, backward ? d->dz_stride : 0, ndz) || d->groups > 65535 ||
      !mul_ok(d->rows, d->groups, &units) || units > INT32_MAX)
    return SSD_ERR_UNSUPPORTED;
  // the span of the strided rows ends with the last row's columns
  if (d->rows > 0) {
    *nz -= d->z_stride - d->cols;
    if (backward) *ndz -= d->dz_stride - d->cols;
  }
  return SSD_OK;
}

ssd_status add_norm(const ssd_add_norm_desc* d, const void* x, const float* residual,
                    const float* weight, void* y, int8_t* q, float* qscale, float* residual_out,
                    bool q8, hipStream_t stream) {
  int64_t n = 0;
  const ssd_status st = check_add_norm(d, &n);
  if (st != SSD_OK) return st;
  if (d->rows == 0) return SSD_OK;
  if (!x || !weight || (q8 ? (!q || !qscale) : !y)) return SSD_ERR_INVALID_ARG;
  const size_t es = io_size(d->io_dtype);
  if (!aligned_to(x, es) || !aligned_to(y, es) || !aligned4(residual) || !aligned4(weight) ||
      !aligned4(residual_out) || !aligned4(qscale) || !aligned16(q))
    return SSD_ERR_ALIGNMENT;
  const int64_t Dp = pad_q8(d->cols);
  const Range r_res = range_of(residual, n * 4);
  const bool in_place = residual_out && residual_out == residual;
  const Range outs[] = {range_of(y, n * (int64_t)es), range_of(q, q8 ? d->rows * Dp : 0),
                        range_of(qscale, d->rows * 4), range_of(residual_out, n * 4)};
  const Range ins[] = {range_of(x, n * (int64_t)es), range_of(weight, d->cols * 4),
                       in_place ? Range{0, 0} : r_res};
  if (!outputs_clear(outs, ins)) return SSD_ERR_INVALID_ARG;

  AddNormArgs a = {};
  a.x = x; a.residual = residual; a.weight = weight; a.y = y; a.q = q; a.qscale = qscale;
  a.residual_out = residual_out;
  a.R = d->rows; a.D = (int32_t)d->cols; a.Dp = (int32_t)Dp;
  a.scale = d->scale; a.eps = d->eps;
  return status_of(launch_add_norm(a, d->io_dtype == SSD_BF16, stream));
}

ssd_status gated_norm(const ssd_gated_norm_desc* d, const void* y, const void* z,
                      const float* weight, void* out, int8_t* q, float* qscale, bool q8,
                      hipStream_t stream) {
  int64_t n = 0, nz = 0, ndz = 0;
  const ssd_status st = check_gated_norm(d, false, &n, &nz, &ndz);
  if (st != SSD_OK) return st;
  if (q8 && (d->groups > SSD_NORM_MAX_GROUPS_Q8 || d->cols > SSD_NORM_MAX_COLS))
    return SSD_ERR_UNSUPPORTED;
  if (d->rows == 0) return SSD_OK;
  if (!y || !z || !weight || (q8 ? (!q || !qscale) : !out)) return SSD_ERR_INVALID_ARG;
  const size_t es = io_size(d->io_dtype);
  if (!aligned_to(y, es) || !aligned_to(z, es) || !aligned_to(out, es) || !aligned4(weight) ||
      !aligned4(qscale) || !aligned16(q))
    return SSD_ERR_ALIGNMENT;
  const int64_t Dp = pad_q8(d->cols);
  const Range outs[] = {range_of(out, n * (int64_t)es), range_of(q, q8 ? d->rows * Dp : 0),
                        range_of(qscale, d->rows * 4)};
  const Range ins[] = {range_of(y, n * (int64_t)es), range_of(z, nz * (int64_t)es),
                       range_of(weight, d->cols * 4)};
  if (!outputs_clear(outs, ins)) return SSD_ERR_INVALID_ARG;

  GatedNormArgs a = {};
  a.y = y; a.z = z; a.weight = weight; a.out = out; a.q = q; a.qscale = qscale;
  a.R = d->rows; a.D = d->cols; a.z_stride = d->z_stride;
  a.G = (int32_t)d->groups; a.W = (int32_t)(d->cols / d->groups); a.Dp = (int32_t)Dp;
  a.eps = d->eps;
  return status_of(launch_gated_norm(a, d->io_dtype == SSD_BF16, stream));
}

}  // namespace

extern "C" {

ssd_status ssd_add_norm(const ssd_add_norm_desc* d, const void* x, const float* residual,
                        const float* weight, void* y, float* residual_out, hipStream_t stream) {
  return add_norm(d, x, residual, weight, y, nullptr, nullptr, residual_out, false, stream);
}

ssd_status ssd_add_norm_q8(const ssd_add_norm_desc* d, const void* x, const float* residual,
                           const float* weight, int8_t* q, float* qscale, float* residual_out,
                           hipStream_t stream) {
  return add_norm(d, x, residual, weight, nullptr, q, qscale, residual_out, true, stream);
}

size_t ssd_add_norm_backward_workspace_bytes(const ssd_add_norm_desc* d) {
  int64_t n = 0;
  if (check_add_norm(d, &n) != SSD_OK) return 0;
  return round_up((size_t)(add_norm_backward_parts(d->rows, d->cols, d->io_dtype == SSD_BF16) * d->cols) * 4, kAlign);
}

ssd_status ssd_add_norm_backward(const ssd_add_norm_desc* d, const float* residual_out,
                                 const float* weight, const void* dy, const float* dresidual_out,
                                 void* dx, float* dresidual, float* dweight, void* workspace,
                                 size_t workspace_bytes, hipStream_t stream) {
  int64_t n = 0;
  const ssd_status st = check_add_norm(d, &n);
  if (st != SSD_OK) return st;
  if (!dweight) return SSD_ERR_INVALID_ARG;
  if (d->rows > 0 && (!residual_out || !weight || !dy)) return SSD_ERR_INVALID_ARG;
  const size_t es = io_size(d->io_dtype);
  if (!aligned4(residual_out) || !aligned4(weight) || !aligned_to(dy, es) ||
      !aligned4(dresidual_out) || !aligned_to(dx, es) || !aligned4(dresidual) ||
      !aligned4(dweight) || !aligned16(workspace))
    return SSD_ERR_ALIGNMENT;
  const size_t need = ssd_add_norm_backward_workspace_bytes(d);
  if (d->rows > 0 && (!workspace || workspace_bytes < need)) return SSD_ERR_WORKSPACE;
  const bool in_place = dresidual && dresidual == dresidual_out;
  const Range outs[] = {range_of(dx, n * (int64_t)es), range_of(dresidual, n * 4),
                        range_of(dweight, d->cols * 4),
                        range_of(workspace, d->rows > 0 ? (int64_t)need : 0)};
  const Range ins[] = {range_of(residual_out, n * 4), range_of(weight, d->cols * 4),
                       range_of(dy, n * (int64_t)es),
                       in_place ? Range{0, 0} : range_of(dresidual_out, n * 4)};
  if (!outputs_clear(outs, ins)) return SSD_ERR_INVALID_ARG;
  if (d->rows == 0)
    return status_of(launch_backward_zero_heads(dweight, nullptr, nullptr, d->cols, stream));

  AddNormArgs a = {};
  a.residual_out = const_cast<float*>(residual_out); a.weight = weight; a.dy = dy;
  a.dres_out = dresidual_out; a.dx = dx; a.dres = dresidual; a.dweight = dweight;
  a.part = static_cast<float*>(workspace);
  a.R = d->rows; a.D = (int32_t)d->cols; a.scale = d->scale; a.eps = d->eps;
  return status_of(launch_add_norm_backward(a, d->io_dtype == SSD_BF16, stream));
}

ssd_status ssd_gated_norm(const ssd_gated_norm_desc* d, const void* y, const void* z,
                          const float* weight, void* out, hipStream_t stream) {
  return gated_norm(d, y, z, weight, out, nullptr, nullptr, false, stream);
}

ssd_status ssd_gated_norm_q8(const ssd_gated_norm_desc* d, const void* y, const void* z,
                             const float* weight, int8_t* q, float* qscale, hipStream_t stream) {
  return gated_norm(d, y, z, weight, nullptr, q, qscale, true, stream);
}

size_t ssd_gated_norm_backward_workspace_bytes(const ssd_gated_norm_desc* d) {
  int64_t n = 0, nz = 0, ndz = 0;
  if (check_gated_norm(d, true, &n, &nz, &ndz) != SSD_OK) return 0;
  return round_up((size_t)(gated_norm_backward_parts(d->rows, d->groups, d->cols / d->groups,
                                                       d->io_dtype == SSD_BF16) *
                           d->cols) * 4, kAlign);
}

ssd_status ssd_gated_norm_backward(const ssd_gated_norm_desc* d, const void* y, const void* z,
                                   const float* weight, const void* dout, void* dy, void* dz,
                                   float* dweight, void* workspace, size_t workspace_bytes,
                                   hipStream_t stream) {
  int64_t n = 0, nz = 0, ndz = 0;
  const ssd_status st = check_gated_norm(d, true, &n, &nz, &ndz);
  if (st != SSD_OK) return st;
  if (!dweight) return SSD_ERR_INVALID_ARG;
  if (d->rows > 0 && (!y || !z || !weight || !dout || !dy || !dz)) return SSD_ERR_INVALID_ARG;
  const size_t es = io_size(d->io_dtype);
  for (const void* p : {y, z, dout, static_cast<const void*>(dy), static_cast<const void*>(dz)})
    if (!aligned_to(p, es)) return SSD_ERR_ALIGNMENT;
  if (!aligned4(weight) || !aligned4(dweight) || !aligned16(workspace)) return SSD_ERR_ALIGNMENT;
  const size_t need = ssd_gated_norm_backward_workspace_bytes(d);
  if (d->rows > 0 && (!workspace || workspace_bytes < need)) return SSD_ERR_WORKSPACE;
  const int64_t e = (int64_t)es;
  const Range outs[] = {range_of(dy, n * e), range_of(dz, ndz * e), range_of(dweight, d->cols * 4),
                        range_of(workspace, d->rows > 0 ? (int64_t)need : 0)};
  const Range ins[] = {range_of(y, n * e), range_of(z, nz * e), range_of(weight, d->cols * 4),
                       range_of(dout, n * e)};
  if (!outputs_clear(outs, ins)) return SSD_ERR_INVALID_ARG;
  if (d->rows == 0)
    return status_of(launch_backward_zero_heads(dweight, nullptr, nullptr, d->cols, stream));

  GatedNormArgs a = {};
  a.y = y; a.z = z; a.weight = weight; a.dout = dout; a.dy = dy; a.dz = dz; a.dweight = dweight;
  a.part = static_cast<float*>(workspace);
  a.R = d->rows; a.D = d->cols; a.z_stride = d->z_stride; a.dz_stride = d->dz_stride;
  a.G = (int32_t)d->groups; a.W = (int32_t)(d->cols / d->groups); a.eps = d->eps;
  return status_of(launch_gated_norm_backward(a, d->io_dtype == SSD_BF16, stream));
}

ssd_status ssd_quantize_q8(int64_t rows, int64_t cols, int32_t dtype, const void* v, int8_t* q,
                           float* qscale, hipStream_t stream) {
  if (!io_dtype_ok(dtype)) return SSD_ERR_DTYPE;
  if (rows < 0 || cols <= 0) return SSD_ERR_SHAPE;
  int64_t n = 0;
  if (rows > INT32_MAX || cols > SSD_Q8_MAX_COLS || !elems_ok(rows, cols, &n)) return SSD_ERR_UNSUPPORTED;
  if (rows == 0) return SSD_OK;
  if (!v || !q || !qscale) return SSD_ERR_INVALID_ARG;
  if (!aligned_to(v, io_size(dtype)) || !aligned16(q) || !aligned4(qscale))
    return SSD_ERR_ALIGNMENT;
  const int64_t Kp = pad_q8(cols);
  const Range outs[] = {range_of(q, rows * Kp), range_of(qscale, rows * 4)};
  const Range ins[] = {range_of(v, n * (int64_t)io_size(dtype))};
  if (!outputs_clear(outs, ins)) return SSD_ERR_INVALID_ARG;
  return status_of(launch_quantize_q8(v, dtype == SSD_BF16, rows, (int32_t)cols, (int32_t)Kp, q,
                                      qscale, stream));
}

ssd_status ssd_linear_q8(const ssd_linear_q8_desc* d, const int8_t* q, const float* qscale,
                         const int8_t* wq, const float* wscale, void* out, hipStream_t stream) {
  if (!d) return SSD_ERR_INVALID_ARG;
  if (!io_dtype_ok(d->out_dtype)) return SSD_ERR_DTYPE;
  if (d->rows < 0 || d->cols <= 0 || d->outs <= 0 || d->cols % SSD_Q8_PAD != 0)
    return SSD_ERR_SHAPE;
  int64_t nq = 0, nw = 0, no = 0;
  // 2^14 * SSD_Q8_MAX_COLS < 2^31 bounds the integer sum for any 8-bit operands;
  // a grid's threads (256 per 64 x 64 tile, 512 per 16 outputs) count in 32 bits
  if (d->cols > SSD_Q8_MAX_COLS || d->rows > (1 << 30) || d->outs > (1 << 27) - 16 ||
      !elems_ok(d->rows, d->cols, &nq) || !elems_ok(d->outs, d->cols, &nw) ||
      !elems_ok(d->rows, d->outs, &no) || (d->rows / 64 + 1) * (d->outs / 64 + 1) >= (1 << 24))
    return SSD_ERR_UNSUPPORTED;
  if (d->rows == 0) return SSD_OK;
  if (!q || !qscale || !wq || !wscale || !out) return SSD_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(wq) || !aligned4(qscale) || !aligned4(wscale) ||
      !aligned_to(out, io_size(d->out_dtype)))
    return SSD_ERR_ALIGNMENT;
  const Range outs[] = {range_of(out, no * (int64_t)io_size(d->out_dtype))};
  const Range ins[] = {range_of(q, nq), range_of(qscale, d->rows * 4), range_of(wq, nw),
                       range_of(wscale, d->outs * 4)};
  if (!outputs_clear(outs, ins)) return SSD_ERR_INVALID_ARG;

  LinearQ8Args a = {};
  a.q = q; a.qscale = qscale; a.wq = wq; a.wscale = wscale; a.out = out;
  a.M = d->rows; a.N = d->outs; a.K = (int32_t)d->cols;
  return status_of(launch_linear_q8(a, d->out_dtype == SSD_BF16, stream));
}

namespace {

struct ConvBwdSizes {
  int64_t n = 0, n_state = 0;
};

ssd_status check_conv_backward(const ssd_conv_desc* d, ConvBwdSizes* s) {
  if (!d) return SSD_ERR_INVALID_ARG;
  if (!io_dtype_ok(d->io_dtype)) return SSD_ERR_DTYPE;
  if (d->batch < 0 || d->seqlen < 0 || d->channels <= 0 || d->width <= 0) return SSD_ERR_SHAPE;
  int64_t bt = 0, bd = 0;
  if (!conv_width_supported(d->width) || !mul_ok(d->batch, d->seqlen, &bt) ||
      !elems_ok(bt, d->channels, &s->n) || !mul_ok(d->batch, d->channels, &bd) ||
      !elems_ok(bd, d->width - 1, &s->n_state) ||
      !conv_backward_shape_supported(d->batch, d->seqlen, d->channels, d->width))
    return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

}  // namespace

size_t ssd_conv1d_backward_workspace_bytes(const ssd_conv_desc* d) {
  ConvBwdSizes s;
  if (check_conv_backward(d, &s) != SSD_OK) return 0;
  return round_up((size_t)(conv_backward_parts(d->batch, d->seqlen, d->channels) *
                           (d->width + 1) * d->channels) * 4, kAlign);
}

ssd_status ssd_conv1d_backward(const ssd_conv_desc* d, int32_t dy_dtype, const void* x,
                               const float* w, const float* bias, const void* state_in,
                               const void* dy, const void* dstate_out, void* dx, float* dw,
                               float* dbias, void* dstate, void* workspace,
                               size_t workspace_bytes, hipStream_t stream) {
  ConvBwdSizes s;
  const ssd_status st = check_conv_backward(d, &s);
  if (st != SSD_OK) return st;
  if (dy_dtype != SSD_F32 && dy_dtype != d->io_dtype) return SSD_ERR_DTYPE;
  const bool tokens = d->batch > 0 && d->seqlen > 0;
  if (!w || !dw || (tokens && (!x || !dy || !dx))) return SSD_ERR_INVALID_ARG;
  for (const void* p : {x, state_in, dy, dstate_out, static_cast<const void*>(dx),
                        static_cast<const void*>(dstate), static_cast<const void*>(workspace)})
    if (!aligned16(p)) return SSD_ERR_ALIGNMENT;
  if (!aligned4(w) || !aligned4(bias) || !aligned4(dw) || !aligned4(dbias))
    return SSD_ERR_ALIGNMENT;
  const size_t need = ssd_conv1d_backward_workspace_bytes(d);
  if (tokens && (!workspace || workspace_bytes < need)) return SSD_ERR_WORKSPACE;
  const int64_t es = (int64_t)io_size(d->io_dtype), gs = (int64_t)io_size(dy_dtype);
  const Range outs[] = {range_of(dx, s.n * es), range_of(dw, d->channels * d->width * 4),
                        range_of(dbias, d->channels * 4), range_of(dstate, s.n_state * es),
                        range_of(workspace, tokens ? (int64_t)need : 0)};
  const Range ins[] = {range_of(x, s.n * es), range_of(w, d->channels * d->width * 4),
                       range_of(bias, d->channels * 4), range_of(state_in, s.n_state * es),
                       range_of(dy, s.n * gs), range_of(dstate_out, s.n_state * es)};
  if (!outputs_clear(outs, ins)) return SSD_ERR_INVALID_ARG;

  ConvBwdArgs a = {};
  a.x = x; a.w = w; a.bias = bias; a.state_in = state_in; a.dy = dy; a.dstate_out = dstate_out;
  a.dx = dx; a.dw = dw; a.dbias = dbias; a.dstate = dstate;
  a.part = static_cast<float*>(workspace);
  a.Bt = d->batch; a.T = d->seqlen; a.D = d->channels;
  a.K = (int32_t)d->width; a.silu = d->silu ? 1 : 0;
  return status_of(launch_conv_backward(a, d->io_dtype == SSD_BF16, dy_dtype == SSD_BF16, stream));
}

}  // extern "C"
