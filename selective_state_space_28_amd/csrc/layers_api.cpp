// layers_api.cpp -- the C ABI of the gated linear recurrence (include/ssm_gated.h)
// and of the layer norm (include/ssm_norm.h): argument validation and the calls
// into the kernels.  Every check happens before the first HIP call.
#include <climits>
#include <cmath>
#include <cstdint>

#include "api_checks.hpp"
#include "ssm_gated.h"
#include "ssm_kernels.hpp"
#include "ssm_norm.h"

namespace {

using namespace ssm;

static_assert(SSM_GATED_CKPT_STEPS == kGatedBlock, "the kept states are those entering a wave's block");

bool dtype_ok(int dtype) { return dtype == SSM_F32 || dtype == SSM_BF16; }

Dtype dtype_of(int dtype) { return dtype == SSM_BF16 ? Dtype::BF16 : Dtype::F32; }

int status_of(hipError_t e) { return e == hipSuccess ? SSM_OK : SSM_ERR_HIP; }

bool gate_flags_ok(int flags) { return (flags & ~(SSM_GATE_SOFTPLUS | SSM_GATE_UNIT)) == 0; }

// Rows (b, d) are numbered in 32 bits.
bool gated_shape_ok(int batch, int dim, int64_t seqlen) {
  return shapes_fit(batch, dim, seqlen) && (int64_t)batch * dim <= INT_MAX - 512;
}

size_t gated_ckpt_bytes(int batch, int dim, int64_t seqlen) {
  const int64_t nblk = (seqlen + kGatedBlock - 1) / kGatedBlock;
  return (size_t)batch * (size_t)nblk * (size_t)dim * sizeof(float);
}

// Backward workspace: the three sums of every row (batch > 1: with one batch
// row they are the results).
size_t gated_bwd_ws_bytes(int batch, int dim) {
  return batch > 1 ? round256((size_t)3 * (size_t)batch * (size_t)dim * sizeof(float)) : 0;
}

GatedLaunch gated_launch(const void* x, const void* r, const float* A, const float* r_bias, const void* i,
                         const float* i_bias, const void* z, int flags, const uint8_t* starts, int batch,
                         int dim, int64_t seqlen, int dtype) {
  GatedLaunch a{};
  a.x = x;
  a.r = r;
  a.A = A;
  a.r_bias = r_bias;
  a.i = i;
  a.i_bias = i_bias;
  a.z = z;
  a.starts = starts;
  a.softplus = (flags & SSM_GATE_SOFTPLUS) ? 1 : 0;
  a.unit = (flags & SSM_GATE_UNIT) ? 1 : 0;
  a.batch = batch;
  a.dim = dim;
  a.seqlen = seqlen;
  a.dtype = dtype_of(dtype);
  return a;
}

// The norm numbers its workgroups in 32 bits: tiles of 8 steps and more, or
// tokens where a row has fewer or is too long for 32-bit offsets.
bool norm_shape_ok(int batch, int dim, int64_t seqlen) {
  if (dim < 1 || dim > INT_MAX - 65536 || !shapes_fit(batch, dim, seqlen)) return false;
  const bool by_token = seqlen < 8 || seqlen >= INT_MAX / 4;
  return (int64_t)batch * (by_token ? seqlen : (seqlen + 7) / 8) <= INT_MAX - 4096;
}

size_t norm_bwd_ws_bytes(int batch, int dim, int64_t seqlen, int dtype) {
  return round256((size_t)norm_bwd_parts(batch, dim, seqlen, elem_bytes(dtype)) * 2 * (size_t)dim * sizeof(float));
}

}  // namespace

extern "C" {

size_t ssm_gated_scan_ckpt_bytes(int batch, int dim, int64_t seqlen) {
  return gated_shape_ok(batch, dim, seqlen) ? gated_ckpt_bytes(batch, dim, seqlen) : 0;
}

int ssm_gated_scan_fwd(const void* x, const void* r, const float* A, const float* r_bias, const void* i,
                       const float* i_bias, const void* z, int flags, const uint8_t* starts, const float* h0,
                       void* y, float* last_state, float* ckpt, size_t ckpt_bytes, int batch, int dim,
                       int64_t seqlen, int dtype, void* stream) {
  if (!dtype_ok(dtype)) return SSM_ERR_DTYPE;
  if (!gate_flags_ok(flags)) return SSM_ERR_FLAGS;
  if (!gated_shape_ok(batch, dim, seqlen)) return SSM_ERR_SHAPE;
  const bool empty = batch == 0 || dim == 0;
  if (!empty && seqlen > 0 && (!x || !r || !A || !y)) return SSM_ERR_NULL;
  const size_t es = (size_t)elem_bytes(dtype);
  if (!aligned(x, es) || !aligned(r, es) || !aligned(i, es) || !aligned(z, es) || !aligned(y, es) ||
      !aligned(A, 4) || !aligned(r_bias, 4) || !aligned(i_bias, 4) || !aligned(h0, 4) ||
      !aligned(last_state, 4) || !aligned(ckpt, 4))
    return SSM_ERR_ALIGN;
  if (empty) return SSM_OK;
  const size_t ckb = ckpt != nullptr ? gated_ckpt_bytes(batch, dim, seqlen) : 0;
  if (ckpt_bytes < ckb) return SSM_ERR_WORKSPACE;
  const size_t plane = (size_t)batch * (size_t)dim, tok = plane * (size_t)seqlen * es, ch = (size_t)dim * 4;
  {
    const Span outs[] = {span(y, tok), span(last_state, plane * 4), span(ckpt, ckb)};
    const Span ins[] = {span(x, tok), span(r, tok), span(i, tok), span(z, tok), span(A, ch),
                        span(r_bias, ch), span(i_bias, i != nullptr ? ch : 0),
                        span(starts, (size_t)batch * (size_t)seqlen), span(h0, plane * 4)};
    if (writes_overlap(outs, ins)) return SSM_ERR_ALIAS;
  }
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (seqlen == 0) return last_state == nullptr ? SSM_OK : status_of(launch_fill_state(last_state, h0, (int64_t)plane, st));
  GatedLaunch a = gated_launch(x, r, A, r_bias, i, i_bias, z, flags, starts, batch, dim, seqlen, dtype);
  a.h0 = h0;
  a.y = y;
  a.last_state = last_state;
  a.ckpt = ckpt;
  return status_of(launch_gated_fwd(a, st));
}

size_t ssm_gated_scan_bwd_workspace_bytes(int batch, int dim, int64_t seqlen, int dtype) {
  if (!dtype_ok(dtype) || !gated_shape_ok(batch, dim, seqlen)) return 0;
  if (batch == 0 || dim == 0 || seqlen == 0) return 0;
  return gated_bwd_ws_bytes(batch, dim);
}

int ssm_gated_scan_bwd(const void* x, const void* r, const float* A, const float* r_bias, const void* i,
                       const float* i_bias, const void* z, int flags, const uint8_t* starts, const float* ckpt,
                       size_t ckpt_bytes, const void* dy, const float* dlast_state, void* dx, void* dr, float* dA,
                       float* dr_bias, void* di, float* di_bias, void* dz, float* dh0, int batch, int dim,
                       int64_t seqlen, int dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (!dtype_ok(dtype)) return SSM_ERR_DTYPE;
  if (!gate_flags_ok(flags)) return SSM_ERR_FLAGS;
  if (!gated_shape_ok(batch, dim, seqlen)) return SSM_ERR_SHAPE;
  if (dim > 0 && !dA) return SSM_ERR_NULL;
  const bool empty = batch == 0 || dim == 0 || seqlen == 0;
  if (!empty && (!x || !r || !A || !ckpt || !dy || !dx || !dr || (i && !di) || (z && !dz))) return SSM_ERR_NULL;
  const size_t es = (size_t)elem_bytes(dtype);
  if (!aligned(x, es) || !aligned(r, es) || !aligned(i, es) || !aligned(z, es) || !aligned(dy, es) ||
      !aligned(dx, es) || !aligned(dr, es) || !aligned(di, es) || !aligned(dz, es) || !aligned(A, 4) ||
      !aligned(r_bias, 4) || !aligned(i_bias, 4) || !aligned(ckpt, 4) || !aligned(dlast_state, 4) ||
      !aligned(dA, 4) || !aligned(dr_bias, 4) || !aligned(di_bias, 4) || !aligned(dh0, 4) ||
      !aligned(workspace, 256))
    return SSM_ERR_ALIGN;
  if (dim == 0) return SSM_OK;
  const size_t ckb = gated_ckpt_bytes(batch, dim, seqlen);
  if (!empty && ckpt_bytes < ckb) return SSM_ERR_WORKSPACE;
  const size_t need = ssm_gated_scan_bwd_workspace_bytes(batch, dim, seqlen, dtype);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return SSM_ERR_WORKSPACE;
  const size_t plane = (size_t)batch * (size_t)dim, tok = plane * (size_t)seqlen * es, ch = (size_t)dim * 4;
  {
    const Span outs[] = {span(dx, tok), span(dr, tok), span(i != nullptr ? di : nullptr, tok),
                         span(z != nullptr ? dz : nullptr, tok), span(dA, ch), span(dr_bias, ch),
                         span(di_bias, ch), span(dh0, plane * 4), span(workspace, need)};
    const Span ins[] = {span(x, tok), span(r, tok), span(i, tok), span(z, tok), span(dy, tok), span(A, ch),
                        span(r_bias, ch), span(i_bias, i != nullptr ? ch : 0),
                        span(starts, (size_t)batch * (size_t)seqlen), span(ckpt, ckb),
                        span(dlast_state, plane * 4)};
    if (writes_overlap(outs, ins)) return SSM_ERR_ALIAS;
  }
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (empty) {  // nothing was scanned: zero sums, and the state's gradient passes through
    hipError_t e = launch_fill_state(dA, nullptr, dim, st);
    if (e == hipSuccess && dr_bias != nullptr) e = launch_fill_state(dr_bias, nullptr, dim, st);
    // (i is not asked: the pointer of an empty tensor may be null)
    if (e == hipSuccess && di_bias != nullptr) e = launch_fill_state(di_bias, nullptr, dim, st);
    if (e == hipSuccess && dh0 != nullptr && plane > 0) e = launch_fill_state(dh0, dlast_state, (int64_t)plane, st);
    return status_of(e);
  }
  GatedLaunch a = gated_launch(x, r, A, r_bias, i, i_bias, z, flags, starts, batch, dim, seqlen, dtype);
  a.ckpt = const_cast<float*>(ckpt);
  a.dy = dy;
  a.dlast = dlast_state;
  a.dx = dx;
  a.dr = dr;
  a.di = di;
  a.dz = dz;
  a.dA = dA;
  a.dr_bias = dr_bias;
  a.di_bias = di_bias;
  a.dh0 = dh0;
  a.part = static_cast<float*>(workspace);
  return status_of(launch_gated_bwd(a, st));
}

int ssm_gated_state_update(float* state, const void* x, const void* r, const float* A, const float* r_bias,
                           const void* i, const float* i_bias, const void* z, int flags, const uint8_t* starts,
                           void* y, float* state_out, int batch, int dim, int dtype, void* stream) {
  if (!dtype_ok(dtype)) return SSM_ERR_DTYPE;
  if (!gate_flags_ok(flags)) return SSM_ERR_FLAGS;
  if (!shapes_fit(batch, dim, 1) || dim > INT_MAX - 2048) return SSM_ERR_SHAPE;
  const bool empty = batch == 0 || dim == 0;
  if (!empty && (!state || !x || !r || !A || !y)) return SSM_ERR_NULL;
  const size_t es = (size_t)elem_bytes(dtype);
  if (!aligned(state, 4) || !aligned(x, es) || !aligned(r, es) || !aligned(i, es) || !aligned(z, es) ||
      !aligned(y, es) || !aligned(A, 4) || !aligned(r_bias, 4) || !aligned(i_bias, 4) || !aligned(state_out, 4))
    return SSM_ERR_ALIGN;
  if (empty) return SSM_OK;
  if (state_out == nullptr) state_out = state;
  const size_t plane = (size_t)batch * (size_t)dim, tok = plane * es, ch = (size_t)dim * 4;
  {
    const Span outs[] = {span(y, tok), span(state_out, plane * 4)};
    const Span ins[] = {span(x, tok), span(r, tok), span(i, tok), span(z, tok), span(A, ch), span(r_bias, ch),
                        span(i_bias, i != nullptr ? ch : 0), span(starts, (size_t)batch),
                        // in place is each element's own read and write
                        span(state_out != state ? state : nullptr, plane * 4)};
    if (writes_overlap(outs, ins)) return SSM_ERR_ALIAS;
  }
  GatedLaunch a = gated_launch(x, r, A, r_bias, i, i_bias, z, flags, starts, batch, dim, 1, dtype);
  a.h0 = state;
  a.y = y;
  a.last_state = state_out;
  return status_of(launch_gated_step(a, static_cast<hipStream_t>(stream)));
}

int ssm_layer_norm_fwd(const void* x, const void* residual, const float* weight, const float* bias, float eps,
                       void* y, void* sum_out, float* mean, float* rstd, int batch, int dim, int64_t seqlen,
                       int dtype, void* stream) {
  if (!dtype_ok(dtype)) return SSM_ERR_DTYPE;
  if (!norm_shape_ok(batch, dim, seqlen) || !(eps >= 0.0f) || !std::isfinite(eps)) return SSM_ERR_SHAPE;
  const bool empty = batch == 0 || seqlen == 0;
  if (!empty && (!x || !weight || !y || (residual == nullptr) != (sum_out == nullptr))) return SSM_ERR_NULL;
  const size_t es = (size_t)elem_bytes(dtype);
  if (!aligned(x, es) || !aligned(residual, es) || !aligned(y, es) || !aligned(sum_out, es) ||
      !aligned(weight, 4) || !aligned(bias, 4) || !aligned(mean, 4) || !aligned(rstd, 4))
    return SSM_ERR_ALIGN;
  if (empty) return SSM_OK;
  const size_t tokens = (size_t)batch * (size_t)seqlen, all = tokens * (size_t)dim * es, ch = (size_t)dim * 4;
  const Span outs[] = {span(y, all), span(sum_out, all), span(mean, tokens * 4), span(rstd, tokens * 4)};
  const Span ins[] = {span(x, all), span(residual, all), span(weight, ch), span(bias, ch)};
  if (writes_overlap(outs, ins)) return SSM_ERR_ALIAS;
  NormLaunch a{};
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.bias = bias;
  a.eps = eps;
  a.y = y;
  a.sum_out = sum_out;
  a.mean = mean;
  a.rstd = rstd;
  a.batch = batch;
  a.dim = dim;
  a.seqlen = seqlen;
  a.dtype = dtype_of(dtype);
  return status_of(launch_norm_fwd(a, static_cast<hipStream_t>(stream)));
}

size_t ssm_layer_norm_bwd_workspace_bytes(int batch, int dim, int64_t seqlen, int dtype) {
  if (!dtype_ok(dtype) || !norm_shape_ok(batch, dim, seqlen) || batch == 0 || seqlen == 0) return 0;
  return norm_bwd_ws_bytes(batch, dim, seqlen, dtype);
}

int ssm_layer_norm_bwd(const void* s, const float* weight, const float* mean, const float* rstd, const void* dy,
                       const void* dsum, void* dx, float* dweight, float* dbias, int batch, int dim,
                       int64_t seqlen, int dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (!dtype_ok(dtype)) return SSM_ERR_DTYPE;
  if (!norm_shape_ok(batch, dim, seqlen)) return SSM_ERR_SHAPE;
  if (!dweight) return SSM_ERR_NULL;
  const bool empty = batch == 0 || seqlen == 0;
  if (!empty && (!s || !weight || !mean || !rstd || !dy || !dx)) return SSM_ERR_NULL;
  const size_t es = (size_t)elem_bytes(dtype);
  if (!aligned(s, es) || !aligned(dy, es) || !aligned(dsum, es) || !aligned(dx, es) || !aligned(weight, 4) ||
      !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(dweight, 4) || !aligned(dbias, 4) ||
      !aligned(workspace, 256))
    return SSM_ERR_ALIGN;
  const size_t need = empty ? 0 : norm_bwd_ws_bytes(batch, dim, seqlen, dtype);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return SSM_ERR_WORKSPACE;
  const size_t tokens = (size_t)batch * (size_t)seqlen, all = tokens * (size_t)dim * es, ch = (size_t)dim * 4;
  const Span outs[] = {span(dx, all), span(dweight, ch), span(dbias, ch), span(workspace, need)};
  const Span ins[] = {span(s, all), span(dy, all), span(dsum, all), span(weight, ch),
                      span(mean, tokens * 4), span(rstd, tokens * 4)};
  if (writes_overlap(outs, ins)) return SSM_ERR_ALIAS;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (empty) {
    hipError_t e = launch_fill_state(dweight, nullptr, dim, st);
    if (e == hipSuccess && dbias != nullptr) e = launch_fill_state(dbias, nullptr, dim, st);
    return status_of(e);
  }
  NormLaunch a{};
  a.x = s;
  a.weight = weight;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.dy = dy;
  a.dsum = dsum;
  a.dx = dx;
  a.dweight = dweight;
  a.dbias = dbias;
  a.part = static_cast<float*>(workspace);
  a.batch = batch;
  a.dim = dim;
  a.seqlen = seqlen;
  a.dtype = dtype_of(dtype);
  return status_of(launch_norm_bwd(a, st));
}

}  // extern "C"
