// heads_api.cpp -- the C ABI of the linear attention (include/ssm_linear_attn.h) and
// of the group norm (include/ssm_group_norm.h): argument validation and the calls
// into the kernels.  Every check happens before the first HIP call.
#include <climits>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "api_checks.hpp"
#include "linear_attn.hpp"
#include "ssm_group_norm.h"
#include "ssm_kernels.hpp"
#include "ssm_linear_attn.h"

namespace {

using namespace ssm;

static_assert(SSM_LINEAR_ATTN_MAX_DIM == kAttnMaxWidth, "the widest head of the kernels");

bool dtype_ok(int dtype) { return dtype == SSM_F32 || dtype == SSM_BF16; }

Dtype dtype_of(int dtype) { return dtype == SSM_BF16 ? Dtype::BF16 : Dtype::F32; }

int status_of(hipError_t e) { return e == hipSuccess ? SSM_OK : SSM_ERR_HIP; }

struct AttnSizes {
  int batch;
  int64_t seqlen;
  int heads, hq, hk, hv, kd, vd;
};

bool attn_shape_ok(const AttnSizes& s) {
  if (s.batch < 0 || s.heads < 0 || s.seqlen < 0 || s.seqlen > kMaxSeqlen) return false;
  if (s.kd < 1 || s.kd > kAttnMaxWidth || s.vd < 1 || s.vd > kAttnMaxWidth) return false;
  if (s.hq < 1 || s.hk < 1 || s.hv < 1 || s.heads % s.hq || s.heads % s.hk || s.heads % s.hv) return false;
  if ((int64_t)s.batch * s.heads > kMaxSeqlen) return false;
  const long double steps = (long double)s.batch * (long double)(s.seqlen > 0 ? s.seqlen : 1);
  return steps * (long double)(s.heads > 0 ? s.heads : 1) * kAttnMaxWidth < (long double)(INT64_C(1) << 60);
}

// The strides of an operand, the caller's or those of a contiguous one; false
// where they cannot be.  `steps` false: (batch, head) alone.
constexpr int64_t kMaxStride = INT64_C(1) << 40;

bool attn_view(AttnView& w, const void* p, const int64_t* strides, bool steps, int batch, int64_t seqlen, int n, int heads,
               int width) {
  w.p = p;
  w.share = n > 0 ? heads / n : 1;
  if (strides == nullptr) {
    w.sh = width;
    w.st = (int64_t)n * width;
    w.sb = steps ? w.st * seqlen : w.st;
    return true;
  }
  w.sb = strides[0];
  w.st = steps ? strides[1] : 0;
  w.sh = strides[steps ? 2 : 1];
  if (w.sb < 0 || w.st < 0 || w.sh < 0 || w.sb > kMaxStride || w.st > kMaxStride || w.sh > kMaxStride) return false;
  // (a stride that is never taken does not keep the operand from being read in vectors)
  if (batch <= 1) w.sb = 0;
  if (seqlen <= 1) w.st = 0;
  if (n == 1) w.sh = 0;
  return true;
}

// Whether an operand's last element is within 2^60 of its first, and the bytes that it spans.
bool attn_extent_ok(const AttnView& w, int batch, int64_t seqlen, int n, int width) {
  const long double e = (long double)w.sb * (batch - 1) + (long double)w.st * (seqlen - 1) + (long double)w.sh * (n - 1) + width;
  return e < (long double)(INT64_C(1) << 60);
}

Span attn_span(const AttnView& w, int batch, int64_t seqlen, int n, int width, size_t es) {
  return span(w.p, (size_t)(w.sb * (batch - 1) + w.st * (seqlen - 1) + w.sh * (n - 1) + width) * es);
}

// Workspace of one sweep: the states entering the segments, and what they leave of
// them; of the decay's gradient also their derivatives, and the segments' steps.
struct SweepBytes {
  size_t state, through, rate, steps, part;
  size_t all() const { return state + through + rate + steps + part; }
};

// The segments of n sweeps side by side; of the decay's gradient two states each.
AttnSplit split_of(const AttnSizes& s, int blocks, int n, bool decay, int dtype) {
  const int64_t heads = (int64_t)n * s.batch * s.heads;
  return attn_split(heads * blocks, s.seqlen, heads * s.kd * s.vd * (decay ? 2 : 1), dtype_of(dtype));
}

SweepBytes sweep_bytes(const AttnSizes& s, int blocks, int n, bool decay, int dtype) {
  SweepBytes w{};
  const AttnSplit sp = split_of(s, blocks, n, decay, dtype);
  const size_t segs = (size_t)s.batch * (size_t)s.heads * (size_t)sp.nseg;
  if (sp.nseg > 1) {
    w.state = round256(segs * (size_t)s.kd * (size_t)s.vd * 4);
    w.through = round256(segs * 4);
    if (decay) {
      w.rate = w.state;
      w.steps = w.through;
    }
  }
  if (decay) w.part = round256(segs * (size_t)blocks * 8);
  return w;
}

// Of the backward: the sweeps' (dq and dk, with dv where the widths are alike, side by
// side; what follows in the same place), then the heads' gradients (float32) where
// several share one.
struct BwdBytes {
  size_t sweep, dq, dk, dv;
  size_t all() const { return sweep + dq + dk + dv; }
};

int sweeps_together(const AttnSizes& s) { return attn_alike(s.kd, s.vd) ? 3 : 2; }

BwdBytes bwd_bytes(const AttnSizes& s, int dtype) {
  const size_t steps = (size_t)s.batch * (size_t)s.seqlen * (size_t)s.heads * 4;
  const int n = sweeps_together(s);
  BwdBytes w{};
  for (const size_t b : {(size_t)n * sweep_bytes(s, attn_column_blocks(s.kd), n, false, dtype).all(),
                         n == 3 ? (size_t)0 : sweep_bytes(s, attn_column_blocks(s.vd), 1, false, dtype).all(),
                         sweep_bytes(s, attn_decay_blocks(s.vd), 1, true, dtype).all()})
    w.sweep = w.sweep > b ? w.sweep : b;
  if (s.hq != s.heads) w.dq = round256(steps * (size_t)s.kd);
  if (s.hk != s.heads) w.dk = round256(steps * (size_t)s.kd);
  if (s.hv != s.heads) w.dv = round256(steps * (size_t)s.vd);
  return w;
}

// The k-th of n sweeps with contraction width kd and value width vd over the workspace.
AttnSweep attn_sweep(const AttnSizes& s, const float* g, const uint8_t* starts, const int32_t* lengths, int dtype, int kd,
                     int vd, void* workspace, int k, int n, bool decay = false) {
  AttnSweep a{};
  const int blocks = decay ? attn_decay_blocks(vd) : attn_column_blocks(vd);
  const AttnSplit sp = split_of(s, blocks, n, decay, dtype);
  const SweepBytes w = sweep_bytes(s, blocks, n, decay, dtype);
  a.kd = kd;
  a.vd = vd;
  a.batch = s.batch;
  a.heads = s.heads;
  a.seqlen = s.seqlen;
  a.g = g;
  a.starts = starts;
  a.lengths = lengths;
  a.nseg = sp.nseg;
  a.seglen = sp.seglen;
  char* p = static_cast<char*>(workspace) + (size_t)k * w.all();
  a.seg_state = reinterpret_cast<float*>(p);
  a.seg_through = reinterpret_cast<float*>(p + w.state);
  a.seg_rate = reinterpret_cast<float*>(p + w.state + w.through);
  a.seg_steps = reinterpret_cast<float*>(p + w.state + w.through + w.rate);
  a.part = reinterpret_cast<double*>(p + w.state + w.through + w.rate + w.steps);
  a.dtype = dtype_of(dtype);
  return a;
}

bool group_shape_ok(int64_t tokens, int dim, int groups) {
  return tokens >= 0 && dim >= 1 && groups >= 1 && dim % groups == 0 && dim / groups <= SSM_GROUP_NORM_MAX_WIDTH &&
         dim <= INT_MAX - 65536 && tokens <= kMaxSeqlen / groups;
}

// Rows of `stride` elements: of at most 2^31 - 1, and not overlapping.
bool row_stride_ok(int64_t stride, int dim) { return stride >= dim && stride <= INT_MAX; }

Span row_span(const void* p, int64_t stride, int64_t tokens, int dim, size_t es) {
  return span(p, ((size_t)stride * (size_t)(tokens - 1) + (size_t)dim) * es);
}

bool act_ok(int act) { return act == SSM_ACT_NONE || act == SSM_ACT_SILU || act == SSM_ACT_SIGMOID; }

size_t group_ws_bytes(int64_t tokens, int dim, int groups) {
  return round256((size_t)group_norm_bwd_parts(tokens, dim, groups) * 2 * (size_t)dim * sizeof(float));
}

GroupNormLaunch group_launch(const void* x, int64_t x_stride, const float* weight, const float* bias, const void* z,
                             int64_t z_stride, int act, int64_t tokens, int dim, int groups, int dtype) {
  GroupNormLaunch a{};
  a.x = x;
  a.x_stride = x_stride;
  a.weight = weight;
  a.bias = bias;
  a.z = z;
  a.z_stride = z_stride;
  a.act = act;
  a.tokens = tokens;
  a.dim = dim;
  a.groups = groups;
  a.width = dim / groups;
  a.dtype = dtype_of(dtype);
  return a;
}

}  // namespace

extern "C" {

size_t ssm_linear_attn_fwd_workspace_bytes(int batch, int64_t seqlen, int heads, int key_dim, int value_dim, int dtype) {
  const AttnSizes s{batch, seqlen, heads, 1, 1, 1, key_dim, value_dim};
  if (!dtype_ok(dtype) || !attn_shape_ok(s) || batch == 0 || heads == 0 || seqlen == 0) return 0;
  return sweep_bytes(s, attn_column_blocks(value_dim), 1, false, dtype).all();
}

int ssm_linear_attn_fwd(const void* q, const void* k, const void* v, const int64_t* strides, const float* log_decay,
                        float scale, const uint8_t* starts, const int32_t* lengths, const float* h0, void* y,
                        float* last_state, int batch, int64_t seqlen, int heads, int q_heads, int k_heads, int v_heads,
                        int key_dim, int value_dim, int dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (!dtype_ok(dtype)) return SSM_ERR_DTYPE;
  const AttnSizes s{batch, seqlen, heads, q_heads, k_heads, v_heads, key_dim, value_dim};
  if (!attn_shape_ok(s) || !std::isfinite(scale)) return SSM_ERR_SHAPE;
  AttnView vq, vk, vv;
  if (!attn_view(vq, q, strides, true, batch, seqlen, q_heads, heads, key_dim) ||
      !attn_view(vk, k, strides ? strides + 3 : nullptr, true, batch, seqlen, k_heads, heads, key_dim) ||
      !attn_view(vv, v, strides ? strides + 6 : nullptr, true, batch, seqlen, v_heads, heads, value_dim))
    return SSM_ERR_SHAPE;
  const bool none = batch == 0 || heads == 0, empty = none || seqlen == 0;
  if (!empty && (!attn_extent_ok(vq, batch, seqlen, q_heads, key_dim) || !attn_extent_ok(vk, batch, seqlen, k_heads, key_dim) ||
                 !attn_extent_ok(vv, batch, seqlen, v_heads, value_dim)))
    return SSM_ERR_SHAPE;
  if (!empty && (!q || !k || !v || !log_decay || !y)) return SSM_ERR_NULL;
  const size_t es = (size_t)elem_bytes(dtype);
  if (!aligned(q, es) || !aligned(k, es) || !aligned(v, es) || !aligned(y, es) || !aligned(log_decay, 4) ||
      !aligned(lengths, 4) || !aligned(h0, 4) || !aligned(last_state, 4) || !aligned(workspace, 256))
    return SSM_ERR_ALIGN;
  if (none) return SSM_OK;
  const size_t need = empty ? 0 : sweep_bytes(s, attn_column_blocks(value_dim), 1, false, dtype).all();
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return SSM_ERR_WORKSPACE;
  const size_t rows = (size_t)batch * (size_t)seqlen;
  const size_t state = (size_t)batch * (size_t)heads * (size_t)key_dim * (size_t)value_dim * 4;
  {
    const Span outs[] = {span(y, rows * (size_t)heads * (size_t)value_dim * es), span(last_state, state),
                         span(workspace, need)};
    const Span nil{0, 0};
    const Span ins[] = {empty ? nil : attn_span(vq, batch, seqlen, q_heads, key_dim, es),
                        empty ? nil : attn_span(vk, batch, seqlen, k_heads, key_dim, es),
                        empty ? nil : attn_span(vv, batch, seqlen, v_heads, value_dim, es),
                        span(log_decay, (size_t)heads * 4), span(starts, rows), span(lengths, (size_t)batch * 4),
                        span(h0, state)};
    if (writes_overlap(outs, ins)) return SSM_ERR_ALIAS;
  }
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (empty)
    return last_state == nullptr ? SSM_OK : status_of(launch_fill_state(last_state, h0, (int64_t)(state / 4), st));
  AttnSweeps all{};
  all.n = 1;
  AttnSweep& a = all.s[0];
  a = attn_sweep(s, log_decay, starts, lengths, dtype, key_dim, value_dim, workspace, 0, 1);
  a.q = vq;
  a.k = vk;
  a.v = vv;
  a.out = y;
  a.scale_p = scale;
  a.scale_in = scale;
  a.scale_upd = 1.0f;
  a.state_in = h0;
  a.state_out = last_state;
  return status_of(launch_attn_sweeps(all, st));
}

size_t ssm_linear_attn_bwd_workspace_bytes(int batch, int64_t seqlen, int heads, int q_heads, int k_heads, int v_heads,
                                           int key_dim, int value_dim, int dtype) {
  const AttnSizes s{batch, seqlen, heads, q_heads, k_heads, v_heads, key_dim, value_dim};
  if (!dtype_ok(dtype) || !attn_shape_ok(s) || batch == 0 || heads == 0 || seqlen == 0) return 0;
  return bwd_bytes(s, dtype).all();
}

int ssm_linear_attn_bwd(const void* q, const void* k, const void* v, const int64_t* strides, const float* log_decay,
                        float scale, const uint8_t* starts, const int32_t* lengths, const float* h0, const void* dy,
                        const float* dlast_state, void* dq, void* dk, void* dv, float* dlog_decay, float* dh0, int batch,
                        int64_t seqlen, int heads, int q_heads, int k_heads, int v_heads, int key_dim, int value_dim,
                        int dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (!dtype_ok(dtype)) return SSM_ERR_DTYPE;
  const AttnSizes s{batch, seqlen, heads, q_heads, k_heads, v_heads, key_dim, value_dim};
  if (!attn_shape_ok(s) || !std::isfinite(scale)) return SSM_ERR_SHAPE;
  AttnView vq, vk, vv, vdy;
  if (!attn_view(vq, q, strides, true, batch, seqlen, q_heads, heads, key_dim) ||
      !attn_view(vk, k, strides ? strides + 3 : nullptr, true, batch, seqlen, k_heads, heads, key_dim) ||
      !attn_view(vv, v, strides ? strides + 6 : nullptr, true, batch, seqlen, v_heads, heads, value_dim))
    return SSM_ERR_SHAPE;
  attn_view(vdy, dy, nullptr, true, batch, seqlen, heads, heads, value_dim);
  const bool none = batch == 0 || heads == 0, empty = none || seqlen == 0;
  if (!empty && (!attn_extent_ok(vq, batch, seqlen, q_heads, key_dim) || !attn_extent_ok(vk, batch, seqlen, k_heads, key_dim) ||
                 !attn_extent_ok(vv, batch, seqlen, v_heads, value_dim)))
    return SSM_ERR_SHAPE;
  if (!empty && (!q || !k || !v || !log_decay || !dy || !dq || !dk || !dv)) return SSM_ERR_NULL;
  const size_t es = (size_t)elem_bytes(dtype);
  if (!aligned(q, es) || !aligned(k, es) || !aligned(v, es) || !aligned(dy, es) || !aligned(dq, es) || !aligned(dk, es) ||
      !aligned(dv, es) || !aligned(log_decay, 4) || !aligned(lengths, 4) || !aligned(h0, 4) || !aligned(dlast_state, 4) ||
      !aligned(dlog_decay, 4) || !aligned(dh0, 4) || !aligned(workspace, 256))
    return SSM_ERR_ALIGN;
  if (heads == 0) return SSM_OK;
  const BwdBytes w = empty ? BwdBytes{} : bwd_bytes(s, dtype);
  const size_t need = w.all();
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return SSM_ERR_WORKSPACE;
  const size_t rows = (size_t)batch * (size_t)seqlen;
  const size_t state = (size_t)batch * (size_t)heads * (size_t)key_dim * (size_t)value_dim * 4;
  {
    const Span outs[] = {span(dq, rows * (size_t)q_heads * (size_t)key_dim * es),
                         span(dk, rows * (size_t)k_heads * (size_t)key_dim * es),
                         span(dv, rows * (size_t)v_heads * (size_t)value_dim * es), span(dlog_decay, (size_t)heads * 4),
                         span(dh0, state), span(workspace, need)};
    const Span nil{0, 0};
    const Span ins[] = {empty ? nil : attn_span(vq, batch, seqlen, q_heads, key_dim, es),
                        empty ? nil : attn_span(vk, batch, seqlen, k_heads, key_dim, es),
                        empty ? nil : attn_span(vv, batch, seqlen, v_heads, value_dim, es),
                        span(dy, rows * (size_t)heads * (size_t)value_dim * es), span(log_decay, (size_t)heads * 4),
                        span(starts, rows), span(lengths, (size_t)batch * 4), span(h0, state), span(dlast_state, state)};
    if (writes_overlap(outs, ins)) return SSM_ERR_ALIAS;
  }
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (empty) {  // nothing was swept: no gradient of the decay, and the state's passes through
    hipError_t e = dlog_decay == nullptr ? hipSuccess : launch_fill_state(dlog_decay, nullptr, heads, st);
    if (e == hipSuccess && dh0 != nullptr && batch > 0) e = launch_fill_state(dh0, dlast_state, (int64_t)(state / 4), st);
    return status_of(e);
  }
  char* ws = static_cast<char*>(workspace);
  float* part_q = reinterpret_cast<float*>(ws + w.sweep);
  float* part_k = reinterpret_cast<float*>(ws + w.sweep + w.dq);
  float* part_v = reinterpret_cast<float*>(ws + w.sweep + w.dq + w.dk);

  const int n = sweeps_together(s);
  AttnSweeps all{}, last{};
  all.n = n;
  last.n = 1;
  // dq: forward in time, the state transposed
  AttnSweep& a = all.s[0];
  a = attn_sweep(s, log_decay, starts, lengths, dtype, value_dim, key_dim, ws, 0, n);
  a.q = vdy;
  a.k = vv;
  a.v = vk;
  a.out_f32 = w.dq > 0;
  a.out = a.out_f32 ? part_q : dq;
  a.scale_p = scale;
  a.scale_in = scale;
  a.scale_upd = 1.0f;
  a.state_in = h0;
  a.transposed = 1;
  // dk: backward in time, the state's gradient transposed
  AttnSweep& ak = all.s[1];
  ak = attn_sweep(s, log_decay, starts, lengths, dtype, value_dim, key_dim, ws, 1, n);
  ak.q = vv;
  ak.k = vdy;
  ak.v = vq;
  ak.out_f32 = w.dk > 0;
  ak.out = ak.out_f32 ? part_k : dk;
  ak.scale_p = scale;
  ak.scale_in = 1.0f;
  ak.scale_upd = scale;
  ak.state_in = dlast_state;
  ak.transposed = 1;
  ak.rev = 1;
  // dv: backward in time
  AttnSweep& av = n == 3 ? all.s[2] : last.s[0];
  av = attn_sweep(s, log_decay, starts, lengths, dtype, key_dim, value_dim, ws, n == 3 ? 2 : 0, n == 3 ? 3 : 1);
  av.q = vk;
  av.k = vq;
  av.v = vdy;
  av.out_f32 = w.dv > 0;
  av.out = av.out_f32 ? part_v : dv;
  av.scale_p = scale;
  av.scale_in = 1.0f;
  av.scale_upd = scale;
  av.state_in = dlast_state;
  av.state_out = dh0;
  av.rev = 1;
  hipError_t e = launch_attn_sweeps(all, st);
  if (e == hipSuccess && n != 3) e = launch_attn_sweeps(last, st);
  if (e == hipSuccess && w.dq > 0) e = launch_attn_gather(part_q, dq, (int64_t)rows, heads, q_heads, key_dim, a.dtype, st);
  if (e == hipSuccess && w.dk > 0) e = launch_attn_gather(part_k, dk, (int64_t)rows, heads, k_heads, key_dim, a.dtype, st);
  if (e == hipSuccess && w.dv > 0) e = launch_attn_gather(part_v, dv, (int64_t)rows, heads, v_heads, value_dim, a.dtype, st);

  if (e == hipSuccess && dlog_decay != nullptr) {
    AttnSweep d = attn_sweep(s, log_decay, starts, lengths, dtype, key_dim, value_dim, ws, 0, 1, true);
    d.q = vq;
    d.k = vk;
    d.v = vv;
    d.dy = vdy;
    d.scale_p = scale;
    d.scale_in = scale;
    d.scale_upd = 1.0f;
    d.state_in = h0;
    e = launch_attn_decay_grad(d, dlast_state, dlog_decay, st);
  }
  return status_of(e);
}

int ssm_linear_attn_state_update(float* state, const void* q, const void* k, const void* v, const int64_t* strides,
                                 const float* log_decay, float scale, const uint8_t* starts, void* y, float* state_out,
                                 int batch, int heads, int q_heads, int k_heads, int v_heads, int key_dim, int value_dim,
                                 int dtype, void* stream) {
  if (!dtype_ok(dtype)) return SSM_ERR_DTYPE;
  const AttnSizes s{batch, 1, heads, q_heads, k_heads, v_heads, key_dim, value_dim};
  if (!attn_shape_ok(s) || !std::isfinite(scale)) return SSM_ERR_SHAPE;
  AttnStep a{};
  if (!attn_view(a.q, q, strides, false, batch, 1, q_heads, heads, key_dim) ||
      !attn_view(a.k, k, strides ? strides + 2 : nullptr, false, batch, 1, k_heads, heads, key_dim) ||
      !attn_view(a.v, v, strides ? strides + 4 : nullptr, false, batch, 1, v_heads, heads, value_dim))
    return SSM_ERR_SHAPE;
  const bool empty = batch == 0 || heads == 0;
  if (!empty && (!attn_extent_ok(a.q, batch, 1, q_heads, key_dim) || !attn_extent_ok(a.k, batch, 1, k_heads, key_dim) ||
                 !attn_extent_ok(a.v, batch, 1, v_heads, value_dim)))
    return SSM_ERR_SHAPE;
  if (!empty && (!state || !q || !k || !v || !log_decay || !y)) return SSM_ERR_NULL;
  const size_t es = (size_t)elem_bytes(dtype);
  if (!aligned(state, 4) || !aligned(q, es) || !aligned(k, es) || !aligned(v, es) || !aligned(y, es) ||
      !aligned(log_decay, 4) || !aligned(state_out, 4))
    return SSM_ERR_ALIGN;
  if (empty) return SSM_OK;
  if (state_out == nullptr) state_out = state;
  const size_t rows = (size_t)batch * (size_t)heads, bytes = rows * (size_t)key_dim * (size_t)value_dim * 4;
  {
    const Span outs[] = {span(y, rows * (size_t)value_dim * es), span(state_out, bytes)};
    const Span ins[] = {attn_span(a.q, batch, 1, q_heads, key_dim, es), attn_span(a.k, batch, 1, k_heads, key_dim, es),
                        attn_span(a.v, batch, 1, v_heads, value_dim, es), span(log_decay, (size_t)heads * 4),
                        span(starts, (size_t)batch),
                        // in place is each element's own read and write
                        span(state_out != state ? state : nullptr, bytes)};
    if (writes_overlap(outs, ins)) return SSM_ERR_ALIAS;
  }
  a.g = log_decay;
  a.scale = scale;
  a.starts = starts;
  a.state = state;
  a.state_out = state_out;
  a.y = y;
  a.batch = batch;
  a.heads = heads;
  a.kd = key_dim;
  a.vd = value_dim;
  a.dtype = dtype_of(dtype);
  return status_of(launch_attn_step(a, static_cast<hipStream_t>(stream)));
}

int ssm_group_norm_fwd(const void* x, int64_t x_stride, const float* weight, const float* bias, const void* z,
                       int64_t z_stride, int act, float eps, void* y, float* mean, float* rstd, int64_t tokens, int dim,
                       int groups, int dtype, void* stream) {
  if (!dtype_ok(dtype)) return SSM_ERR_DTYPE;
  if (!act_ok(act)) return SSM_ERR_FLAGS;
  if (!group_shape_ok(tokens, dim, groups) || !(eps >= 0.0f) || !std::isfinite(eps) || !row_stride_ok(x_stride, dim) ||
      (z != nullptr && !row_stride_ok(z_stride, dim)))
    return SSM_ERR_SHAPE;
  if (tokens > 0 && (!x || !y)) return SSM_ERR_NULL;
  const size_t es = (size_t)elem_bytes(dtype);
  if (!aligned(x, es) || !aligned(z, es) || !aligned(y, es) || !aligned(weight, 4) || !aligned(bias, 4) ||
      !aligned(mean, 4) || !aligned(rstd, 4))
    return SSM_ERR_ALIGN;
  if (tokens == 0) return SSM_OK;
  const size_t all = (size_t)tokens * (size_t)dim * es, ch = (size_t)dim * 4;
  const size_t stats = (size_t)tokens * (size_t)groups * 4;
  const Span outs[] = {span(y, all), span(mean, stats), span(rstd, stats)};
  const Span ins[] = {row_span(x, x_stride, tokens, dim, es), row_span(z, z_stride, tokens, dim, es), span(weight, ch),
                      span(bias, ch)};
  if (writes_overlap(outs, ins)) return SSM_ERR_ALIAS;
  GroupNormLaunch a = group_launch(x, x_stride, weight, bias, z, z_stride, act, tokens, dim, groups, dtype);
  a.eps = eps;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  return status_of(launch_group_norm_fwd(a, static_cast<hipStream_t>(stream)));
}

size_t ssm_group_norm_bwd_workspace_bytes(int64_t tokens, int dim, int groups, int dtype) {
  if (!dtype_ok(dtype) || !group_shape_ok(tokens, dim, groups) || tokens == 0) return 0;
  return group_ws_bytes(tokens, dim, groups);
}

int ssm_group_norm_bwd(const void* x, int64_t x_stride, const float* weight, const float* bias, const void* z,
                       int64_t z_stride, int act, const float* mean, const float* rstd, const void* dy, void* dx, void* dz,
                       float* dweight, float* dbias, int64_t tokens, int dim, int groups, int dtype, void* workspace,
                       size_t workspace_bytes, void* stream) {
  if (!dtype_ok(dtype)) return SSM_ERR_DTYPE;
  if (!act_ok(act)) return SSM_ERR_FLAGS;
  if (!group_shape_ok(tokens, dim, groups) || !row_stride_ok(x_stride, dim) ||
      (z != nullptr && !row_stride_ok(z_stride, dim)))
    return SSM_ERR_SHAPE;
  if (tokens > 0 && (!x || !mean || !rstd || !dy || !dx || (z && !dz))) return SSM_ERR_NULL;
  const size_t es = (size_t)elem_bytes(dtype);
  if (!aligned(x, es) || !aligned(z, es) || !aligned(dy, es) || !aligned(dx, es) || !aligned(dz, es) ||
      !aligned(weight, 4) || !aligned(bias, 4) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(dweight, 4) ||
      !aligned(dbias, 4) || !aligned(workspace, 256))
    return SSM_ERR_ALIGN;
  const bool sums = dweight != nullptr || dbias != nullptr;
  const size_t need = tokens == 0 || !sums ? 0 : group_ws_bytes(tokens, dim, groups);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return SSM_ERR_WORKSPACE;
  const size_t all = (size_t)tokens * (size_t)dim * es, ch = (size_t)dim * 4;
  const size_t stats = (size_t)tokens * (size_t)groups * 4;
  if (tokens > 0) {
    const Span outs[] = {span(dx, all), span(z != nullptr ? dz : nullptr, all), span(dweight, ch), span(dbias, ch),
                         span(workspace, need)};
    const Span ins[] = {row_span(x, x_stride, tokens, dim, es), row_span(z, z_stride, tokens, dim, es), span(dy, all),
                        span(weight, ch), span(bias, ch), span(mean, stats), span(rstd, stats)};
    if (writes_overlap(outs, ins)) return SSM_ERR_ALIAS;
  } else {
    const Span outs[] = {span(dweight, ch), span(dbias, ch)};
    const Span ins[] = {span(weight, ch), span(bias, ch)};
    if (writes_overlap(outs, ins)) return SSM_ERR_ALIAS;
  }
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (tokens == 0) {
    hipError_t e = dweight == nullptr ? hipSuccess : launch_fill_state(dweight, nullptr, dim, st);
    if (e == hipSuccess && dbias != nullptr) e = launch_fill_state(dbias, nullptr, dim, st);
    return status_of(e);
  }
  GroupNormLaunch a = group_launch(x, x_stride, weight, bias, z, z_stride, act, tokens, dim, groups, dtype);
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.dy = dy;
  a.dx = dx;
  a.dz = dz;
  a.dweight = dweight;
  a.dbias = dbias;
  a.part = sums ? static_cast<float*>(workspace) : nullptr;
  return status_of(launch_group_norm_bwd(a, st));
}

}  // extern "C"
