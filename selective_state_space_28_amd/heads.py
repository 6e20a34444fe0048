"""torch-tensor wrappers of the linear attention (include/ssm_linear_attn.h) and
the group norm (include/ssm_group_norm.h): marshalling only, as in ops.py."""
from __future__ import annotations

import ctypes

import torch

from ._lib import SSM_ACT_NONE, SSM_ACT_SIGMOID, SSM_ACT_SILU, load
from .layers import _F32, _call, _gpu, _in, _int32, _workspace
from .ops import _DTYPES, _check, _code, _ptr

_ACTS = {"none": SSM_ACT_NONE, "silu": SSM_ACT_SILU, "sigmoid": SSM_ACT_SIGMOID}
_MAX_WIDTH = 256


def _refuse(name, t, lead, width, dtype, dev):
    """What is wrong with an operand (*lead, heads, width), as an error."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dim() != len(lead) + 2 or t.shape[:-2] != lead or (width is not None and t.shape[-1] != width):
        wide = "width" if width is None else width
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(*lead, 'heads', wide)}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must be contiguous along its last axis")


def _heads_in(q, k, v, log_decay, lead, dev):
    """(addresses of q, k, v; host array of their strides or None; heads and widths; address of log_decay)."""
    dt, idx = q.dtype, dev.index
    if k is None or v is None or log_decay is None:
        raise ValueError("q, k, v and log_decay are required")
    qs, ks, vs, gs = q.shape, k.shape, v.shape, log_decay.shape
    # (a token's call is mostly host time: what fits is seen to at once)
    whole = q.is_contiguous() and k.is_contiguous() and v.is_contiguous()
    if not (whole and k.dtype is dt and v.dtype is dt and k.get_device() == idx and v.get_device() == idx
            and len(ks) == len(qs) and len(vs) == len(qs) and ks[:-2] == lead and vs[:-2] == lead and ks[-1] == qs[-1]):
        _refuse("q", q, lead, None, dt, dev)
        _refuse("k", k, lead, qs[-1], dt, dev)
        _refuse("v", v, lead, None, dt, dev)
    if len(gs) != 1:
        raise ValueError("log_decay must be (heads,)")
    heads, hq, hk, hv, kd, vd = gs[0], qs[-2], ks[-2], vs[-2], qs[-1], vs[-1]
    pg = _in("log_decay", log_decay, gs, _F32, dev)
    if not (hq == hk == hv == heads < 2 ** 31 and 1 <= kd <= _MAX_WIDTH and 1 <= vd <= _MAX_WIDTH):
        _int32("heads", heads)
        for name, n in (("q", hq), ("k", hk), ("v", hv)):
            if heads > 0 and (n < 1 or heads % n != 0):
                raise ValueError(f"{name} has {n} heads, which do not divide the {heads} of log_decay")
        for name, n in (("q and k", kd), ("v", vd)):
            if not 1 <= n <= _MAX_WIDTH:
                raise ValueError(f"{name} are {n} wide, not 1 to {_MAX_WIDTH}")
    strides = None
    if not whole:
        steps = q.stride()[:-1] + k.stride()[:-1] + v.stride()[:-1]
        strides = (ctypes.c_int64 * len(steps))(*steps)
    return (q.data_ptr(), k.data_ptr(), v.data_ptr()), strides, (heads, hq, hk, hv, kd, vd), pg


def _scale(scale, kd):
    return kd ** -0.5 if scale is None else float(scale)


def _starts_in(starts, shape, dev):
    if starts is None:
        return None
    if starts.dtype not in (torch.uint8, torch.bool):
        raise TypeError(f"starts has dtype {starts.dtype}, expected uint8 or bool")
    _check("starts", starts, shape, starts.dtype, dev)
    return starts.data_ptr()


def _rows_in(q, starts, lengths, dev):
    if q.dim() != 4:
        raise ValueError(f"q must be (batch, seqlen, heads, width), not {tuple(q.shape)}")
    lead = q.shape[:2]
    _int32("batch", lead[0])
    return lead, _starts_in(starts, lead, dev), _in("lengths", lengths, lead[:1], torch.int32, dev, required=False)


def ssm_linear_attn_fwd_workspace_bytes(batch: int, seqlen: int, heads: int, key_dim: int, value_dim: int,
                                        dtype: torch.dtype) -> int:
    return int(load().ssm_linear_attn_fwd_workspace_bytes(batch, seqlen, heads, key_dim, value_dim, _DTYPES[dtype]))


def ssm_linear_attn_fwd(q, k, v, log_decay, *, scale=None, starts=None, lengths=None, h0=None,
                        return_last_state=False, out=None, workspace=None):
    """Linear attention S = exp(log_decay) S + k v^T, y = scale q S over whole
    sequences; see include/ssm_linear_attn.h.

    q: (batch, L, q_heads, key_dim), k: (batch, L, k_heads, key_dim), v: (batch,
    L, v_heads, value_dim), float32 or bfloat16 (one dtype for all), any strides
    with the widths contiguous; log_decay: (heads,) float32, of which each number
    of heads is a divisor (shared by consecutive ones).  scale: 1/sqrt(key_dim)
    by default.  starts: (batch, L) uint8 or bool, set at the first step of each
    sequence packed into a row; lengths: (batch,) int32, the steps of each row of
    a padded batch (y is 0 behind them); h0: (batch, heads, key_dim, value_dim)
    float32.  Returns y (batch, L, heads, value_dim), then last_state (if
    return_last_state)."""
    lib = load()
    dev = _gpu(q)
    code = _code(q)
    lead, ps, pl = _rows_in(q, starts, lengths, dev)
    ins, strides, sizes, pg = _heads_in(q, k, v, log_decay, lead, dev)
    batch, L = lead
    heads, _, _, _, kd, vd = sizes
    state = (batch, heads, kd, vd)
    p0 = _in("h0", h0, state, _F32, dev, required=False)
    y = out if out is not None else torch.empty((batch, L, heads, vd), dtype=q.dtype, device=dev)
    py = _in("out", y, (batch, L, heads, vd), q.dtype, dev)
    last = torch.empty(state, dtype=_F32, device=dev) if return_last_state else None
    workspace, ws_bytes = _workspace(workspace, lib.ssm_linear_attn_fwd_workspace_bytes(batch, L, heads, kd, vd, code), dev)
    _call(lib.ssm_linear_attn_fwd, "ssm_linear_attn_fwd", dev, *ins, strides, pg, _scale(scale, kd), ps, pl, p0, py,
          _ptr(last), batch, L, *sizes, code, _ptr(workspace), ws_bytes)
    return (y, last) if return_last_state else y


def ssm_linear_attn_bwd_workspace_bytes(batch: int, seqlen: int, heads: int, q_heads: int, k_heads: int, v_heads: int,
                                        key_dim: int, value_dim: int, dtype: torch.dtype) -> int:
    return int(load().ssm_linear_attn_bwd_workspace_bytes(batch, seqlen, heads, q_heads, k_heads, v_heads, key_dim,
                                                          value_dim, _DTYPES[dtype]))


def ssm_linear_attn_bwd(q, k, v, log_decay, *, scale=None, starts=None, lengths=None, h0=None, dy, dlast_state=None,
                        decay_grad=True, workspace=None):
    """Gradients through ssm_linear_attn_fwd, called with the same inputs, from
    dy = dL/dy and optionally dL/dlast_state.  Returns a dict: dq, dk, dv in the
    shapes and the dtype of q, k and v (contiguous; of shared heads the sums),
    dlog_decay (heads,) float32 (None without decay_grad) and dh0 float32 (None
    without h0)."""
    lib = load()
    dev = _gpu(q)
    code = _code(q)
    lead, ps, pl = _rows_in(q, starts, lengths, dev)
    ins, strides, sizes, pg = _heads_in(q, k, v, log_decay, lead, dev)
    batch, L = lead
    heads, hq, hk, hv, kd, vd = sizes
    state = (batch, heads, kd, vd)
    p0 = _in("h0", h0, state, _F32, dev, required=False)
    pdy = _in("dy", dy, (batch, L, heads, vd), q.dtype, dev)
    pdl = _in("dlast_state", dlast_state, state, _F32, dev, required=False)

    def like(t):
        return torch.empty(t.shape, dtype=t.dtype, device=dev)

    g = dict(dq=like(q), dk=like(k), dv=like(v), dlog_decay=like(log_decay) if decay_grad else None,
             dh0=torch.empty(state, dtype=_F32, device=dev) if h0 is not None else None)
    workspace, ws_bytes = _workspace(
        workspace, lib.ssm_linear_attn_bwd_workspace_bytes(batch, L, *sizes, code), dev)
    _call(lib.ssm_linear_attn_bwd, "ssm_linear_attn_bwd", dev, *ins, strides, pg, _scale(scale, kd), ps, pl, p0, pdy, pdl,
          _ptr(g["dq"]), _ptr(g["dk"]), _ptr(g["dv"]), _ptr(g["dlog_decay"]), _ptr(g["dh0"]), batch, L, *sizes, code,
          _ptr(workspace), ws_bytes)
    return g


def ssm_linear_attn_state_update(state, q, k, v, log_decay, *, scale=None, starts=None, out=None, state_out=None):
    """One token of the linear attention: state (batch, heads, key_dim,
    value_dim) float32 is updated in place, or kept and the new one written to
    state_out.  q, k, v: (batch, their heads, width); starts: (batch,), set where
    the token is its sequence's first.  Returns y (batch, heads, value_dim)."""
    lib = load()
    dev = _gpu(q)
    code = _code(q)
    lead = q.shape[:1]
    if q.dim() != 3:
        raise ValueError(f"q must be (batch, heads, width), not {tuple(q.shape)}")
    batch = _int32("batch", lead[0])
    ps = _starts_in(starts, lead, dev)
    ins, strides, sizes, pg = _heads_in(q, k, v, log_decay, lead, dev)
    heads, _, _, _, kd, vd = sizes
    shape = (batch, heads, kd, vd)
    p0 = _in("state", state, shape, _F32, dev)
    po = _in("state_out", state_out, shape, _F32, dev, required=False)
    if out is None:  # (a third quicker than empty with a shape)
        y = torch.empty_like(v) if strides is None and sizes[3] == heads else torch.empty((batch, heads, vd), dtype=q.dtype,
                                                                                          device=dev)
        py = y.data_ptr()
    else:
        y, py = out, _in("out", out, (batch, heads, vd), q.dtype, dev)
    _call(lib.ssm_linear_attn_state_update, "ssm_linear_attn_state_update", dev, p0, *ins, strides, pg, _scale(scale, kd),
          ps, py, po, batch, *sizes, code)
    return y


def _rows(name, t, shape, dtype, dev):
    """The address of (..., dim) rows and the elements from one to the next."""
    if t.is_contiguous():
        return _in(name, t, shape, dtype, dev), shape[-1]
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    row = None  # of the axes with more than one entry the last's stride, the others' its multiples
    step = 0
    for n, s in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if row is None:
            row, step = s, s * n
        elif s == step:
            step = s * n
        else:
            row = -1
            break
    if row is None:
        row = shape[-1]
    if row < shape[-1] or (t.stride(-1) != 1 and shape[-1] > 1):
        raise ValueError(f"{name} must be rows of contiguous channels, one stride apart")
    return t.data_ptr(), row


def _group_sizes(x, groups):
    if x.dim() < 1:
        raise ValueError("x must be (..., dim)")
    dim = _int32("dim", x.shape[-1])
    if groups < 1 or dim < 1 or dim % groups != 0:
        raise ValueError(f"{groups} groups do not divide {dim} channels")
    tokens = 1
    for n in x.shape[:-1]:
        tokens *= n
    return tokens, dim


def _act(act):
    if act not in _ACTS:
        raise ValueError(f"act must be 'none', 'silu' or 'sigmoid', not {act!r}")
    return _ACTS[act]


def ssm_group_norm_fwd(x, groups, weight=None, bias=None, z=None, *, act="none", eps=1e-5, return_stats=False, out=None):
    """The norm of each of `groups` groups of x's channels (last axis), then
    act, or with z the product with act(z); see include/ssm_group_norm.h.

    x, z: (..., dim) float32 or bfloat16, z x's shape; each may be a block of the
    channels of a wider tensor (rows of contiguous channels, one stride apart);
    weight, bias: (dim,) float32; act: "none", "silu" or "sigmoid".  Returns y,
    then mean and rstd (if return_stats), float32 (..., groups)."""
    lib = load()
    dev = _gpu(x)
    code = _code(x)
    tokens, dim = _group_sizes(x, groups)
    shape, dt = x.shape, x.dtype
    px, xs = _rows("x", x, shape, dt, dev)
    pz, zs = _rows("z", z, shape, dt, dev) if z is not None else (None, 0)
    pw = _in("weight", weight, (dim,), _F32, dev, required=False)
    pb = _in("bias", bias, (dim,), _F32, dev, required=False)
    if out is None:
        y = torch.empty_like(x) if xs == dim and x.is_contiguous() else torch.empty(shape, dtype=dt, device=dev)
        py = y.data_ptr()
    else:
        y, py = out, _in("out", out, shape, dt, dev)
    mean = rstd = None
    if return_stats:
        mean = torch.empty((*shape[:-1], groups), dtype=_F32, device=dev)
        rstd = torch.empty_like(mean)
    _call(lib.ssm_group_norm_fwd, "ssm_group_norm_fwd", dev, px, xs, pw, pb, pz, zs, _act(act), eps, py, _ptr(mean),
          _ptr(rstd), tokens, dim, groups, code)
    return (y, mean, rstd) if return_stats else y


def ssm_group_norm_bwd_workspace_bytes(tokens: int, dim: int, groups: int, dtype: torch.dtype) -> int:
    return int(load().ssm_group_norm_bwd_workspace_bytes(tokens, dim, groups, _DTYPES[dtype]))


def ssm_group_norm_bwd(x, groups, weight=None, bias=None, z=None, *, act="none", mean, rstd, dy, workspace=None):
    """Gradients through ssm_group_norm_fwd, called with the same inputs, from
    the mean and rstd it returned.  Returns a dict: dx, dz (None without z) in
    the input dtype, contiguous; dweight, dbias float32 (None where the parameter
    is)."""
    lib = load()
    dev = _gpu(x)
    code = _code(x)
    tokens, dim = _group_sizes(x, groups)
    shape, dt = x.shape, x.dtype
    px, xs = _rows("x", x, shape, dt, dev)
    pz, zs = _rows("z", z, shape, dt, dev) if z is not None else (None, 0)
    pw = _in("weight", weight, (dim,), _F32, dev, required=False)
    pb = _in("bias", bias, (dim,), _F32, dev, required=False)
    pm = _in("mean", mean, (*shape[:-1], groups), _F32, dev)
    pr = _in("rstd", rstd, (*shape[:-1], groups), _F32, dev)
    pdy = _in("dy", dy, shape, dt, dev)
    act = _act(act)
    g = dict(dx=torch.empty(shape, dtype=dt, device=dev),
             dz=torch.empty(shape, dtype=dt, device=dev) if z is not None else None,
             dweight=torch.empty_like(weight) if weight is not None else None,
             dbias=torch.empty_like(bias) if bias is not None else None)
    need = 0
    if weight is not None or bias is not None:
        need = lib.ssm_group_norm_bwd_workspace_bytes(tokens, dim, groups, code)
    workspace, ws_bytes = _workspace(workspace, need, dev)
    _call(lib.ssm_group_norm_bwd, "ssm_group_norm_bwd", dev, px, xs, pw, pb, pz, zs, act, pm, pr, pdy, _ptr(g["dx"]),
          _ptr(g["dz"]), _ptr(g["dweight"]), _ptr(g["dbias"]), tokens, dim, groups, code, _ptr(workspace), ws_bytes)
    return g
