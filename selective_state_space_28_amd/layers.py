"""torch-tensor wrappers of the gated recurrence (include/ssm_gated.h) and the
layer norm (include/ssm_norm.h): marshalling only, as in ops.py."""
from __future__ import annotations

import torch

from ._lib import SSM_GATE_SOFTPLUS, SSM_GATE_UNIT, SsmError, load
from .ops import _DTYPES, _check, _code, _ptr

CKPT_STEPS = 512
_GATES = {"sigmoid": 0, "softplus": SSM_GATE_SOFTPLUS}
_WEIGHTS = {"convex": 0, "unit": SSM_GATE_UNIT}
_INT_MAX = 2**31 - 1
_F32 = torch.float32


def _rule(gate, weight):
    if gate not in _GATES:
        raise ValueError(f"gate must be 'sigmoid' or 'softplus', not {gate!r}")
    if weight not in _WEIGHTS:
        raise ValueError(f"weight must be 'unit' or 'convex', not {weight!r}")
    return _GATES[gate] | _WEIGHTS[weight]


# The current stream's handle without making a torch.cuda.Stream of it (0.1
# against 1.8 us of a single token's 12).
_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(fn, where, dev, *args):
    """The entry point on the tensors' device and its current stream.  (A
    launch goes to the current device, so another one is made current for it.)"""
    if dev.index == torch.cuda.current_device():
        rc = fn(*args, _stream(dev.index))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _stream(dev.index))
    if rc != 0:
        raise SsmError(rc, where)


def _gpu(x):
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("libssm runs on the GPU: tensors must be on a cuda device")
    return dev


# A token's call is mostly host time, so its tensors are looked at quickly here;
# what does not fit goes to _check, which says why.
def _ok(t, shape, dtype, idx):
    return t.dtype is dtype and t.shape == shape and t.get_device() == idx and t.is_contiguous()


def _in(name, t, shape, dtype, dev, required=True):
    """The address of a tensor that fits, None for None; else _check's error."""
    if t is None:
        if required:
            raise ValueError(f"{name} is required")
        return None
    if not _ok(t, shape, dtype, dev.index):
        _check(name, t, shape, dtype, dev)
    return t.data_ptr()


def _int32(what, n):
    if n > _INT_MAX:
        raise ValueError(f"{what} is {n}, more than {_INT_MAX}")
    return n


def _check_gates(x, r, A, r_bias, i, i_bias, z, starts, shape, dev):
    f32, channels = torch.float32, (shape[1],)
    _check("x", x, shape, x.dtype, dev)
    _check("r", r, shape, x.dtype, dev)
    _check("A", A, channels, f32, dev)
    _check("r_bias", r_bias, channels, f32, dev, required=False)
    _check("i", i, shape, x.dtype, dev, required=False)
    if i_bias is not None and i is None:
        raise ValueError("i_bias needs i")
    _check("i_bias", i_bias, channels, f32, dev, required=False)
    _check("z", z, shape, x.dtype, dev, required=False)
    if starts is not None:
        if starts.dtype not in (torch.uint8, torch.bool):
            raise TypeError(f"starts has dtype {starts.dtype}, expected uint8 or bool")
        _check("starts", starts, shape[:1] + shape[2:], starts.dtype, dev)


def _gates_in(x, r, A, r_bias, i, i_bias, z, starts, shape, dev):
    """_check_gates, and the addresses: (x, r, A, r_bias, i, i_bias, z), starts."""
    dt, idx, channels = x.dtype, dev.index, (shape[1],)
    fits = (_ok(x, shape, dt, idx) and _ok(r, shape, dt, idx) and _ok(A, channels, _F32, idx)
            and (r_bias is None or _ok(r_bias, channels, _F32, idx)) and (i is None or _ok(i, shape, dt, idx))
            and (i_bias is None or (i is not None and _ok(i_bias, channels, _F32, idx)))
            and (z is None or _ok(z, shape, dt, idx)) and starts is None) if r is not None and A is not None else False
    if not fits:
        _check_gates(x, r, A, r_bias, i, i_bias, z, starts, shape, dev)
    return (x.data_ptr(), r.data_ptr(), A.data_ptr(), _ptr(r_bias), _ptr(i), _ptr(i_bias), _ptr(z)), _ptr(starts)


def _workspace(workspace, need, dev):
    """(workspace tensor or None, its bytes): the caller's, or a new one where it is missing or too small."""
    if need == 0:
        return None, 0
    if workspace is not None and (workspace.device != dev or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    return workspace, workspace.numel() * workspace.element_size()


def _sizes3(x, name="x"):
    if x.dim() != 3:
        raise ValueError(f"{name} must be (batch, dim, seqlen), not {tuple(x.shape)}")
    shape = tuple(x.shape)
    _int32("batch", shape[0])
    _int32("dim", shape[1])
    return shape


def ssm_gated_scan_bwd_workspace_bytes(batch: int, dim: int, seqlen: int, dtype: torch.dtype) -> int:
    return int(load().ssm_gated_scan_bwd_workspace_bytes(batch, dim, seqlen, _DTYPES[dtype]))


def ssm_gated_scan_ckpt_bytes(batch: int, dim: int, seqlen: int) -> int:
    return int(load().ssm_gated_scan_ckpt_bytes(batch, dim, seqlen))


def ssm_gated_scan_fwd(x, r, A, r_bias=None, i=None, i_bias=None, z=None, *, gate="sigmoid",
                       weight="unit", starts=None, h0=None, return_last_state=False,
                       return_ckpt=False, out=None):
    """The gated recurrence h = a h + w sigmoid(i) x, a = exp(A g(r)), over
    (batch, dim, L) inputs; see include/ssm_gated.h.

    x, r, i, z: (batch, dim, L) float32 or bfloat16 (one dtype for all); A,
    r_bias, i_bias: (dim,) float32; h0: (batch, dim) float32.  gate: g is
    "sigmoid" or "softplus"; weight: w is "unit" (sqrt(1 - a^2)) or "convex"
    (1 - a).  starts: (batch, L) uint8 or bool, set at the first step of each
    sequence packed into a row.  Returns y, then last_state (if
    return_last_state), then what ssm_gated_scan_bwd starts from (if
    return_ckpt): (batch, ceil(L/512), dim) float32."""
    lib = load()
    dev = _gpu(x)
    code = _code(x)
    batch, dim, L = shape = _sizes3(x)
    flags = _rule(gate, weight)
    ins, ps = _gates_in(x, r, A, r_bias, i, i_bias, z, starts, shape, dev)
    p0 = _in("h0", h0, (batch, dim), _F32, dev, required=False)
    y = out if out is not None else torch.empty_like(x)
    py = _in("out", y, shape, x.dtype, dev)
    last = torch.empty((batch, dim), dtype=_F32, device=dev) if return_last_state else None
    ckpt = torch.empty((batch, -(-L // CKPT_STEPS), dim), dtype=_F32, device=dev) if return_ckpt else None
    _call(lib.ssm_gated_scan_fwd, "ssm_gated_scan_fwd", dev, *ins, flags, ps, p0, py, _ptr(last), _ptr(ckpt),
          ckpt.numel() * 4 if return_ckpt else 0, batch, dim, L, code)
    res = (y,)
    if return_last_state:
        res += (last,)
    if return_ckpt:
        res += (ckpt,)
    return res[0] if len(res) == 1 else res


def ssm_gated_scan_bwd(x, r, A, r_bias=None, i=None, i_bias=None, z=None, *, gate="sigmoid",
                       weight="unit", starts=None, ckpt, dy, dlast_state=None, workspace=None):
    """Gradients through ssm_gated_scan_fwd, called with the same inputs and
    rules, from the ckpt it returned (which holds h0), dy = dL/dy and
    optionally dL/dlast_state.  Returns a dict: dx, dr, di (None without i),
    dz (None without z) in the input dtype; dA, dr_bias, di_bias (None without
    i), dh0 in float32."""
    lib = load()
    dev = _gpu(x)
    code = _code(x)
    batch, dim, L = shape = _sizes3(x)
    flags = _rule(gate, weight)
    ins, ps = _gates_in(x, r, A, r_bias, i, i_bias, z, starts, shape, dev)
    pc = _in("ckpt", ckpt, (batch, -(-L // CKPT_STEPS), dim), _F32, dev)
    pdy = _in("dy", dy, shape, x.dtype, dev)
    pdl = _in("dlast_state", dlast_state, (batch, dim), _F32, dev, required=False)
    like = torch.empty_like  # (a third quicker than empty with a shape)
    g = dict(dx=like(x), dr=like(x), dA=like(A), dr_bias=like(A), di=like(x) if i is not None else None,
             di_bias=like(A) if i is not None else None, dz=like(x) if z is not None else None,
             dh0=torch.empty((batch, dim), dtype=_F32, device=dev))
    workspace, ws_bytes = _workspace(workspace, lib.ssm_gated_scan_bwd_workspace_bytes(batch, dim, L, code), dev)
    _call(lib.ssm_gated_scan_bwd, "ssm_gated_scan_bwd", dev, *ins, flags, ps, pc, ckpt.numel() * 4, pdy, pdl,
          _ptr(g["dx"]), _ptr(g["dr"]), _ptr(g["dA"]), _ptr(g["dr_bias"]), _ptr(g["di"]), _ptr(g["di_bias"]),
          _ptr(g["dz"]), _ptr(g["dh0"]), batch, dim, L, code, _ptr(workspace), ws_bytes)
    return g


def ssm_gated_state_update(state, x, r, A, r_bias=None, i=None, i_bias=None, z=None, *,
                           gate="sigmoid", weight="unit", starts=None, out=None, state_out=None):
    """One token of the gated recurrence: state (batch, dim) float32 is updated
    in place, or kept and the new one written to state_out.  x, r, i, z:
    (batch, dim); starts: (batch,), set where the token is its sequence's
    first.  Returns y (batch, dim)."""
    lib = load()
    dev = _gpu(x)
    code = _code(x)
    if x.dim() != 2:
        raise ValueError(f"x must be (batch, dim), not {tuple(x.shape)}")
    batch, dim = shape = x.shape
    _int32("batch", batch)
    _int32("dim", dim)
    flags = _rule(gate, weight)
    p0 = _in("state", state, shape, _F32, dev)
    ins, ps = _gates_in(x, r, A, r_bias, i, i_bias, z, starts, shape, dev)
    y = out if out is not None else torch.empty_like(x)
    py = y.data_ptr() if out is None else _in("out", y, shape, x.dtype, dev)
    _call(lib.ssm_gated_state_update, "ssm_gated_state_update", dev, p0, *ins, flags, ps, py,
          _in("state_out", state_out, shape, _F32, dev, required=False), batch, dim, code)
    return y


def _norm_sizes(x, axis):
    """(batch, dim, seqlen, shape of the statistics) of a norm over `axis`."""
    shape = tuple(x.shape)
    n = len(shape)
    if n < 1 or not -n <= axis < n:
        raise ValueError(f"axis {axis} is not one of x, {shape}")
    axis %= n
    if axis == n - 1:
        stats = shape[:-1]
        tokens = 1
        for v in stats:
            tokens *= v
        return _int32("the number of tokens", tokens), _int32("dim", shape[-1]), 1, stats
    if n == 3 and axis == 1:
        return _int32("batch", shape[0]), _int32("dim", shape[1]), shape[2], (shape[0], shape[2])
    raise ValueError("the norm goes over the last axis, or over axis 1 of (batch, dim, seqlen)")


def ssm_layer_norm_bwd_workspace_bytes(batch: int, dim: int, seqlen: int, dtype: torch.dtype) -> int:
    return int(load().ssm_layer_norm_bwd_workspace_bytes(batch, dim, seqlen, _DTYPES[dtype]))


def ssm_layer_norm_fwd(x, weight, bias=None, residual=None, *, eps=1e-5, axis=-1,
                       return_stats=False, out=None):
    """Layer norm of x (+ residual) over its channels; see include/ssm_norm.h.

    x, residual: float32 or bfloat16, the channels on the last axis (axis=-1,
    any leading shape) or on axis 1 of (batch, dim, seqlen), the layout of the
    scans (axis=1); weight, bias: (dim,) float32.  Returns y, then with a
    residual the sum x + residual (what the norm was taken of), then mean and
    rstd (if return_stats), float32 in x's shape without the axis."""
    lib = load()
    dev = _gpu(x)
    code = _code(x)
    batch, dim, L, stats = _norm_sizes(x, axis)
    shape, dt = x.shape, x.dtype
    px = _in("x", x, shape, dt, dev)
    pr = _in("residual", residual, shape, dt, dev, required=False)
    pw = _in("weight", weight, (dim,), _F32, dev)
    pb = _in("bias", bias, (dim,), _F32, dev, required=False)
    y = out if out is not None else torch.empty_like(x)
    py = y.data_ptr() if out is None else _in("out", y, shape, dt, dev)
    total = torch.empty_like(x) if residual is not None else None
    mean = rstd = None
    if return_stats:
        mean = torch.empty(stats, dtype=_F32, device=dev)
        rstd = torch.empty_like(mean)
    _call(lib.ssm_layer_norm_fwd, "ssm_layer_norm_fwd", dev, px, pr, pw, pb, eps, py, _ptr(total), _ptr(mean),
          _ptr(rstd), batch, dim, L, code)
    res = (y,)
    if residual is not None:
        res += (total,)
    if return_stats:
        res += (mean, rstd)
    return res[0] if len(res) == 1 else res


def ssm_layer_norm_bwd(x, weight, mean, rstd, dy, dsum=None, *, axis=-1, workspace=None):
    """Gradients through ssm_layer_norm_fwd: x is what was normalised (the
    returned sum where there was a residual), mean and rstd what the forward
    pass returned, dsum the gradient arriving at the sum by its other way.
    Returns a dict: dx (of x and of the residual alike), dweight, dbias."""
    lib = load()
    dev = _gpu(x)
    code = _code(x)
    batch, dim, L, stats = _norm_sizes(x, axis)
    shape, dt = x.shape, x.dtype
    px = _in("x", x, shape, dt, dev)
    pw = _in("weight", weight, (dim,), _F32, dev)
    pm = _in("mean", mean, stats, _F32, dev)
    prs = _in("rstd", rstd, stats, _F32, dev)
    pdy = _in("dy", dy, shape, dt, dev)
    pds = _in("dsum", dsum, shape, dt, dev, required=False)
    g = dict(dx=torch.empty_like(x), dweight=torch.empty_like(weight), dbias=torch.empty_like(weight))
    workspace, ws_bytes = _workspace(workspace, lib.ssm_layer_norm_bwd_workspace_bytes(batch, dim, L, code), dev)
    _call(lib.ssm_layer_norm_bwd, "ssm_layer_norm_bwd", dev, px, pw, pm, prs, pdy, pds, _ptr(g["dx"]),
          _ptr(g["dweight"]), _ptr(g["dbias"]), batch, dim, L, code, _ptr(workspace), ws_bytes)
    return g
