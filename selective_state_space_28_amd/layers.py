"""torch-tensor wrappers of the gated recurrence (include/ssm_gated.h) and the
layer norm (include/ssm_norm.h): marshalling only, as in ops.py."""
from __future__ import annotations

import contextlib

import torch

from ._lib import SSM_GATE_SOFTPLUS, SSM_GATE_UNIT, SsmError, load
from .ops import _DTYPES, _check, _code, _ptr

CKPT_STEPS = 512
_GATES = {"sigmoid": 0, "softplus": SSM_GATE_SOFTPLUS}
_WEIGHTS = {"convex": 0, "unit": SSM_GATE_UNIT}
_INT_MAX = 2**31 - 1
_HERE = contextlib.nullcontext()


def _rule(gate, weight):
    if gate not in _GATES:
        raise ValueError(f"gate must be 'sigmoid' or 'softplus', not {gate!r}")
    if weight not in _WEIGHTS:
        raise ValueError(f"weight must be 'unit' or 'convex', not {weight!r}")
    return _GATES[gate] | _WEIGHTS[weight]


def _on(dev):
    """The context that makes `dev` the current device (launches go there)."""
    if dev.type != "cuda":
        raise ValueError("libssm runs on the GPU: tensors must be on a cuda device")
    return _HERE if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)


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
    return _int32("batch", x.shape[0]), _int32("dim", x.shape[1]), x.shape[2]


def ssm_gated_scan_fwd_workspace_bytes(batch: int, dim: int, seqlen: int, dtype: torch.dtype) -> int:
    return int(load().ssm_gated_scan_fwd_workspace_bytes(batch, dim, seqlen, _DTYPES[dtype]))


def ssm_gated_scan_bwd_workspace_bytes(batch: int, dim: int, seqlen: int, dtype: torch.dtype) -> int:
    return int(load().ssm_gated_scan_bwd_workspace_bytes(batch, dim, seqlen, _DTYPES[dtype]))


def ssm_gated_scan_ckpt_bytes(batch: int, dim: int, seqlen: int) -> int:
    return int(load().ssm_gated_scan_ckpt_bytes(batch, dim, seqlen))


def ssm_gated_scan_fwd(x, r, A, r_bias=None, i=None, i_bias=None, z=None, *, gate="sigmoid",
                       weight="unit", starts=None, h0=None, return_last_state=False,
                       return_ckpt=False, out=None, workspace=None):
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
    dev = x.device
    here = _on(dev)
    code = _code(x)
    batch, dim, L = _sizes3(x)
    flags = _rule(gate, weight)
    _check_gates(x, r, A, r_bias, i, i_bias, z, starts, (batch, dim, L), dev)
    _check("h0", h0, (batch, dim), torch.float32, dev, required=False)
    y = out if out is not None else torch.empty_like(x)
    _check("out", y, (batch, dim, L), x.dtype, dev)
    last = torch.empty((batch, dim), dtype=torch.float32, device=dev) if return_last_state else None
    ckpt = None
    if return_ckpt:
        ckpt = torch.empty((batch, -(-L // CKPT_STEPS), dim), dtype=torch.float32, device=dev)
    workspace, ws_bytes = _workspace(workspace, int(lib.ssm_gated_scan_fwd_workspace_bytes(batch, dim, L, code)), dev)
    with here:
        rc = lib.ssm_gated_scan_fwd(
            _ptr(x), _ptr(r), _ptr(A), _ptr(r_bias), _ptr(i), _ptr(i_bias), _ptr(z), flags, _ptr(starts),
            _ptr(h0), _ptr(y), _ptr(last), _ptr(ckpt), ckpt.numel() * 4 if return_ckpt else 0, batch, dim, L,
            code, _ptr(workspace), ws_bytes, torch.cuda.current_stream(dev).cuda_stream)
    if rc != 0:
        raise SsmError(rc, "ssm_gated_scan_fwd")
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
    dev = x.device
    here = _on(dev)
    code = _code(x)
    batch, dim, L = _sizes3(x)
    flags = _rule(gate, weight)
    _check_gates(x, r, A, r_bias, i, i_bias, z, starts, (batch, dim, L), dev)
    _check("ckpt", ckpt, (batch, -(-L // CKPT_STEPS), dim), torch.float32, dev)
    _check("dy", dy, (batch, dim, L), x.dtype, dev)
    _check("dlast_state", dlast_state, (batch, dim), torch.float32, dev, required=False)
    f32 = dict(dtype=torch.float32, device=dev)
    g = dict(dx=torch.empty_like(x), dr=torch.empty_like(x), dA=torch.empty(dim, **f32),
             dr_bias=torch.empty(dim, **f32), di=torch.empty_like(x) if i is not None else None,
             di_bias=torch.empty(dim, **f32) if i is not None else None,
             dz=torch.empty_like(x) if z is not None else None, dh0=torch.empty((batch, dim), **f32))
    workspace, ws_bytes = _workspace(workspace, int(lib.ssm_gated_scan_bwd_workspace_bytes(batch, dim, L, code)), dev)
    with here:
        rc = lib.ssm_gated_scan_bwd(
            _ptr(x), _ptr(r), _ptr(A), _ptr(r_bias), _ptr(i), _ptr(i_bias), _ptr(z), flags, _ptr(starts),
            _ptr(ckpt), ckpt.numel() * 4, _ptr(dy), _ptr(dlast_state), _ptr(g["dx"]), _ptr(g["dr"]),
            _ptr(g["dA"]), _ptr(g["dr_bias"]), _ptr(g["di"]), _ptr(g["di_bias"]), _ptr(g["dz"]),
            _ptr(g["dh0"]), batch, dim, L, code, _ptr(workspace), ws_bytes,
            torch.cuda.current_stream(dev).cuda_stream)
    if rc != 0:
        raise SsmError(rc, "ssm_gated_scan_bwd")
    return g


def ssm_gated_state_update(state, x, r, A, r_bias=None, i=None, i_bias=None, z=None, *,
                           gate="sigmoid", weight="unit", starts=None, out=None, state_out=None):
    """One token of the gated recurrence: state (batch, dim) float32 is updated
    in place, or kept and the new one written to state_out.  x, r, i, z:
    (batch, dim); starts: (batch,), set where the token is its sequence's
    first.  Returns y (batch, dim)."""
    lib = load()
    dev = x.device
    here = _on(dev)
    code = _code(x)
    if x.dim() != 2:
        raise ValueError(f"x must be (batch, dim), not {tuple(x.shape)}")
    batch, dim = shape = _int32("batch", x.shape[0]), _int32("dim", x.shape[1])
    flags = _rule(gate, weight)
    _check("state", state, shape, torch.float32, dev)
    _check_gates(x, r, A, r_bias, i, i_bias, z, starts, shape, dev)
    y = out if out is not None else torch.empty_like(x)
    _check("out", y, shape, x.dtype, dev)
    _check("state_out", state_out, shape, torch.float32, dev, required=False)
    with here:
        rc = lib.ssm_gated_state_update(
            _ptr(state), _ptr(x), _ptr(r), _ptr(A), _ptr(r_bias), _ptr(i), _ptr(i_bias), _ptr(z), flags,
            _ptr(starts), _ptr(y), _ptr(state_out), batch, dim, code,
            torch.cuda.current_stream(dev).cuda_stream)
    if rc != 0:
        raise SsmError(rc, "ssm_gated_state_update")
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
    dev = x.device
    here = _on(dev)
    code = _code(x)
    batch, dim, L, stats = _norm_sizes(x, axis)
    _check("x", x, x.shape, x.dtype, dev)
    _check("residual", residual, x.shape, x.dtype, dev, required=False)
    _check("weight", weight, (dim,), torch.float32, dev)
    _check("bias", bias, (dim,), torch.float32, dev, required=False)
    y = out if out is not None else torch.empty_like(x)
    _check("out", y, x.shape, x.dtype, dev)
    total = torch.empty_like(x) if residual is not None else None
    mean = rstd = None
    if return_stats:
        mean = torch.empty(stats, dtype=torch.float32, device=dev)
        rstd = torch.empty(stats, dtype=torch.float32, device=dev)
    with here:
        rc = lib.ssm_layer_norm_fwd(_ptr(x), _ptr(residual), _ptr(weight), _ptr(bias), eps, _ptr(y),
                                    _ptr(total), _ptr(mean), _ptr(rstd), batch, dim, L, code,
                                    torch.cuda.current_stream(dev).cuda_stream)
    if rc != 0:
        raise SsmError(rc, "ssm_layer_norm_fwd")
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
    dev = x.device
    here = _on(dev)
    code = _code(x)
    batch, dim, L, stats = _norm_sizes(x, axis)
    _check("x", x, x.shape, x.dtype, dev)
    _check("weight", weight, (dim,), torch.float32, dev)
    _check("mean", mean, stats, torch.float32, dev)
    _check("rstd", rstd, stats, torch.float32, dev)
    _check("dy", dy, x.shape, x.dtype, dev)
    _check("dsum", dsum, x.shape, x.dtype, dev, required=False)
    f32 = dict(dtype=torch.float32, device=dev)
    g = dict(dx=torch.empty_like(x), dweight=torch.empty(dim, **f32), dbias=torch.empty(dim, **f32))
    workspace, ws_bytes = _workspace(workspace, int(lib.ssm_layer_norm_bwd_workspace_bytes(batch, dim, L, code)), dev)
    with here:
        rc = lib.ssm_layer_norm_bwd(_ptr(x), _ptr(weight), _ptr(mean), _ptr(rstd), _ptr(dy), _ptr(dsum),
                                    _ptr(g["dx"]), _ptr(g["dweight"]), _ptr(g["dbias"]), batch, dim, L, code,
                                    _ptr(workspace), ws_bytes, torch.cuda.current_stream(dev).cuda_stream)
    if rc != 0:
        raise SsmError(rc, "ssm_layer_norm_bwd")
    return g
