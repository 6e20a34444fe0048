"""The gated recurrence and the layer norm in 64 bits, step by step from their
formulas (include/ssm_gated.h, include/ssm_norm.h), with every gradient; and the
comparison that their tests use."""
from __future__ import annotations

import numpy as np

EPS32 = 2.0 ** -24            # half a step of float32, relative
HALF = {"f32": EPS32, "bf16": 2.0 ** -8}


def _sig(v):
    # exp of a negative number only: no overflow at either end
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


def gates(p, gate, weight):
    """(a, w, g, dg/dr, sigmoid of the input gate or 1) of each step."""
    pre = p["r"] + (0.0 if p.get("r_bias") is None else p["r_bias"][:, None])
    if gate == "sigmoid":
        g, slope = _sig(pre), _sig(pre) * _sig(-pre)
    else:
        g, slope = np.maximum(pre, 0) + np.log1p(np.exp(-np.abs(pre))), _sig(pre)
    e = p["A"][:, None] * g
    a = np.exp(e)
    w = np.sqrt(-np.expm1(2 * e)) if weight == "unit" else -np.expm1(e)
    gi = np.ones_like(a)
    if p.get("i") is not None:
        gi = _sig(p["i"] + (0.0 if p.get("i_bias") is None else p["i_bias"][:, None]))
    return a, w, g, slope, gi


def gated_fwd(p, gate="sigmoid", weight="unit"):
    """p: dict of float64 arrays x, r, A, r_bias, i, i_bias, z, starts, h0.  Returns (y, last, states h_0 .. h_L)."""
    a, w, _, _, gi = gates(p, gate, weight)
    b, d, L = p["x"].shape
    h = np.zeros((b, d)) if p.get("h0") is None else p["h0"].astype(np.float64)
    hs = np.empty((L + 1, b, d))
    hs[0] = h
    for t in range(L):
        before = h
        if p.get("starts") is not None:
            before = np.where(p["starts"][:, t, None] != 0, 0.0, h)
        h = a[:, :, t] * before + w[:, :, t] * gi[:, :, t] * p["x"][:, :, t]
        hs[t + 1] = h
    states = np.moveaxis(hs, 0, 2)
    y = states[:, :, 1:]
    if p.get("z") is not None:
        y = y * p["z"] * _sig(p["z"])
    return y, h, states


def gated_bwd(p, dy, dlast=None, gate="sigmoid", weight="unit"):
    a, w, g, slope, gi = gates(p, gate, weight)
    _, _, states = gated_fwd(p, gate, weight)
    b, d, L = p["x"].shape
    has_i, has_z = p.get("i") is not None, p.get("z") is not None
    before = states[:, :, :-1].copy()
    if p.get("starts") is not None:
        before[np.broadcast_to(p["starts"][:, None, :] != 0, before.shape)] = 0.0
    dh = dy
    dz = None
    if has_z:
        s = _sig(p["z"])
        dh = dy * p["z"] * s
        dz = dy * states[:, :, 1:] * s * (1 + p["z"] * (1 - s))
    lam = np.empty((b, d, L))
    m = np.zeros((b, d)) if dlast is None else dlast.astype(np.float64)
    for t in range(L - 1, -1, -1):
        lam[:, :, t] = dh[:, :, t] + m
        m = a[:, :, t] * lam[:, :, t]
        if p.get("starts") is not None:
            m = np.where(p["starts"][:, t, None] != 0, 0.0, m)
    with np.errstate(divide="ignore", invalid="ignore"):
        bend = np.where(w > 0, -a * a / w, 0.0) if weight == "unit" else -a
    dw = lam * gi * p["x"]
    de = lam * before * a + dw * bend
    dr = de * p["A"][:, None] * slope
    di = lam * w * p["x"] * gi * (1 - gi) if has_i else None
    return dict(dx=lam * w * gi, dr=dr, dA=(de * g).sum((0, 2)), dr_bias=dr.sum((0, 2)), di=di,
                di_bias=di.sum((0, 2)) if has_i else None, dz=dz, dh0=m,
                # sums of the terms' sizes: what an error of each term adds up to
                size=dict(dA=np.abs(de * g).sum((0, 2)), dr_bias=np.abs(dr).sum((0, 2)),
                          di_bias=np.abs(di).sum((0, 2)) if has_i else None))


def norm_fwd(x, weight, bias, eps, axis):
    mean = x.mean(axis, keepdims=True)
    rstd = 1.0 / np.sqrt(((x - mean) ** 2).mean(axis, keepdims=True) + eps)
    shape = [1] * x.ndim
    shape[axis] = -1
    y = (x - mean) * rstd * weight.reshape(shape) + (0.0 if bias is None else bias.reshape(shape))
    return y, np.squeeze(mean, axis), np.squeeze(rstd, axis)


def norm_bwd(x, weight, mean, rstd, dy, dsum, axis):
    shape = [1] * x.ndim
    shape[axis] = -1
    xh = (x - np.expand_dims(mean, axis)) * np.expand_dims(rstd, axis)
    dn = dy * weight.reshape(shape)
    dx = np.expand_dims(rstd, axis) * (dn - dn.mean(axis, keepdims=True) - xh * (dn * xh).mean(axis, keepdims=True))
    if dsum is not None:
        dx = dx + dsum
    over = tuple(k for k in range(x.ndim) if k != axis % x.ndim)
    return dict(dx=dx, dweight=(dy * xh).sum(over), dbias=dy.sum(over))


def memory(p, gate):
    """Steps that an error of one decay stays in the state: 1 / (1 - the largest decay), at most the sequence."""
    a = gates(p, gate, "convex")[0]
    return float(min(a.shape[-1], 1.0 / (1.0 - min(a.max(), 1 - 1e-12)))) + 1.0


def close(got, ref, dtype, slack, what, size=None):
    """|got - ref| <= half a step of the type + slack * max|ref| (or, of a sum, slack * the sizes of its terms),
    everywhere; returns the worst error over its bound."""
    ref = np.asarray(ref, np.float64)
    got = np.asarray(got, np.float64)
    assert got.shape == ref.shape, f"{what}: shape {got.shape}, expected {ref.shape}"
    if ref.size == 0:
        return 0.0
    assert np.all(np.isfinite(got)), f"{what}: non-finite values"
    bound = HALF[dtype] * np.abs(ref) + slack * np.max(np.abs(ref) if size is None else size) + 1e-37
    worst = float(np.max(np.abs(got - ref) / bound))
    assert worst <= 1.0, f"{what}: error {worst:.2f} times the bound (slack {slack:.1e})"
    return worst
