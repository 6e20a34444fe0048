"""Linear attention with a decay for each head and the group norm in 64 bits, from
their formulas (include/ssm_linear_attn.h, include/ssm_group_norm.h), with every
gradient; and the comparison that their tests use.

The attention is written out over all pairs of steps of a row, not as a
recurrence; tests/test_heads_abi.py holds it against the recurrence and against
differences."""
from __future__ import annotations

import torch

EPS32 = 2.0 ** -24            # half a step of float32, relative
HALF = {"f32": EPS32, "bf16": 2.0 ** -8}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def spread(t, heads):
    return t.repeat_interleave(heads // t.shape[-2], -2)


def gathered(t, n):
    return t.unflatten(-2, (n, t.shape[-2] // n)).sum(-2)


def _dbl(t):
    return None if t is None else t.detach().cpu().double()


def attn(q, k, v, g, scale, *, starts=None, lengths=None, h0=None, dy=None, dlast=None):
    """y, last_state and, with dy, every gradient; and under "pairs" the sums of |(weighted q.k) v| that the outputs are
    sums of (what a rounding of each product q.k adds up to), of the products of an operand alike for dq, dk and dv."""
    q, k, v, g, h0, dy, dlast = (_dbl(t) for t in (q, k, v, g, h0, dy, dlast))
    b, L, dk = q.shape[0], q.shape[1], q.shape[3]
    heads, (hq, hk, hv) = g.shape[0], (t.shape[2] for t in (q, k, v))
    dv = v.shape[3]
    q, k, v = (spread(t, heads).transpose(1, 2) for t in (q, k, v))  # (b, heads, L, d)
    n = torch.full((b,), L) if lengths is None else lengths.cpu().long().clamp(0, L)
    t = torch.arange(L)
    live = t < n[:, None]
    q, k, v = (torch.where(live[:, None, :, None], x, 0.0) for x in (q, k, v))
    seen = torch.zeros(b, L, dtype=torch.long)
    if starts is not None:
        seen = ((starts.cpu() != 0) & live).long().cumsum(1)

    def power(steps, kept):  # e^{g steps}, 1 for none
        e = g.view([1, heads] + [1] * (steps.dim() - 1)) * steps.unsqueeze(1).double()
        e = torch.where(steps.unsqueeze(1) == 0, torch.zeros_like(e), e)
        return torch.where(kept.unsqueeze(1), e.exp(), 0.0)

    apart = (t[:, None] - t[None, :]).expand(b, L, L)
    pair = live[:, :, None] & live[:, None, :] & (apart >= 0) & (seen[:, :, None] == seen[:, None, :])
    W = power(apart.clamp(min=0), pair)
    total = seen[torch.arange(b), (n - 1).clamp(min=0)] if L else torch.zeros(b, dtype=torch.long)
    total = torch.where(n > 0, total, 0)
    enter = power((t + 1).expand(b, L), live & (seen == 0))
    left = (n[:, None] - 1 - t).clamp(min=0)
    leave = power(left, live & (seen == total[:, None]))
    through = power(n[:, None], (total == 0)[:, None])[..., 0]
    S0 = torch.zeros(b, heads, dk, dv, dtype=torch.float64) if h0 is None else h0
    P = scale * W * (q @ k.transpose(-1, -2))
    out = dict(y=(P @ v + scale * enter[..., None] * (q @ S0)).transpose(1, 2),
               last=through[..., None, None] * S0 + (k * leave[..., None]).transpose(-1, -2) @ v)
    pairs = dict(y=(P.abs() @ v.abs()).transpose(1, 2))
    out["pairs"] = pairs
    if dy is None:
        return out
    dy = torch.where(live[:, None, :, None], dy.transpose(1, 2), 0.0)
    dP = scale * W * (dy @ v.transpose(-1, -2))
    dS = torch.zeros_like(S0) if dlast is None else dlast
    grads = dict(dq=dP @ k + scale * enter[..., None] * (dy @ S0.transpose(-1, -2)),
                 dk=dP.transpose(-1, -2) @ q + leave[..., None] * (v @ dS.transpose(-1, -2)),
                 dv=P.transpose(-1, -2) @ dy + leave[..., None] * (k @ dS))
    pairs.update(dq=dP.abs() @ k.abs(), dk=dP.abs().transpose(-1, -2) @ q.abs(), dv=P.abs().transpose(-1, -2) @ dy.abs())
    for name, m in (("dq", hq), ("dk", hk), ("dv", hv)):
        out[name] = gathered(grads[name].transpose(1, 2), m)
        pairs[name] = gathered(pairs[name].transpose(1, 2), m)
    out["dh0"] = through[..., None, None] * dS + scale * (q * enter[..., None]).transpose(-1, -2) @ dy
    out["dlog_decay"] = ((apart.unsqueeze(1) * P * (dy @ v.transpose(-1, -2))).sum((0, 2, 3))
                         + scale * ((t + 1) * enter * ((q @ S0) * dy).sum(-1)).sum((0, 2))
                         + (left.unsqueeze(1) * leave * (k * (v @ dS.transpose(-1, -2))).sum(-1)).sum((0, 2))
                         + (n[:, None] * through * (S0 * dS).sum((-1, -2))).sum(0))
    return out


def attn_sizes(q, k, v, g, scale, *, h0=None, dy=None, dlast=None, **rows):
    """The same of the operands' absolute values: what the terms of every sum add up to."""
    mag = [None if t is None else t.detach().abs() for t in (q, k, v, h0, dy, dlast)]
    return attn(*mag[:3], g, abs(scale), h0=mag[3], dy=mag[4], dlast=mag[5], **rows)


def attn_steps(q, k, v, g, scale, *, starts=None, lengths=None, h0=None):
    """(y, last_state) step by step."""
    q, k, v, g, h0 = (_dbl(t) for t in (q, k, v, g, h0))
    b, L, dk, heads, dv = q.shape[0], q.shape[1], q.shape[3], g.shape[0], v.shape[3]
    q, k, v = (spread(t, heads) for t in (q, k, v))
    S = torch.zeros(b, heads, dk, dv, dtype=torch.float64) if h0 is None else h0.clone()
    y = torch.zeros(b, L, heads, dv, dtype=torch.float64)
    for row in range(b):
        for t in range(L if lengths is None else min(max(int(lengths[row]), 0), L)):
            if starts is not None and starts[row, t]:
                S[row] = 0
            else:
                S[row] *= g.exp()[:, None, None]
            S[row] += k[row, t][:, :, None] * v[row, t][:, None, :]
            y[row, t] = scale * (q[row, t][:, :, None] * S[row]).sum(1)
    return y, S


def act(kind, t):
    if kind == "none":
        return t, torch.ones_like(t)
    p, m = torch.sigmoid(t), torch.sigmoid(-t)
    return (p, p * m) if kind == "sigmoid" else (t * p, p * (1 + t * m))


def group_fwd(x, groups, weight, bias, z, kind, eps):
    """(y, mean, rstd, n)"""
    x, weight, bias, z = (_dbl(t) for t in (x, weight, bias, z))
    split = (*x.shape[:-1], groups, x.shape[-1] // groups)
    v = x.reshape(split)
    mean = v.mean(-1, keepdim=True)
    rstd = ((v - mean).square().mean(-1, keepdim=True) + eps).rsqrt()
    n = ((v - mean) * rstd).reshape(x.shape)
    n = n * (1.0 if weight is None else weight) + (0.0 if bias is None else bias)
    y = act(kind, n)[0] if z is None else n * act(kind, z)[0]
    return y, mean[..., 0], rstd[..., 0], n


def group_bwd(x, groups, weight, bias, z, kind, mean, rstd, dy):
    """dx, dz, dweight, dbias, and under "size" the sizes of the terms of each."""
    x, weight, bias, z, mean, rstd, dy = (_dbl(t) for t in (x, weight, bias, z, mean, rstd, dy))
    shape, width = x.shape, x.shape[-1] // groups
    split = (*shape[:-1], groups, width)
    rs = rstd[..., None]
    xh = (x.reshape(split) - mean[..., None]) * rs
    flat = xh.reshape(shape)
    n = flat * (1.0 if weight is None else weight) + (0.0 if bias is None else bias)
    dz = None
    if z is None:
        dn = dy * act(kind, n)[1]
    else:
        a, slope = act(kind, z)
        dn, dz = dy * a, dy * n * slope
    d = (dn * (1.0 if weight is None else weight)).reshape(split)
    dx = rs * (d - d.mean(-1, keepdim=True) - xh * (d * xh).mean(-1, keepdim=True))
    over = tuple(range(len(shape) - 1))
    size = dict(dx=(rs * (d.abs() + d.abs().mean(-1, keepdim=True)
                          + xh.abs() * (d * xh).abs().mean(-1, keepdim=True))).reshape(shape),
                dz=None if dz is None else dz.abs(), dweight=(dn * flat).abs().sum(over), dbias=dn.abs().sum(over))
    return dict(dx=dx.reshape(shape), dz=dz, dweight=(dn * flat).sum(over), dbias=dn.sum(over), size=size)


def within(got, want, bound, what):
    """|got - want| <= bound, everywhere; returns the worst error over its bound."""
    got, want = got.detach().cpu().double(), want.double()
    assert got.shape == want.shape, f"{what}: shape {tuple(got.shape)}, expected {tuple(want.shape)}"
    if got.numel() == 0:
        return 0.0
    assert bool(torch.isfinite(got).all()), f"{what}: non-finite values"
    worst = ((got - want).abs() / (bound + 1e-37)).max().item()
    assert worst <= 1.0, f"{what}: error {worst:.2f} times the bound"
    return worst
