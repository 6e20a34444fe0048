"""The gated recurrence (include/ssm_gated.h) and its gradients in 64 bits over
torch tensors, the recurrences as log-depth scans: for shapes whose step-by-step
reference (tests/layers_ref.py) would take too long.  Where the state at a step is
f_t = a_t f_{t-1} + v_t, the pairs (a, v) are composed by doubling."""
from __future__ import annotations

import torch
import torch.nn.functional as F

EPS32 = 2.0 ** -24


def scan(a, v, first):
    """f_t = a_t f_{t-1} + v_t along the last axis, f_{-1} = first."""
    f = v.clone()
    f[..., 0] += a[..., 0] * first
    p, step, n = a.clone(), 1, a.shape[-1]
    while step < n:
        f[..., step:] = f[..., step:] + p[..., step:] * f[..., :-step].clone()
        p[..., step:] = p[..., step:] * p[..., :-step].clone()
        step *= 2
    return f


def gated(x, r, A, r_bias=None, i=None, i_bias=None, z=None, *, gate="sigmoid", weight="unit", starts=None, h0=None,
          dy=None, dlast=None):
    """y, last_state, the states before each step, and with dy the gradients: a dict, with sizes of terms under "size" (the
    summands of dA, dr_bias and di_bias; of each dr, and of dA once more, the two that the decay's gradient adds)."""
    x, r, A, r_bias, i, i_bias, z, h0, dy, dlast = (
        None if v is None else v.double() for v in (x, r, A, r_bias, i, i_bias, z, h0, dy, dlast))
    pre = r if r_bias is None else r + r_bias[:, None]
    slope = torch.sigmoid(pre)
    g = slope if gate == "sigmoid" else F.softplus(pre, threshold=1e9)
    if gate == "sigmoid":
        slope = slope * torch.sigmoid(-pre)
    e = A[:, None] * g
    a = torch.exp(e)
    w = torch.sqrt(-torch.expm1(2 * e)) if weight == "unit" else -torch.expm1(e)
    gi = torch.ones_like(x) if i is None else torch.sigmoid(i if i_bias is None else i + i_bias[:, None])
    first = torch.zeros_like(x[..., 0]) if h0 is None else h0
    cut = torch.zeros_like(a, dtype=torch.bool) if starts is None else (starts != 0)[:, None].expand_as(a)
    kept = torch.where(cut, torch.zeros_like(a), a)  # the decay of the state that enters
    h = scan(kept, w * gi * x, first)
    before = torch.cat([first[..., None], h[..., :-1]], -1)
    before = torch.where(cut, torch.zeros_like(before), before)
    y = h if z is None else h * F.silu(z)
    if dy is None:
        return y, h[..., -1], before
    dh, dz = dy, None
    if z is not None:
        s = torch.sigmoid(z)
        dh, dz = dy * z * s, dy * h * s * (1 + z * torch.sigmoid(-z))
    # lambda_t = dh_t + (decay of step t+1 on h_t) lambda_{t+1}, from the right
    after = torch.cat([kept[..., 1:], torch.ones_like(kept[..., :1])], -1)
    end = torch.zeros_like(first) if dlast is None else dlast
    lam = scan(after.flip(-1), dh.flip(-1), end).flip(-1)
    bend = -a if weight == "convex" else torch.where(w > 0, -a * a / torch.where(w > 0, w, torch.ones_like(w)),
                                                     torch.zeros_like(w))
    de = lam * (before * a + gi * x * bend)
    dr = de * A[:, None] * slope
    grads = dict(dx=lam * w * gi, dr=dr, dA=(de * g).sum((0, 2)), dr_bias=dr.sum((0, 2)), di=None, di_bias=None, dz=dz,
                 dh0=kept[..., 0] * lam[..., 0])
    both = lam.abs() * ((before * a).abs() + (gi * x * bend).abs())
    size = dict(dA=(de * g).abs().sum((0, 2)), dr_bias=dr.abs().sum((0, 2)), dr_terms=both * A[:, None].abs() * slope,
                dA_terms=(both * g).sum((0, 2)))
    if i is not None:
        grads["di"] = di = lam * w * x * gi * torch.sigmoid(-(i if i_bias is None else i + i_bias[:, None]))
        grads["di_bias"], size["di_bias"] = di.sum((0, 2)), di.abs().sum((0, 2))
    grads["size"] = size
    return y, h[..., -1], before, grads


def close(got, want, half, slack, what, size=None):
    """|got - want| <= half |want| + slack max|want| (of a sum: slack times the sizes of its terms), everywhere."""
    got, want = got.double(), want.double()
    assert got.shape == want.shape, what
    assert bool(torch.isfinite(got).all()), f"{what}: non-finite values"
    bound = half * want.abs() + slack * (want.abs() if size is None else size).max() + 1e-37
    worst = ((got - want).abs() / bound).max().item()
    assert worst <= 1.0, f"{what}: error {worst:.2f} times the bound (slack {slack:.1e})"
