"""GPU tests of the values that the linear attention (include/ssm_linear_attn.h) gives: how near they are to its formula
in 64 bits (tests/heads_ref.py)."""
import math

import pytest
import torch

from tests import heads_ref as ref
from tests.test_gpu_linear_attn import make, rows_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import selective_state_space_28_amd as ssm
    ssm.load()
    return torch.device("cuda:0")


def wanted(p, dtype, L):
    """The formula's outputs, and how far off they may be.  A float32 sum of N terms is off by N half steps (2^-24) of its
    terms' sizes: N is the width of a product, the steps of a row, 16 for the decays' roundings and the scales of each 32
    steps, and the heads that are added up.  With bf16 the decayed products q.k, and the state as q meets it, are two bf16
    parts: the first has 8 bits, so 2^-7 of the value are left at most, of which the second's rounding leaves half a step
    of 8 bits more, 2^-16 of the value; outputs of bf16 are rounded once, 2^-8 of their own value.  The decay's gradient
    has no such part: it is float32 with float32's sums."""
    scale = p["q"].shape[-1] ** -0.5
    args = (p["q"], p["k"], p["v"], p["g"], scale)
    kw = dict(rows_of(p), dy=p["dy"], dlast=p["dlast"])
    want, size = ref.attn(*args, **kw), ref.attn_sizes(*args, **kw)
    n = (max(p["q"].shape[-1], p["v"].shape[-1]) + L + 16 * (L // 32 + 1) + p["g"].shape[0]) * ref.EPS32
    bound = {name: n * size[name] for name in ("y", "last", "dq", "dk", "dv", "dlog_decay", "dh0")}
    if dtype == "bf16":
        for name in ("y", "dq", "dk", "dv"):
            bound[name] += ref.HALF[dtype] * want[name].abs() + 2.0 ** -16 * (size[name] + want["pairs"][name])
    else:
        for name in ("y", "dq", "dk", "dv"):
            bound[name] += ref.EPS32 * want[name].abs()
    return want, bound


def near(p, dtype, L, what=""):
    import selective_state_space_28_amd as ssm
    want, bound = wanted(p, dtype, L)
    args = (p["q"], p["k"], p["v"], p["g"])
    got = {}
    got["y"], got["last"] = ssm.ssm_linear_attn_fwd(*args, **rows_of(p), return_last_state=True)
    got.update(ssm.ssm_linear_attn_bwd(*args, **rows_of(p), dy=p["dy"], dlast_state=p["dlast"]))
    worst = {}
    for name, b in bound.items():
        if name == "dh0" and p["h0"] is None:
            assert got["dh0"] is None
            continue
        worst[name] = round(ref.within(got[name], want[name], b, f"{what} {name}"), 3)
    print(what, worst)
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L,dk,dv,heads,packed", [(64, 32, 48, (2, 2, 2), False), (150, 64, 64, (2, 2, 2), False),
                                                  (200, 128, 128, (2, 2, 2), True), (130, 128, 128, (2, 1, 2), False),
                                                  (77, 100, 200, (2, 2, 1), False), (300, 256, 256, (1, 1, 1), False)])
def test_products_keep_their_bits(dev, dtype, L, dk, dv, heads, packed):
    """Outputs that nearly cancel are as exact as their terms, but for their own rounding: no product q.k is rounded to 8
    bits on its way to v."""
    hq, hk, hv = heads
    h = max(heads)
    near(make(dev, dtype, 2, L, h, dk, dv, hq=hq, hk=hk, hv=hv, packed=packed, seed=21), dtype, L)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("state", [True, False])
@pytest.mark.parametrize("dk,dv", [(32, 48), (128, 128)])
def test_growing_heads_in_long_segments(dev, dtype, state, dk, dv):
    """A head that grows by e^0.3 a step, in a row split into segments of 320 steps and more, over which a factor passes
    range: the states are 0 or small when they enter, so that nothing of the formula's does.

    With bf16 a part of a state below the smallest normal float, 2^-126, counts as 0 on the matrix cores: each element of
    a state loses at most that in each of two parts, 2^-125, where it meets q (or what takes q's place); and a state that
    enters a chunk is weighed behind that product, by up to e^(64 g).  So outputs may be off by 2^-125 e^(64 g) times the
    sum of that operand's absolute values (and the scale, where it is not in the state) besides."""
    import selective_state_space_28_amd as ssm
    L, n = 20480, 500
    p = make(dev, dtype, 1, n, 1, dk, dv, state=state, g=[0.3], seed=22)
    for name in "kv":
        p[name][:, :300] = 0
    p["dy"][:, 200:] = 0
    if state:
        p["h0"] *= 1e-37
        p["dlast"] *= 1e-37
    want, bound = wanted(p, dtype, n)
    if dtype == "bf16":
        lost, scale = 2.0 ** -125 * math.exp(64 * 0.3), dk ** -0.5
        for name, meets, by in (("y", "q", scale), ("dq", "dy", scale), ("dk", "v", 1.0), ("dv", "k", 1.0)):
            bound[name] = bound[name] + by * lost * p[meets].cpu().double().abs().sum(-1, keepdim=True)
    rows = {name: torch.zeros(1, L, *p[name].shape[2:], dtype=p[name].dtype, device=dev) for name in ("q", "k", "v", "dy")}
    for name, t in rows.items():
        t[:, :n] = p[name]
        t[:, n:] = float("nan")
    args = (rows["q"], rows["k"], rows["v"], p["g"])
    kw = dict(h0=p["h0"], lengths=torch.tensor([n], dtype=torch.int32, device=dev))
    got = {}
    got["y"], got["last"] = ssm.ssm_linear_attn_fwd(*args, **kw, return_last_state=True)
    got.update(ssm.ssm_linear_attn_bwd(*args, **kw, dy=rows["dy"], dlast_state=p["dlast"]))
    for name, b in bound.items():
        if name == "dh0" and not state:
            continue
        t = got[name]
        if name in ("y", "dq", "dk", "dv"):
            assert not bool(t[:, n:].any()), name
            t = t[:, :n]
        ref.within(t, want[name], b, name)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("L", [1, 33, 64])
def test_heads_that_grow_fast(dev, dtype, packed, L):
    """e^1.3 a step, 1.4e36 over 64 of them: small keys, and no state, keep the formula's outputs in float32's range."""
    p = make(dev, dtype, 2, L, 2, 32, 48, packed=packed, state=False, g=[1.3, 0.9], seed=24)
    p["k"] *= 1e-30
    near(p, dtype, L)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (128, 64), (64, 128), (100, 200), (200, 100), (256, 256), (256, 40)])
@pytest.mark.parametrize("L,packed,lengths", [(1000, False, None), (1111, True, None), (1030, False, [700])])
def test_split_rows_of_every_width(dev, dtype, dk, dv, L, packed, lengths):
    """Rows in segments, through which a slow decay carries the states from end to end: in every width's kernels, with the
    gradients' sweeps side by side (widths alike) and after one another."""
    import selective_state_space_28_amd as ssm
    p = make(dev, dtype, 1, L, 2, dk, dv, hk=1, packed=packed, lengths=lengths, g=[-0.002, -0.0005], seed=23)
    state = 2 * dk * dv * 4  # of one segment
    assert ssm.ssm_linear_attn_fwd_workspace_bytes(1, L, 2, dk, dv, p["q"].dtype) >= 2 * state
    assert ssm.ssm_linear_attn_bwd_workspace_bytes(1, L, 2, 2, 1, 2, dk, dv, p["q"].dtype) >= 4 * state
    near(p, dtype, L)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L", [1, 64, 200, 900])
def test_decay_gradient_of_a_state_is_float32(dev, dtype, L):
    """A state of one element that meets one query at the last step, or only the last state's gradient: the decay's
    gradient is L e^(g L) times a product without a sum.  16 half steps of float32 for the decays of each 32 steps, 16 for
    the products and the scale."""
    import selective_state_space_28_amd as ssm
    gen = torch.Generator().manual_seed(19 + L)
    heads = 64
    g = -0.02 * torch.rand(heads, generator=gen)
    h0 = 1 + torch.rand(1, heads, 1, 1, generator=gen)  # 24 bits of it
    q, k, v, dy = (torch.zeros(1, L, heads, 1, dtype=ref.TYPES[dtype]) for _ in range(4))
    q[0, -1], dy[0, -1] = ((1 + torch.rand(heads, 1, generator=gen)).to(q.dtype) for _ in range(2))
    dlast = 1 + torch.rand(1, heads, 1, 1, generator=gen)
    state = L * torch.exp(L * g.double()) * h0[0, :, 0, 0].double()
    slack = (16 * (L // 32 + 1) + 16) * ref.EPS32
    ops = [t.to(dev) for t in (q, k, v, g)]
    got = ssm.ssm_linear_attn_bwd(*ops, scale=0.75, h0=h0.to(dev), dy=dy.to(dev))["dlog_decay"]
    want = 0.75 * state * q[0, -1, :, 0].double() * dy[0, -1, :, 0].double()
    ref.within(got, want, slack * want.abs(), "by a query")
    got = ssm.ssm_linear_attn_bwd(*ops, scale=0.75, h0=h0.to(dev), dy=torch.zeros_like(dy).to(dev),
                                  dlast_state=dlast.to(dev))["dlog_decay"]
    want = state * dlast[0, :, 0, 0].double()
    ref.within(got, want, slack * want.abs(), "by the last state")
