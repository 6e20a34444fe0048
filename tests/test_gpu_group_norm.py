"""GPU tests of the group norm (include/ssm_group_norm.h) against its formula in 64
bits (tests/heads_ref.py).

Tolerance.  A sum of a group's terms, in runs of up to 32 and a tree of lanes and
waves, is off by at most 40 half steps (2^-24) of the terms' sizes; mean and
variance are such sums, n takes a handful of roundings more, and the activation
some 16 (the exponential's argument of up to 10 is rounded, which moves it by 10
half steps): 160 half steps of the largest value cover it when the values are
within a few times their spread.  bfloat16 outputs add their rounding, 2^-8 of the
value.  A sum over tokens adds a half step of its size for each."""
import pytest
import torch

from tests import heads_ref as ref

pytestmark = pytest.mark.gpu

SLACK = 160 * ref.EPS32


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import selective_state_space_28_amd as ssm
    ssm.load()
    return torch.device("cuda:0")


def check(dev, dtype, lead, groups, width, *, gate=True, act="silu", affine=(True, True), eps=1e-5, seed=0, off=0,
          fused=False):
    import selective_state_space_28_amd as ssm
    gen = torch.Generator().manual_seed(seed * 1009 + groups * 31 + width)
    dim, dt = groups * width, ref.TYPES[dtype]

    def put(t):
        flat = torch.empty(t.numel() + off, dtype=t.dtype, device=dev)[off:]
        return flat.copy_(t.flatten()).view(t.shape)

    def draw(*shape, dtype=dt, mean=0.0):
        return put((torch.randn(shape, generator=gen) + mean).to(dtype))

    if fused:
        rows = draw(*lead, 3 * dim, mean=0.3)
        x, z = rows[..., dim:2 * dim], rows[..., 2 * dim:]
    else:
        x, z = draw(*lead, dim, mean=0.3), draw(*lead, dim)
    if not gate:
        z = None
    w = put(1 + 0.3 * torch.randn(dim, generator=gen)) if affine[0] else None
    c = put(0.3 * torch.randn(dim, generator=gen)) if affine[1] else None
    dy = draw(*lead, dim)
    y, mean, rstd = ssm.ssm_group_norm_fwd(x, groups, w, c, z, act=act, eps=eps, return_stats=True)
    want, wm, wr, n = ref.group_fwd(x, groups, w, c, z, act, eps)
    top = n.abs().max() * (1.0 if z is None else max(1.0, ref.act(act, z.cpu().double())[0].abs().max()))
    ref.within(mean, wm, SLACK * x.abs().max().item(), "mean")
    ref.within(rstd, wr, SLACK * wr.abs().max(), "rstd")
    ref.within(y, want, ref.HALF[dtype] * want.abs() + SLACK * top, "y")
    g = ssm.ssm_group_norm_bwd(x, groups, w, c, z, act=act, mean=mean, rstd=rstd, dy=dy)
    r = ref.group_bwd(x, groups, w, c, z, act, mean, rstd, dy)
    tokens = max(1, x.numel() // dim)
    for name in ("dx", "dz", "dweight", "dbias"):
        if r[name] is None or (name == "dweight" and w is None) or (name == "dbias" and c is None):
            assert g[name] is None, name
            continue
        size = r["size"][name].max()
        if name in ("dx", "dz"):
            size = max(size, (dy.abs().max() * n.abs().max().item()).item() if name == "dz" else 0.0)
            bound = ref.HALF[dtype] * r[name].abs() + SLACK * size
        else:  # the derivative of an activation is off by SLACK of at most 1.1, whatever it is itself
            terms = dy.cpu().double().abs() * (1.0 if name == "dbias" else (n.abs().max() + 1))
            bound = (SLACK + tokens * ref.EPS32) * (r["size"][name] + terms.flatten(0, -2).sum(0)).max()
        ref.within(g[name], r[name], bound, name)
    return y, g


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("width", [1, 2, 3, 7, 8, 9, 15, 16, 17, 31, 32, 33, 64, 65, 100, 128, 129, 200, 256, 257, 500, 512, 513,
                                   1000, 1024, 1025, 2000, 2048, 2049, 4096, 4097, 8000, 8192])
def test_widths(dev, dtype, width):
    for groups in (1, 3):
        check(dev, dtype, (5,), groups, width, seed=width)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tokens,groups,width", [(1, 40, 128), (2, 5, 16), (17, 1, 8), (1000, 7, 24), (3001, 10, 100),
                                                 (4099, 2, 3), (700, 40, 64), (9000, 1, 1), (2500, 3, 600), (300, 2, 4096)])
def test_tokens(dev, dtype, tokens, groups, width):
    check(dev, dtype, (tokens,), groups, width, seed=1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("act", ["none", "silu", "sigmoid"])
@pytest.mark.parametrize("affine", [(True, True), (True, False), (False, True), (False, False)])
def test_forms(dev, dtype, gate, act, affine):
    check(dev, dtype, (2, 9), 6, 40, gate=gate, act=act, affine=affine, seed=2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("width", [8, 40, 33])
@pytest.mark.parametrize("off", [0, 1, 4])
def test_strided_and_unaligned(dev, dtype, width, off):
    check(dev, dtype, (3, 7), 4, width, fused=True, off=off, seed=3)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_equal_values_and_ends(dev, dtype):
    import selective_state_space_28_amd as ssm
    dt = ref.TYPES[dtype]
    low = torch.finfo(dt).min
    x = torch.zeros(6, 96, dtype=dt, device=dev)
    for r, v in enumerate((0.0, 1.1, -7.3e4, low, -low, 3.3e-30)):
        x[r] = v
    c = torch.randn(96, device=dev)
    y, mean, rstd = ssm.ssm_group_norm_fwd(x, 3, None, c, return_stats=True)
    assert torch.equal(mean, x.float()[:, ::32])
    assert torch.equal(y, c.to(dt).expand_as(y))
    ref.within(rstd, torch.full(rstd.shape, 1e-5 ** -0.5, dtype=torch.float64), SLACK * 1e-5 ** -0.5, "rstd")
    # one group of the lowest value (a mask) beside others: they are what they were
    x = torch.randn(4, 96, device=dev).to(dt)
    z = torch.randn(4, 96, device=dev).to(dt)
    clean = ssm.ssm_group_norm_fwd(x, 3, None, c, z, act="silu")
    for v in (low, float("nan"), float("inf"), float("-inf")):
        x2 = x.clone()
        x2[1, 32:64] = v
        y = ssm.ssm_group_norm_fwd(x2, 3, None, c, z, act="silu")
        keep = torch.ones_like(x, dtype=torch.bool)
        keep[1, 32:64] = False
        assert torch.equal(y[keep], clean[keep])
        if v == low:
            assert torch.isfinite(y).all()
        else:
            assert torch.isnan(y[1, 32:64]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gates_far_out(dev, dtype):
    import selective_state_space_28_amd as ssm
    dt = ref.TYPES[dtype]
    big = torch.finfo(dt).max
    x = torch.randn(2, 32, device=dev).to(dt)
    z = torch.tensor([-big, big, -200.0, 200.0, -90.0, 90.0, 0.0, -0.0], device=dev).to(dt).repeat(2, 4)
    z[:, 1::8] = 1e30
    for act in ("silu", "sigmoid"):
        y, mean, rstd = ssm.ssm_group_norm_fwd(x, 2, None, None, z, act=act, return_stats=True)
        want, _, _, n = ref.group_fwd(x, 2, None, None, z, act, 1e-5)
        ok = want.abs() < big
        # y = n act(z): n is off by SLACK of its largest, which act(z) of up to 1e30 multiplies; act(z) itself is off by
        # SLACK of its size (e^-z by |z| half steps, where that is at most 200 or the exponential has no weight)
        gate = ref.act(act, z.cpu().double())[0].abs()
        ref.within(torch.where(ok.to(dev), y, 0), torch.where(ok, want, 0.0),
                   ref.HALF[dtype] * want.abs() + SLACK * (n.abs().max() + n.abs()) * gate + 1e-30, act)
        g = ssm.ssm_group_norm_bwd(x, 2, None, None, z, act=act, mean=mean, rstd=rstd, dy=torch.ones_like(x))
        assert torch.isfinite(g["dz"]).all()
        r = ref.group_bwd(x, 2, None, None, z, act, mean, rstd, torch.ones_like(x))
        ref.within(g["dz"], r["dz"], ref.HALF[dtype] * r["dz"].abs() + SLACK * 300, "dz")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_empty(dev, dtype):
    import selective_state_space_28_amd as ssm
    dt = ref.TYPES[dtype]
    x, w = torch.empty(0, 64, dtype=dt, device=dev), torch.ones(64, device=dev)
    y, mean, rstd = ssm.ssm_group_norm_fwd(x, 4, w, w.clone(), return_stats=True)
    assert y.shape == (0, 64) and mean.shape == (0, 4)
    g = ssm.ssm_group_norm_bwd(x, 4, w, w.clone(), mean=mean, rstd=rstd, dy=x)
    assert not g["dweight"].any() and not g["dbias"].any()
