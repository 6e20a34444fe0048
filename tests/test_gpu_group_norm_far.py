"""GPU tests of the group norm (include/ssm_group_norm.h) where a group's deviations are so large that their squares, or
they themselves, pass float32's range: a part of a group at the type's lowest value, as a mask leaves it.

Tolerance as in tests/test_gpu_group_norm.py: 160 half steps of float32 of the largest value, and the output's own
rounding.  rstd may be subnormal, and is then off by half of 2^-149 besides; the backward is held against the formula with
the mean and rstd that the forward returned."""
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


def far_rows(dt, groups, width, far, gen):
    """Rows of ordinary values: with the first group's first, half of it, and all but one at `far`; with values of both
    signs; and one left as it is."""
    x = torch.randn(5, groups * width, generator=gen).to(dt)
    x[0, 0] = far
    x[1, :(width + 1) // 2] = far
    x[2, :width - 1] = far
    x[3, :width:2] = far
    x[3, 1:width:2] = -far
    return x


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("width", [2, 8, 40, 128, 500, 1000, 1500, 2048, 4096, 8192])
@pytest.mark.parametrize("far", [1e20, -1e25, 1e33, "lowest"])
@pytest.mark.parametrize("gate", [True, False])
def test_far_values(dev, dtype, width, far, gate):
    import selective_state_space_28_amd as ssm
    dt = ref.TYPES[dtype]
    far = torch.finfo(dt).min if far == "lowest" else far
    gen = torch.Generator().manual_seed(width)
    groups = 3
    x = far_rows(dt, groups, width, far, gen).to(dev)
    dim = groups * width
    z = torch.randn(5, dim, generator=gen).to(dt).to(dev) if gate else None
    w, c = (1 + 0.3 * torch.randn(dim, generator=gen)).to(dev), (0.3 * torch.randn(dim, generator=gen)).to(dev)
    dy = torch.randn(5, dim, generator=gen).to(dt).to(dev)
    y, mean, rstd = ssm.ssm_group_norm_fwd(x, groups, w, c, z, act="silu", return_stats=True)
    want, wm, wr, n = ref.group_fwd(x, groups, w, c, z, "silu", 1e-5)
    top = n.abs().max() * (1.0 if z is None else max(1.0, ref.act("silu", z.cpu().double())[0].abs().max()))
    over = 1e37  # (the comparison's own slack of 1e-37 would hide what is smaller)
    size = x.cpu().double().abs().reshape(5, groups, width).amax(-1)
    ref.within(mean, wm, SLACK * size, "mean")
    ref.within(rstd.double() * over, wr * over, (SLACK * wr + 2.0 ** -150) * over, "rstd")
    ref.within(y, want, ref.HALF[dtype] * want.abs() + SLACK * top, "y")
    # the row and the groups without such values are what they are alone
    alone, m, r = ssm.ssm_group_norm_fwd(x[4:].clone(), groups, w, c, None if z is None else z[4:].clone(), act="silu",
                                         return_stats=True)
    assert torch.equal(alone[0], y[4]) and torch.equal(m[0], mean[4]) and torch.equal(r[0], rstd[4])

    g = ssm.ssm_group_norm_bwd(x, groups, w, c, z, act="silu", mean=mean, rstd=rstd, dy=dy)
    b = ref.group_bwd(x, groups, w, c, z, "silu", mean, rstd, dy)
    for name in ("dx", "dz", "dweight", "dbias"):
        if b[name] is None:
            assert g[name] is None
            continue
        if name == "dx":  # each group by its own size; subnormal results are off by half of their step
            size = b["size"]["dx"].reshape(5, groups, width).amax(-1, keepdim=True).expand(5, groups, width).reshape(5, dim)
            least = 2.0 ** (-134 if dtype == "bf16" else -150)
            bound = (ref.HALF[dtype] * b["dx"].abs() + SLACK * size + least) * over
            ref.within(g["dx"].double() * over, b["dx"] * over, bound, "dx")
            continue
        size = b["size"][name].max()
        if name == "dz":
            size = max(size, (dy.abs().max() * n.abs().max().item()).item())
            bound = ref.HALF[dtype] * b["dz"].abs() + SLACK * size
        else:
            terms = dy.cpu().double().abs() * (1.0 if name == "dbias" else (n.abs().max() + 1))
            bound = (SLACK + 5 * ref.EPS32) * (b["size"][name] + terms.sum(0)).max()
        ref.within(g[name], b[name], bound, name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("eps", [0.0, 1e30])
def test_far_values_and_eps(dev, dtype, eps):
    """The eps of a scaled variance is scaled with it."""
    import selective_state_space_28_amd as ssm
    gen = torch.Generator().manual_seed(3)
    x = far_rows(ref.TYPES[dtype], 2, 64, 3e19, gen).to(dev)
    y, mean, rstd = ssm.ssm_group_norm_fwd(x, 2, eps=eps, return_stats=True)
    want, _, wr, n = ref.group_fwd(x, 2, None, None, None, "none", eps)
    ref.within(rstd, wr, SLACK * wr, "rstd")
    ref.within(y, want, ref.HALF[dtype] * want.abs() + SLACK * n.abs().max(), "y")
