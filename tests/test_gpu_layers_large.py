"""GPU tests of the gated recurrence and the layer norm at the sizes that
training takes: the variants which smaller calls do not reach (a wave to a row
over many blocks, inputs read past the caches, whole lines written past them,
long sums), against 64 bits.

Tolerances as in the tests of the small sizes: a state is within 32 half steps
of float32 (2^-24) times the steps that a decay's error stays in it, a gradient
three times that; a norm's results within 128 half steps of the largest; what
is stored as bfloat16 rounds by 2^-8 of the value.  A sum is off by its terms'
errors, and by half a step of its terms' sizes for each addition in a chain."""
import pytest

from tests import layers_ref as ref
from tests import layers_torch_ref as tref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import selective_state_space_28_amd as ssm
    ssm.load()
    return torch.device("cuda:0")


def check_scan(dev, dtype, b, d, L, seed, *, gate="sigmoid", weight="unit", i=True, z=True, packed=False, h0=True,
               channels=None):
    """Forward and gradients, of every channel or of `channels` of them spread over all."""
    import torch
    import selective_state_space_28_amd as ssm
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    rnd = lambda *s: torch.randn(s, generator=gen, device=dev)  # noqa: E731
    tok = lambda: rnd(b, d, L).clamp_(-4, 4).to(dt)  # noqa: E731
    x, r, dy = tok(), tok(), tok()
    gi, gz = tok() if i else None, tok() if z else None
    A, rb = -0.2 - 1.8 * torch.rand(d, generator=gen, device=dev), 0.3 * rnd(d)
    ib = 0.3 * rnd(d) if i else None
    start = rnd(b, d) if h0 else None
    dl = rnd(b, d)
    starts = None
    if packed:
        starts = (torch.rand((b, L), generator=gen, device=dev) < 4.0 / L).to(torch.uint8)
        starts[0, [0, L - 1]] = 1
    kw = dict(gate=gate, weight=weight, starts=starts)
    y, last, ckpt = ssm.ssm_gated_scan_fwd(x, r, A, rb, gi, ib, gz, h0=start, return_last_state=True, return_ckpt=True,
                                           **kw)
    g = ssm.ssm_gated_scan_bwd(x, r, A, rb, gi, ib, gz, ckpt=ckpt, dy=dy, dlast_state=dl, **kw)
    at = slice(None)
    if channels is not None:
        at = torch.linspace(0, d - 1, channels, device=dev).long()
    cut = lambda v: None if v is None else v[at] if v.dim() == 1 else v[:, at]  # noqa: E731
    yr, lr, before, want = tref.gated(cut(x), cut(r), cut(A), cut(rb), cut(gi), cut(ib), cut(gz), h0=cut(start),
                                      dy=cut(dy), dlast=cut(dl), **kw)
    # the decay nearest 1 is that of the most closed gate
    pre = (cut(r).double() + cut(rb).double()[:, None]).amin((0, 2))
    g_min = torch.sigmoid(pre) if gate == "sigmoid" else torch.nn.functional.softplus(pre)
    memory = min(L, 1.0 / (1.0 - torch.exp(cut(A).double() * g_min).max().item())) + 1.0
    slack, half = 32 * ref.EPS32 * memory, ref.HALF[dtype]
    tref.close(cut(y), yr, half, slack, "y")
    tref.close(cut(last), lr, ref.EPS32, slack, "last_state")
    entering = before[:, :, ::512].transpose(1, 2)
    if packed:  # kept as it was before a start
        entering = torch.where(starts[:, ::512, None] != 0, ckpt[:, :, at].double(), entering)
    tref.close(ckpt[:, :, at], entering, ref.EPS32, slack, "ckpt")
    for k in ("dx", "dr", "di", "dz", "dA", "dr_bias", "di_bias", "dh0"):
        if want[k] is not None:
            tref.close(cut(g[k]), want[k], half if k in ("dx", "dr", "di", "dz") else ref.EPS32, 3 * slack, k,
                       want["size"].get(k))


@pytest.mark.parametrize("gate,weight,i,z", [("sigmoid", "unit", True, True), ("softplus", "convex", True, False),
                                             ("softplus", "unit", False, True)])
@pytest.mark.parametrize("packed,h0", [(False, True), (False, False), (True, True)])
@pytest.mark.parametrize("L", [1100, 1536])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_wave_a_row_over_several_blocks(dev, dtype, L, packed, h0, gate, weight, i, z):
    check_scan(dev, dtype, 2, 4100, L, 1, gate=gate, weight=weight, i=i, z=z, packed=packed, h0=h0)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtype,b,d,L", [("bf16", 2, 4096, 6720), ("f32", 2, 4096, 3360),       # a wave to a row
                                         ("bf16", 1, 2048, 26304), ("f32", 1, 2048, 13120),     # four
                                         ("bf16", 1, 512, 104896), ("f32", 1, 512, 52480)])     # sixteen
def test_inputs_read_past_the_caches(dev, dtype, b, d, L, packed):
    """Whole lines and more than 512 MiB of tensors in either direction; the last blocks are not whole."""
    assert b * d * L * (2 if dtype == "bf16" else 4) * 5 > 2**29
    check_scan(dev, dtype, b, d, L, 2, packed=packed, channels=40)


@pytest.mark.parametrize("gate,weight", [("sigmoid", "unit"), ("softplus", "convex")])
@pytest.mark.parametrize("b,d,L", [(300, 70, 40), (4097, 5, 17), (257, 300, 3)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sums_over_many_sequences(dev, dtype, b, d, L, gate, weight):
    check_scan(dev, dtype, b, d, L, 3, gate=gate, weight=weight, z=False)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dim", [96, 700, 1300, 2570, 5120, 5121, 8200])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_columns_of_whole_lines(dev, dtype, dim, residual):
    """Two lines to a row of every channel, enough of them for the chip: the channels fill the registers, then LDS,
    and are then read again."""
    import torch
    import selective_state_space_28_amd as ssm
    dt, L = (torch.bfloat16, 128) if dtype == "bf16" else (torch.float32, 64)
    gen = torch.Generator(device=dev)
    gen.manual_seed(dim)
    rnd = lambda *s: torch.randn(s, generator=gen, device=dev)  # noqa: E731
    b = 130
    x, dy = (rnd(b, dim, L) + 0.3).to(dt), rnd(b, dim, L).to(dt)
    res, ds = (rnd(b, dim, L).to(dt), rnd(b, dim, L).to(dt)) if residual else (None, None)
    w, bias = 1 + 0.3 * rnd(dim), 0.3 * rnd(dim)
    out = ssm.ssm_layer_norm_fwd(x, w, bias, res, axis=1, return_stats=True)
    s = x if res is None else (x.float() + res.float()).to(dt)
    if residual:
        assert torch.equal(out[1], s)
    s64, w64 = s.double(), w.double()[:, None]
    mean, var = s64.mean(1, keepdim=True), s64.var(1, unbiased=False, keepdim=True)
    rstd = (var + 1e-5).rsqrt()
    half, slack = ref.HALF[dtype], 129 * ref.EPS32
    tref.close(out[0], (s64 - mean) * rstd * w64 + bias.double()[:, None], half, slack, "y")
    tref.close(out[-2], mean[:, 0], ref.EPS32, slack, "mean", torch.ones((), device=dev))
    tref.close(out[-1], rstd[:, 0], ref.EPS32, slack, "rstd")
    g = ssm.ssm_layer_norm_bwd(s, w, out[-2], out[-1], dy, ds, axis=1)
    rs = out[-1].double()[:, None]
    xh, d64 = (s64 - out[-2].double()[:, None]) * rs, dy.double()
    tref.close(g["dweight"], (d64 * xh).sum((0, 2)), ref.EPS32, slack, "dweight", (d64 * xh).abs().sum((0, 2)))
    tref.close(g["dbias"], d64.sum((0, 2)), ref.EPS32, slack, "dbias", d64.abs().sum((0, 2)))
    dn = d64 * w64
    dx = rs * (dn - dn.mean(1, keepdim=True) - xh * (dn * xh).mean(1, keepdim=True))
    tref.close(g["dx"], dx if ds is None else dx + ds.double(), half, slack, "dx")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,dim", [(400000, 1100), (1000003, 40)])
def test_gradients_of_many_tokens(dev, dtype, rows, dim):
    """dweight and dbias over half a million tokens: a workgroup of 768 adds some 550 rows one after another (of few
    channels, 512 workgroups of 64 rows at a time some 32), and the sums of the workgroups follow."""
    import torch
    import selective_state_space_28_amd as ssm
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    gen = torch.Generator(device=dev)
    gen.manual_seed(dim)
    x = torch.empty((rows, dim), dtype=dt, device=dev).normal_(generator=gen)
    dy = torch.empty_like(x).normal_(generator=gen)
    w = 1 + 0.3 * torch.randn(dim, generator=gen, device=dev)
    _, m, rs = ssm.ssm_layer_norm_fwd(x, w, return_stats=True)
    g = ssm.ssm_layer_norm_bwd(x, w, m, rs, dy)
    dw = torch.zeros((2, dim), dtype=torch.float64, device=dev)
    db = torch.zeros_like(dw)
    for k in range(0, rows, 50000):
        at = slice(k, k + 50000)
        d64 = dy[at].double()
        t = d64 * (x[at].double() - m[at].double()[:, None]) * rs[at].double()[:, None]
        dw += torch.stack([t.sum(0), t.abs().sum(0)])
        db += torch.stack([d64.sum(0), d64.abs().sum(0)])
    slack = (128 + (rows // 700 if dim > 1000 else 64)) * ref.EPS32
    for name, s in (("dweight", dw), ("dbias", db)):
        bound = slack * s[1]
        assert bool(((g[name].double() - s[0]).abs() <= bound).all()), name
