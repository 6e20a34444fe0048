"""GPU tests of the layer norm (include/ssm_norm.h) against its formula in 64
bits (tests/layers_ref.py).

Tolerance.  A sum of dim float32 terms added in a tree of lanes, waves and runs
of up to 32 terms is off by at most 40 half steps (2^-24) of the terms' sizes;
mean and variance are such sums, and an output takes a handful of roundings
more: 128 half steps of the largest value cover it when the values are within
a few times their spread.  A mean of m spreads costs the rounding of x - mean,
m half steps of a spread, and is added.  bfloat16 outputs add their rounding,
2^-8 of the value."""
import numpy as np
import pytest

import synth
from tests import layers_ref as ref
from tests.helpers import to_torch

pytestmark = pytest.mark.gpu

SLACK = 128 * ref.EPS32


@pytest.fixture(scope="module")
def dev():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import selective_state_space_28_amd as ssm
    ssm.load()
    return torch.device("cuda:0")


def draws(dtype, seed):
    rng = np.random.default_rng(seed)

    def tok(*shape, scale=1.0, mean=0.0):
        v = (rng.standard_normal(shape) * scale + mean).astype(np.float32)
        return synth.widen(synth.bf16_bits(v), "bf16") if dtype == "bf16" else v.astype(np.float64)

    def par(n, mean=0.0):
        return (rng.standard_normal(n) * 0.3 + mean).astype(np.float32).astype(np.float64)

    return tok, par


def place(v, dtype, dev, off=0):
    import torch
    if v is None:
        return None
    t = to_torch(v.astype(np.float32), "f32", dev).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    flat = torch.empty(t.numel() + off, dtype=t.dtype, device=dev)
    w = flat[off:].view(t.shape)
    w.copy_(t)
    return w


def np64(t):
    return None if t is None else t.float().cpu().numpy().astype(np.float64)


def check(dev, dtype, shape, axis, seed, *, residual=True, bias=True, eps=1e-5, mean=0.3, off=0):
    import selective_state_space_28_amd as ssm
    tok, par = draws(dtype, [seed, *shape])
    n = shape[axis]
    x, res = tok(*shape, mean=mean), tok(*shape) if residual else None
    w, b = par(n, 1.0), par(n) if bias else None
    dy, ds = tok(*shape), tok(*shape) if residual else None
    s = x
    if residual:
        s = (x + res).astype(np.float32)
        s = synth.widen(synth.bf16_bits(s), "bf16") if dtype == "bf16" else s.astype(np.float64)
    p = lambda v, t=dtype: place(v, t, dev, off)  # noqa: E731
    out = ssm.ssm_layer_norm_fwd(p(x), p(w, "f32"), p(b, "f32"), p(res), eps=eps, axis=axis, return_stats=True)
    slack = SLACK + abs(mean) * ref.EPS32
    yr, mr, rr = ref.norm_fwd(s, w, b, eps, axis)
    ref.close(np64(out[0]), yr, dtype, slack, "y")
    if residual:
        assert np.array_equal(np64(out[1]), s), "the sum, rounded once"
    ref.close(np64(out[-2]), mr, "f32", slack * max(1.0, 1.0 / max(np.abs(mr).max(), 1e-3)), "mean")
    ref.close(np64(out[-1]), rr, "f32", slack, "rstd")
    g = ssm.ssm_layer_norm_bwd(p(s), p(w, "f32"), out[-2], out[-1], p(dy), p(ds), axis=axis)
    gr = ref.norm_bwd(s, w, np64(out[-2]), np64(out[-1]), dy, ds, axis)
    # dx is a difference of rstd dn, rstd mean(dn) and rstd xhat mean(dn xhat), each with roundings relative to itself
    # and none larger than the token's largest rstd |dn| (|xhat| and the mean over it multiply to at most that, as
    # mean(xhat^2) <= 1 bounds mean(dn xhat) by the spread of dn, and xhat by sqrt(dim) only where the token is one
    # peak); where they cancel (dim = 1: dx = 0) the error is relative to them, not to dx
    wide = [1] * len(shape)
    wide[axis] = -1
    terms = np.abs(dy * w.reshape(wide)) * np.expand_dims(np64(out[-1]), axis)
    ref.close(np64(g["dx"]), gr["dx"], dtype, slack, "dx", np.maximum(terms, np.abs(gr["dx"])))
    over = tuple(k for k in range(len(shape)) if k != axis % len(shape))
    xh = (s - np.expand_dims(np64(out[-2]), axis)) * np.expand_dims(np64(out[-1]), axis)
    ref.close(np64(g["dweight"]), gr["dweight"], "f32", slack, "dweight", np.abs(dy * xh).sum(over))
    ref.close(np64(g["dbias"]), gr["dbias"], "f32", slack, "dbias", np.abs(dy).sum(over))
    return out, g


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [1, 2, 7, 8, 9, 63, 64, 100, 511, 512, 513, 1000, 1024, 1025, 1536, 2560, 5120, 8192,
                                 8193, 16385, 32768, 32769])
def test_rows(dev, dtype, dim):
    for rows in (1, 5):
        check(dev, dtype, (rows, dim), -1, dim, residual=dim % 2 == 0, bias=dim % 3 != 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,dim", [(2, 256), (17, 64), (255, 512), (1000, 96), (2049, 1536), (16400, 24), (4099, 7)])
def test_row_counts(dev, dtype, rows, dim):
    check(dev, dtype, (rows, dim), -1, 7)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("b,dim,L", [(1, 1, 2), (2, 5, 7), (1, 64, 31), (3, 16, 32), (2, 17, 33), (1, 100, 8),
                                     (1, 255, 9), (2, 257, 64), (1, 512, 65), (2, 1000, 100), (1, 2048, 37),
                                     (1, 5120, 66), (1, 5121, 5), (1, 9000, 40), (4, 96, 515), (40, 24, 130)])
def test_columns(dev, dtype, b, dim, L):
    check(dev, dtype, (b, dim, L), 1, 11, residual=(b + L) % 2 == 0, bias=L % 3 != 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("b,dim,L,residual", [(256, 500, 64, False), (260, 500, 20, True), (130, 700, 70, False),
                                              (260, 1100, 20, False), (260, 1100, 20, True), (130, 1300, 66, True),
                                              (260, 1500, 20, False), (260, 1600, 20, False)])
def test_columns_of_many_tiles(dev, dtype, b, dim, L, residual):
    """A line of 128 bytes to a channel's piece, held in registers, in LDS, and what neither holds."""
    check(dev, dtype, (b, dim, L), 1, 21, residual=residual)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_layouts_agree(dev, dtype):
    """The same tokens with their channels together and in the scans' layout."""
    import selective_state_space_28_amd as ssm
    tok, par = draws(dtype, 12)
    x, w, b = tok(3, 300, 45), par(300, 1.0), par(300)
    cols = ssm.ssm_layer_norm_fwd(place(x, dtype, dev), place(w, "f32", dev), place(b, "f32", dev), axis=1)
    rows = ssm.ssm_layer_norm_fwd(place(np.moveaxis(x, 1, 2).copy(), dtype, dev), place(w, "f32", dev),
                                  place(b, "f32", dev))
    assert rows.shape == (3, 45, 300)
    # two results, each rounded: they may stand half a step either side of the value, so each is compared with it
    yr = ref.norm_fwd(x, w, b, 1e-5, 1)[0]
    ref.close(np64(cols), yr, dtype, SLACK, "step-contiguous")
    ref.close(np.moveaxis(np64(rows), 1, 2), yr, dtype, SLACK, "channels together")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape,axis", [((5, 515), -1), ((2, 130, 67), 1)])
def test_unaligned_tensors_give_the_same_bits(dev, dtype, shape, axis):
    import torch
    a, ga = check(dev, dtype, shape, axis, 13)
    b, gb = check(dev, dtype, shape, axis, 13, off=1)
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    assert all(torch.equal(ga[k], gb[k]) for k in ga)


@pytest.mark.parametrize("shape,axis", [((4, 1000), -1), ((2, 300, 40), 1)])
def test_far_mean(dev, shape, axis):
    """A mean of 1000 spreads: the variance is taken about the mean, not as a difference of squares."""
    check(dev, "f32", shape, axis, 14, residual=False, mean=1000.0)


@pytest.mark.parametrize("shape,axis", [((3, 200), -1), ((2, 200, 9), 1)])
def test_constant_token(dev, shape, axis):
    """No spread at all: y is the bias, rstd 1/sqrt(eps); with eps = 0 it is NaN, as 0 * inf."""
    import torch
    import selective_state_space_28_amd as ssm
    x = torch.full(shape, 3.0, device=dev)
    w, b = torch.ones(200, device=dev), torch.linspace(-1, 1, 200, device=dev)
    y, mean, rstd = ssm.ssm_layer_norm_fwd(x, w, b, eps=1e-4, axis=axis, return_stats=True)
    assert bool((y == (b if axis == -1 else b[:, None])).all())
    assert bool((mean == 3).all()) and torch.allclose(rstd, torch.full_like(rstd, 100.0))
    assert torch.isnan(ssm.ssm_layer_norm_fwd(x, w, b, eps=0.0, axis=axis)).all()


@pytest.mark.parametrize("bad", [np.nan, np.inf])
@pytest.mark.parametrize("shape,axis,pos", [((6, 700), -1, (2, 5)), ((2, 300, 40), 1, (1, 7, 33))])
def test_non_finite_values_stay_in_their_token(dev, shape, axis, pos, bad):
    import torch
    import selective_state_space_28_amd as ssm
    tok, par = draws("f32", 15)
    x, dy, w = tok(*shape), tok(*shape), par(shape[axis], 1.0)
    y, m, r = ssm.ssm_layer_norm_fwd(place(x, "f32", dev), place(w, "f32", dev), axis=axis, return_stats=True)
    g = ssm.ssm_layer_norm_bwd(place(x, "f32", dev), place(w, "f32", dev), m, r, place(dy, "f32", dev), axis=axis)
    x[pos] = bad
    y2, m2, r2 = ssm.ssm_layer_norm_fwd(place(x, "f32", dev), place(w, "f32", dev), axis=axis, return_stats=True)
    g2 = ssm.ssm_layer_norm_bwd(place(x, "f32", dev), place(w, "f32", dev), m2, r2, place(dy, "f32", dev), axis=axis)
    token = (pos[0],) if axis == -1 else (pos[0], slice(None), pos[2])
    for u, v in ((y, y2), (g["dx"], g2["dx"])):
        assert torch.isnan(v[token]).all()
        v = v.clone()
        v[token] = u[token]
        assert torch.equal(u, v)


def test_two_runs_give_the_same_bits(dev):
    import torch
    for shape, axis in (((3000, 520), -1), ((3, 520, 300), 1)):
        a, ga = check(dev, "bf16", shape, axis, 16)
        b, gb = check(dev, "bf16", shape, axis, 16)
        assert all(torch.equal(u, v) for u, v in zip(a, b)) and all(torch.equal(ga[k], gb[k]) for k in ga)


def test_empty_problems(dev):
    import torch
    import selective_state_space_28_amd as ssm
    w = torch.ones(6, device=dev)
    for x, axis in ((torch.empty(0, 6, device=dev), -1), (torch.empty(2, 6, 0, device=dev), 1)):
        y, m, r = ssm.ssm_layer_norm_fwd(x, w, axis=axis, return_stats=True)
        g = ssm.ssm_layer_norm_bwd(x, w, m, r, x, axis=axis)
        assert y.shape == x.shape and g["dx"].shape == x.shape
        assert not g["dweight"].abs().max().item() and not g["dbias"].abs().max().item()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape,axis", [((3, 515), -1), ((1, 19, 35), 1), ((5, 4200), -1)])
def test_nothing_is_written_beside_the_outputs(dev, dtype, shape, axis):
    import torch
    import selective_state_space_28_amd as ssm
    tok, par = draws(dtype, 17)
    x, w = place(tok(*shape), dtype, dev), place(par(shape[axis], 1.0), "f32", dev)
    n = x.numel()
    buf = torch.full((n + 39,), 7.0, dtype=x.dtype, device=dev)
    y = ssm.ssm_layer_norm_fwd(x, w, axis=axis, out=buf[19:19 + n].view(shape))
    torch.cuda.synchronize()
    assert torch.equal(y, ssm.ssm_layer_norm_fwd(x, w, axis=axis))
    assert bool((buf[:19] == 7).all()) and bool((buf[19 + n:] == 7).all())


def test_offsets_past_32_bits(dev):
    """More than 2^31 elements in either layout: the last tokens are those of a call on them alone.  Another number of
    tokens may add the channels in another order: two roundings to bf16 of values that agree to float32 are then at
    most a step apart, 2^-7 of the value (a value near 0, of float32's error of the largest)."""
    import torch
    import selective_state_space_28_amd as ssm
    w = torch.linspace(0.5, 1.5, 4096, device=dev)
    x = torch.empty((540000, 4096), dtype=torch.bfloat16, device=dev)
    gen = torch.Generator(device=dev)
    gen.manual_seed(3)
    for k in range(0, 540000, 60000):
        x[k:k + 60000].normal_(generator=gen)
    y, m, r = ssm.ssm_layer_norm_fwd(x, w, return_stats=True)
    assert torch.equal(y[-1:], ssm.ssm_layer_norm_fwd(x[-1:].contiguous(), w))
    g = ssm.ssm_layer_norm_bwd(x, w, m, r, y)
    assert torch.equal(g["dx"][-1:], ssm.ssm_layer_norm_bwd(x[-1:], w, m[-1:], r[-1:], y[-1:])["dx"])
    del y, g
    x = x.view(1, 4096, 540000)
    y, m, r = ssm.ssm_layer_norm_fwd(x, w, axis=1, return_stats=True)
    end = x[:, :, -64:].contiguous()
    near = lambda u, v: bool(((u.float() - v.float()).abs()  # noqa: E731
                              <= 2.0 ** -7 * v.float().abs() + 4 * SLACK).all())
    assert near(y[:, :, -64:], ssm.ssm_layer_norm_fwd(end, w, axis=1))
    g = ssm.ssm_layer_norm_bwd(x, w, m, r, y, axis=1)
    one = ssm.ssm_layer_norm_bwd(end, w, m[:, -64:].contiguous(), r[:, -64:].contiguous(), y[:, :, -64:].contiguous(), axis=1)
    assert near(g["dx"][:, :, -64:], one["dx"])


def test_more_threads_than_a_grid_dimension_has(dev):
    """2^32 threads and more: tokens in the middle and at the end are those of a call on them alone, and none is left out."""
    import torch
    import selective_state_space_28_amd as ssm
    gen = torch.Generator(device=dev)
    gen.manual_seed(8)
    w = torch.tensor([0.5, 1.25, -2.0], device=dev)
    # a workgroup a token
    x = torch.empty((2**23 + 5, 3, 2), dtype=torch.bfloat16, device=dev).normal_(generator=gen)
    y = ssm.ssm_layer_norm_fwd(x, w, axis=1, out=torch.full_like(x, float("nan")))
    assert not bool(y.isnan().any())
    for at in (0, 2**22, 2**23 - 9):
        assert torch.equal(y[at:at + 14], ssm.ssm_layer_norm_fwd(x[at:at + 14], w, axis=1))
    # eight lanes a row
    x = torch.empty((2**29 + 7, 2), dtype=torch.bfloat16, device=dev).normal_(generator=gen)
    y = ssm.ssm_layer_norm_fwd(x, w[:2], out=torch.full_like(x, float("nan")))
    assert not bool(y.isnan().any())
    for at in (0, 2**28, 2**29 - 9):
        assert torch.equal(y[at:at + 16], ssm.ssm_layer_norm_fwd(x[at:at + 16], w[:2]))
    del x, y
    # as many sums as channels: one token's are its dy, and dy xhat rounded once
    d = 2**26 + 3
    x = torch.empty((1, d), dtype=torch.bfloat16, device=dev).normal_(generator=gen)
    one = torch.ones(d, device=dev)
    m, r = torch.zeros(1, device=dev), torch.ones(1, device=dev)
    g = ssm.ssm_layer_norm_bwd(x, one, m, r, x)
    assert torch.equal(g["dbias"], x[0].float()) and torch.equal(g["dweight"], x[0].float() ** 2)


def test_refusals(dev):
    import torch
    import selective_state_space_28_amd as ssm
    x, w = torch.randn(4, 6, 5, device=dev), torch.ones(5, device=dev)
    with pytest.raises(TypeError):
        ssm.ssm_layer_norm_fwd(x.half(), w)
    with pytest.raises(ValueError):
        ssm.ssm_layer_norm_fwd(x.transpose(0, 1), w)
    with pytest.raises(ValueError):
        ssm.ssm_layer_norm_fwd(x, torch.ones(6, device=dev))
    with pytest.raises(TypeError):
        ssm.ssm_layer_norm_fwd(x, w.bfloat16())
    with pytest.raises(ValueError):
        ssm.ssm_layer_norm_fwd(x, w, axis=0)
    with pytest.raises(TypeError):
        ssm.ssm_layer_norm_fwd(x, w, None, x.bfloat16())
    with pytest.raises(ssm.SsmError, match="ALIAS"):
        ssm.ssm_layer_norm_fwd(x, w, out=x)
    with pytest.raises(ssm.SsmError, match="SHAPE"):
        ssm.ssm_layer_norm_fwd(x, w, eps=-1.0)
    with pytest.raises(ssm.SsmError, match="SHAPE"):
        ssm.ssm_layer_norm_fwd(torch.empty(3, 0, device=dev), torch.empty(0, device=dev))
    y, m, r = ssm.ssm_layer_norm_fwd(x, w, return_stats=True)
    with pytest.raises(ValueError):
        ssm.ssm_layer_norm_bwd(x, w, m[:2], r, y)
    with pytest.raises(TypeError):
        ssm.ssm_layer_norm_bwd(x, w, m, r, y.bfloat16())
