"""The gated recurrence and the layer norm as a model uses them: two recurrent
blocks trained by hand-chained backward calls against autograd in 64 bits, the
same blocks generating token by token after a prompt, captured training steps,
other streams, and the large step-contiguous norms that keep part of a tile in
registers, part in LDS and read the rest again."""
import numpy as np
import pytest

from tests import layers_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import selective_state_space_28_amd as ssm
    ssm.load()
    return torch.device("cuda:0")


DM, D = 24, 40  # width of the residual stream, channels of the recurrence
NAMES = ("w1", "b1", "Wx", "Wr", "Wi", "Wz", "A", "rb", "ib", "w2", "b2", "Wo")


def make_block(seed):
    import torch
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s, scale=1.0: torch.randn(*s, generator=gen, dtype=torch.float64) * scale  # noqa: E731
    p = dict(w1=1 + n(DM, scale=0.1), b1=n(DM, scale=0.1), w2=1 + n(D, scale=0.1), b2=n(D, scale=0.1),
             A=-0.1 - 0.4 * torch.rand(D, generator=gen, dtype=torch.float64), rb=n(D, scale=0.1), ib=n(D, scale=0.1),
             Wo=n(DM, D, scale=D ** -0.5))
    for k in ("Wx", "Wr", "Wi", "Wz"):
        p[k] = n(D, DM, scale=DM ** -0.5)
    return {k: v.float().double() for k, v in p.items()}


def block64(p, x, res, starts):
    """Autograd in float64 on the CPU.  x, res: (batch, L, DM); returns (block output, residual stream)."""
    import torch
    import torch.nn.functional as F
    res = x + res
    u = F.layer_norm(res, (DM,), p["w1"], p["b1"], 1e-5).transpose(1, 2)
    xx, r, i, z = (p[k] @ u for k in ("Wx", "Wr", "Wi", "Wz"))
    a = torch.exp(p["A"][:, None] * torch.sigmoid(r + p["rb"][:, None]))
    v = torch.sqrt(1 - a * a) * torch.sigmoid(i + p["ib"][:, None]) * xx
    h, ys = torch.zeros_like(v[:, :, 0]), []
    for t in range(v.shape[2]):
        h = a[:, :, t] * torch.where(starts[:, t, None] != 0, torch.zeros_like(h), h) + v[:, :, t]
        ys.append(h)
    y = torch.stack(ys, 2) * F.silu(z)
    y = F.layer_norm(y.transpose(1, 2), (D,), p["w2"], p["b2"], 1e-5).transpose(1, 2)
    return (p["Wo"] @ y).transpose(1, 2), res


def block_fwd(ssm, p, x, res, starts):
    res_in = res
    u, res, m1, s1 = ssm.ssm_layer_norm_fwd(x, p["w1"], p["b1"], res_in, return_stats=True)
    ut = u.transpose(1, 2).contiguous()
    xx, r, i, z = ((p[k] @ ut).contiguous() for k in ("Wx", "Wr", "Wi", "Wz"))
    y, ck = ssm.ssm_gated_scan_fwd(xx, r, p["A"], p["rb"], i, p["ib"], z, starts=starts, return_ckpt=True)
    yn, m2, s2 = ssm.ssm_layer_norm_fwd(y, p["w2"], p["b2"], axis=1, return_stats=True)
    out = (p["Wo"] @ yn).transpose(1, 2).contiguous()
    return out, res, (ut, xx, r, i, z, y, ck, yn, m1, s1, m2, s2, res)


def block_bwd(ssm, p, kept, dout, dres, starts):
    """(gradient of x and of the incoming residual alike, of the parameters)."""
    ut, xx, r, i, z, y, ck, yn, m1, s1, m2, s2, res = kept
    dot = dout.transpose(1, 2).contiguous()
    g = {"Wo": (dot @ yn.transpose(1, 2).contiguous()).sum(0)}
    n2 = ssm.ssm_layer_norm_bwd(y, p["w2"], m2, s2, p["Wo"].t().contiguous() @ dot, axis=1)
    sc = ssm.ssm_gated_scan_bwd(xx, r, p["A"], p["rb"], i, p["ib"], z, starts=starts, ckpt=ck, dy=n2["dx"])
    du = 0
    utt = ut.transpose(1, 2).contiguous()
    for k, d in (("Wx", "dx"), ("Wr", "dr"), ("Wi", "di"), ("Wz", "dz")):
        g[k] = (sc[d] @ utt).sum(0)
        du = du + p[k].t().contiguous() @ sc[d]
    n1 = ssm.ssm_layer_norm_bwd(res, p["w1"], m1, s1, du.transpose(1, 2).contiguous(), dres)
    g.update(A=sc["dA"], rb=sc["dr_bias"], ib=sc["di_bias"], w1=n1["dweight"], b1=n1["dbias"], w2=n2["dweight"],
             b2=n2["dbias"])
    return n1["dx"], g


def test_two_blocks_train_as_autograd(dev):
    """Every gradient of two stacked blocks on packed sequences.  float32 throughout: each of some 20 operations in a
    row is good to 128 half steps (2^-24) of its largest value, the recurrence to its memory of some 50 steps more;
    their product with the gains of the projections (near 1) stays under 20 * 128 * 50 half steps, 8e-3 of the largest
    gradient; a wrong term is of its own size."""
    import torch
    import selective_state_space_28_amd as ssm
    gen = torch.Generator().manual_seed(3)
    b, L = 2, 530
    x = torch.randn(b, L, DM, generator=gen).double()
    res = torch.randn(b, L, DM, generator=gen).double()
    dout = torch.randn(b, L, DM, generator=gen).double()
    dres = torch.randn(b, L, DM, generator=gen).double()
    starts = (torch.rand(b, L, generator=gen) < 0.01).to(torch.uint8)
    blocks = [make_block(k) for k in (1, 2)]
    leaves = [{k: v.clone().requires_grad_() for k, v in p.items()} for p in blocks]
    x64, r64 = x.clone().requires_grad_(), res.clone().requires_grad_()
    o, r_ = block64(leaves[0], x64, r64, starts)
    o, r_ = block64(leaves[1], o, r_, starts)
    ((o * dout).sum() + (r_ * dres).sum()).backward()

    g = lambda v: v.float().to(dev)  # noqa: E731
    ps = [{k: g(v) for k, v in p.items()} for p in blocks]
    st = starts.to(dev)
    o1, s1, k1 = block_fwd(ssm, ps[0], g(x), g(res), st)
    o2, s2, k2 = block_fwd(ssm, ps[1], o1, s1, st)
    slack = 20 * 128 * 50 * ref.EPS32
    ref.close(o2.cpu().numpy(), o.detach().numpy(), "f32", slack, "output")
    ref.close(s2.cpu().numpy(), r_.detach().numpy(), "f32", slack, "residual stream")
    d, g2 = block_bwd(ssm, ps[1], k2, g(dout), g(dres), st)
    d, g1 = block_bwd(ssm, ps[0], k1, d, d, st)
    ref.close(d.cpu().numpy(), x64.grad.numpy(), "f32", slack, "dx")
    ref.close(d.cpu().numpy(), r64.grad.numpy(), "f32", slack, "dresidual")
    for n, (mine, leaf) in enumerate(((g1, leaves[0]), (g2, leaves[1]))):
        for k in NAMES:
            ref.close(mine[k].cpu().numpy(), leaf[k].grad.numpy(), "f32", slack, f"block {n} d{k}")


def test_prompt_then_tokens(dev):
    """A block over a prompt, then over tokens one at a time from its state: what it gives over the whole."""
    import torch
    import selective_state_space_28_amd as ssm
    p = {k: v.float().to(dev) for k, v in make_block(5).items()}
    gen = torch.Generator().manual_seed(6)
    b, L, cut = 3, 140, 133
    x, res = (torch.randn(b, L, DM, generator=gen).to(dev) for _ in range(2))
    starts = torch.zeros(b, L, dtype=torch.uint8, device=dev)
    whole, stream, _ = block_fwd(ssm, p, x, res, starts)
    u, _ = ssm.ssm_layer_norm_fwd(x[:, :cut].contiguous(), p["w1"], p["b1"], res[:, :cut].contiguous())
    ut = u.transpose(1, 2).contiguous()
    _, state = ssm.ssm_gated_scan_fwd((p["Wx"] @ ut).contiguous(), (p["Wr"] @ ut).contiguous(), p["A"], p["rb"],
                                      (p["Wi"] @ ut).contiguous(), p["ib"], return_last_state=True)
    for t in range(cut, L):
        u, s = ssm.ssm_layer_norm_fwd(x[:, t].contiguous(), p["w1"], p["b1"], res[:, t].contiguous())
        xx, r, i, z = ((u @ p[k].t()).contiguous() for k in ("Wx", "Wr", "Wi", "Wz"))
        y = ssm.ssm_gated_state_update(state, xx, r, p["A"], p["rb"], i, p["ib"], z)
        out = ssm.ssm_layer_norm_fwd(y, p["w2"], p["b2"]) @ p["Wo"].t()
        assert torch.equal(s, stream[:, t])
        assert (out - whole[:, t]).abs().max().item() <= 20 * 128 * 50 * ref.EPS32 * whole.abs().max().item(), t


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("b,d,L", [(2, 70, 530), (3, 9, 100), (1, 300, 5000)])
def test_captured_training_step(dev, dtype, b, d, L):
    """Forward and backward of both operators in one graph, replayed with eager work and other inputs between: every
    replay has the bits of an eager step."""
    import torch
    import selective_state_space_28_amd as ssm
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    gen = torch.Generator(device=dev)
    gen.manual_seed(7)
    rnd = lambda *s: torch.randn(s, generator=gen, device=dev)  # noqa: E731
    t = [rnd(b, d, L).to(dt) for _ in range(5)]
    x, r, i, z, dy = t
    A, w = -torch.rand(d, generator=gen, device=dev) - 0.1, 1 + 0.1 * rnd(d)
    starts = (torch.rand((b, L), generator=gen, device=dev) < 0.01)

    def step():
        y, last, ck = ssm.ssm_gated_scan_fwd(x, r, A, None, i, None, z, starts=starts, return_last_state=True,
                                             return_ckpt=True)
        n, m, s = ssm.ssm_layer_norm_fwd(y, w, axis=1, return_stats=True)
        g = ssm.ssm_layer_norm_bwd(y, w, m, s, dy, axis=1)
        h = ssm.ssm_gated_scan_bwd(x, r, A, None, i, None, z, starts=starts, ckpt=ck, dy=g["dx"])
        k, m, s = ssm.ssm_layer_norm_fwd(x.view(b * d, L), torch.ones(L, device=dev), return_stats=True)
        return [y, last, n, g["dx"], g["dweight"], g["dbias"], k] + [h[q] for q in sorted(h)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        for v in t:
            v.copy_(rnd(b, d, L).to(dt))
        graph.replay()
        torch.cuda.synchronize()
        for n, (u, v) in enumerate(zip(out, step())):
            assert torch.equal(u, v), (k, n)
        rnd(64, 64) @ rnd(64, 64)
        torch.cuda.synchronize()


def test_on_another_stream(dev):
    """Calls go to the current stream: inputs made there, results used there, without a wait on the default stream."""
    import torch
    import selective_state_space_28_amd as ssm
    side = torch.cuda.Stream()
    big = torch.randn(4096, 4096, device=dev)
    x0 = torch.randn(4, 200, 700, device=dev)
    A, w = -torch.rand(200, device=dev) - 0.1, torch.ones(200, device=dev)
    want = ssm.ssm_layer_norm_fwd(ssm.ssm_gated_scan_fwd(x0 * 2, x0 * 2, A), w, axis=1)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            big = big @ big * 1e-3
        x = x0 * 2
        got = ssm.ssm_layer_norm_fwd(ssm.ssm_gated_scan_fwd(x, x, A), w, axis=1).clone()
    side.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dim", [640, 650, 1300, 1700, 2570, 3000, 5000, 6500, 9001])
def test_many_channels_step_contiguous(dev, dtype, dim, residual):
    """Enough tiles for whole lines, and channels that fill the registers, then LDS, and then are read again; past the
    parameters that LDS holds (5120 backward, 8192 forward).  Against float64 on the GPU; the tolerance is that of the
    other norm tests: 128 half steps of float32 of the largest value, and the rounding of bf16."""
    import torch
    import selective_state_space_28_amd as ssm
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    L = 71 if dtype == "bf16" else 41   # two tiles to a row, the second ragged
    gen = torch.Generator(device=dev)
    gen.manual_seed(dim)
    rnd = lambda *s: torch.randn(s, generator=gen, device=dev)  # noqa: E731
    b = 130
    x, res = (rnd(b, dim, L) + 0.3).to(dt), rnd(b, dim, L).to(dt) if residual else None
    w, bias, dy = 1 + 0.3 * rnd(dim), 0.3 * rnd(dim), rnd(b, dim, L).to(dt)
    ds = rnd(b, dim, L).to(dt) if residual else None
    out = ssm.ssm_layer_norm_fwd(x, w, bias, res, axis=1, return_stats=True)
    s = x if res is None else (x.float() + res.float()).to(dt)
    if residual:
        assert torch.equal(out[1], s)
    s64, w64 = s.double(), w.double()[:, None]
    mean, var = s64.mean(1, keepdim=True), s64.var(1, unbiased=False, keepdim=True)
    rstd = (var + 1e-5).rsqrt()
    half, slack = (2.0 ** -8 if dtype == "bf16" else ref.EPS32), 129 * ref.EPS32

    def close(got, want, what, size=None, step=half):
        bound = step * want.abs() + slack * (want.abs().max() if size is None else size)
        assert bool(((got.double() - want).abs() <= bound).all()), what

    xh = (s64 - mean) * rstd
    close(out[0], xh * w64 + bias.double()[:, None], "y")
    close(out[-2], mean[:, 0], "mean", 1.0, ref.EPS32)
    close(out[-1], rstd[:, 0], "rstd", None, ref.EPS32)
    g = ssm.ssm_layer_norm_bwd(s, w, out[-2], out[-1], dy, ds, axis=1)
    xh = (s64 - out[-2].double()[:, None]) * out[-1].double()[:, None]
    d64 = dy.double()
    close(g["dweight"], (d64 * xh).sum((0, 2)), "dweight", (d64 * xh).abs().sum((0, 2)).max(), ref.EPS32)
    close(g["dbias"], d64.sum((0, 2)), "dbias", d64.abs().sum((0, 2)).max(), ref.EPS32)
    dn = d64 * w64
    dx = out[-1].double()[:, None] * (dn - dn.mean(1, keepdim=True) - xh * (dn * xh).mean(1, keepdim=True))
    close(g["dx"], dx if ds is None else dx + ds.double(), "dx")
