"""GPU tests of the gated recurrence (include/ssm_gated.h) against its formula
in 64 bits (tests/layers_ref.py).

Tolerance.  A gate's pre-activation of up to 6 in size goes through one
rounding, a product, exp2 and a reciprocal: under 16 half steps of float32
(2^-24) relative; the decay and the input weight inherit that and a few of
their own, under 32 in all.  An error of a decay stays in the state for
memory = 1 / (1 - largest decay) steps, so the state is within
32 * 2^-24 * memory of its largest value.  A gradient multiplies two such
quantities (state and adjoint) and a gate's derivative: three times as much.  A
sum's error is its terms' errors added.  bfloat16 outputs add their rounding,
2^-8 of the value."""
import numpy as np
import pytest

import synth
from tests import layers_ref as ref
from tests.helpers import to_torch

pytestmark = pytest.mark.gpu

TOK = ("x", "r", "i", "z")
PER = ("A", "r_bias", "i_bias", "h0")
GRADS = ("dx", "dr", "dA", "dr_bias", "di", "di_bias", "dz", "dh0")


@pytest.fixture(scope="module")
def dev():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import selective_state_space_28_amd as ssm
    ssm.load()
    return torch.device("cuda:0")


def case(dtype, b, d, L, seed, *, i=True, z=True, packed=False, h0=True, bias=True):
    """float32 or bf16-rounded inputs as float64 arrays (exact)."""
    rng = np.random.default_rng([seed, b, d, L])

    def tok():
        v = np.clip(rng.standard_normal((b, d, L)), -4, 4).astype(np.float32)
        return synth.widen(synth.bf16_bits(v), "bf16") if dtype == "bf16" else v.astype(np.float64)

    f32 = lambda v: v.astype(np.float32).astype(np.float64)  # noqa: E731
    p = dict(x=tok(), r=tok(), A=f32(-rng.uniform(0.2, 2.0, d)),
             r_bias=f32(rng.standard_normal(d) * 0.3) if bias else None, i=tok() if i else None,
             i_bias=f32(rng.standard_normal(d) * 0.3) if i and bias else None, z=tok() if z else None, starts=None,
             h0=f32(rng.standard_normal((b, d))) if h0 else None)
    if packed:
        p["starts"] = (rng.random((b, L)) < min(0.5, 4.0 / L)).astype(np.uint8)
    p["dy"], p["dl"], p["dtype"] = tok(), f32(rng.standard_normal((b, d))), dtype
    return p


def put(p, dev, off=0):
    """The inputs on the GPU; off: each starts that many elements into its buffer."""
    import torch

    def place(v, dtype):
        if v is None:
            return None
        t = to_torch(v.astype(np.float32), "f32", dev).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
        flat = torch.empty(t.numel() + off, dtype=t.dtype, device=dev)
        w = flat[off:].view(t.shape)
        w.copy_(t)
        return w

    t = {k: place(p[k], p["dtype"]) for k in TOK + ("dy",)}
    t.update({k: place(p[k], "f32") for k in PER + ("dl",)})
    t["starts"] = None if p["starts"] is None else torch.from_numpy(p["starts"]).to(dev)
    return t


def args(t):
    return t["x"], t["r"], t["A"], t["r_bias"], t["i"], t["i_bias"], t["z"]


def np64(t):
    return None if t is None else t.float().cpu().numpy().astype(np.float64)


def run_fwd(t, gate, weight, **kw):
    import selective_state_space_28_amd as ssm
    return ssm.ssm_gated_scan_fwd(*args(t), gate=gate, weight=weight, starts=t["starts"], h0=t["h0"],
                                  return_last_state=True, return_ckpt=True, **kw)


def run_bwd(t, ckpt, gate, weight, **kw):
    import selective_state_space_28_amd as ssm
    return ssm.ssm_gated_scan_bwd(*args(t), gate=gate, weight=weight, starts=t["starts"], ckpt=ckpt, dy=t["dy"],
                                  dlast_state=t["dl"], **kw)


def check(p, dev, gate="sigmoid", weight="unit", off=0):
    t = put(p, dev, off)
    dt = p["dtype"]
    slack = 32 * ref.EPS32 * ref.memory(p, gate)
    y, last, ckpt = run_fwd(t, gate, weight)
    yr, lr, states = ref.gated_fwd(p, gate, weight)
    L = p["x"].shape[2]
    ref.close(np64(y), yr, dt, slack, "y")
    ref.close(np64(last), lr, "f32", slack, "last_state")
    ref.close(np64(ckpt), np.moveaxis(states[:, :, 0:L:512], 2, 1), "f32", slack, "ckpt")
    g = run_bwd(t, ckpt, gate, weight)
    gr = ref.gated_bwd(p, p["dy"], p["dl"], gate, weight)
    for k in GRADS:
        if gr[k] is None:
            assert g[k] is None, k
            continue
        ref.close(np64(g[k]), gr[k], dt if k in ("dx", "dr", "di", "dz") else "f32", 3 * slack, k,
                  gr["size"].get(k))
    return y, last, ckpt, g


@pytest.mark.parametrize("i,z", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("weight", ["unit", "convex"])
@pytest.mark.parametrize("gate", ["sigmoid", "softplus"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rules_and_gates(dev, dtype, gate, weight, i, z):
    check(case(dtype, 2, 7, 77, 1, i=i, z=z), dev, gate, weight)
    check(case(dtype, 2, 3, 530, 2, i=i, z=z, packed=True, h0=False, bias=False), dev, gate, weight)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L", [1, 2, 7, 8, 9, 63, 64, 65, 504, 511, 512, 513, 520, 1023, 1025, 2048, 4097, 8195, 16385])
def test_lengths(dev, dtype, L, packed):
    check(case(dtype, 2, 3, L, 3, packed=packed), dev)


@pytest.mark.parametrize("b,d", [(1, 1), (1, 5), (3, 4), (2, 65), (5, 129), (1, 1030)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_row_counts(dev, dtype, b, d):
    check(case(dtype, b, d, 100, 4, packed=True), dev, "softplus", "convex")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_unaligned_tensors_give_the_same_bits(dev, dtype):
    import torch
    p = case(dtype, 2, 5, 1031, 5, packed=True)
    a = check(p, dev)
    b = check(p, dev, off=1)
    for u, v in zip(a[:3], b[:3]):
        assert torch.equal(u, v)
    for k in GRADS:
        assert torch.equal(a[3][k], b[3][k]), k


def test_two_runs_give_the_same_bits(dev):
    import torch
    t = put(case("bf16", 3, 200, 1500, 6, packed=True), dev)
    a, b = run_fwd(t, "sigmoid", "unit"), run_fwd(t, "sigmoid", "unit")
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    g, h = run_bwd(t, a[2], "sigmoid", "unit"), run_bwd(t, a[2], "sigmoid", "unit")
    assert all(torch.equal(g[k], h[k]) for k in GRADS)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_every_step_a_start(dev, dtype):
    """No state is carried at all: h = w u, and the decay gets no gradient from the state."""
    p = case(dtype, 2, 5, 1100, 7)
    p["starts"] = np.full((2, 1100), 3, np.uint8)
    _, _, _, g = check(p, dev)
    assert not g["dh0"].abs().max().item()


def test_packed_rows_are_their_sequences(dev):
    """Each packed sequence gives what it gives alone, to rounding: starts at and beside the edges of the kernel's
    lanes and blocks, a sequence of one step, and the last step its own."""
    p = case("f32", 1, 6, 1600, 8, packed=True, h0=False)
    cuts = [0, 1, 8, 15, 511, 512, 520, 1024, 1025, 1599]
    p["starts"] = np.zeros((1, 1600), np.uint8)
    p["starts"][0, cuts] = 1
    y = np64(check(p, dev)[0])
    for s, e in zip(cuts, cuts[1:] + [1600]):
        q = {k: v[:, :, s:e] if k in TOK and v is not None else v for k, v in p.items()}
        q["starts"] = None
        ref.close(y[:, :, s:e], ref.gated_fwd(q)[0], "f32", 32 * ref.EPS32 * ref.memory(p, "sigmoid"), f"{s}..{e}")


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("b,d,L,cuts,at", [(2, 5, 1300, (0, 600, 640, 1100), 3), (2, 5, 1300, (0, 600, 640, 1100), 700),
                                           (2, 5, 17000, (0, 8000, 16999), 7000), (2, 4200, 600, (0, 100, 520), 130),
                                           (2, 5, 100, (0, 50, 64, 90), 70), (3, 7, 33, (0,), 20), (2, 9, 6, (), 2)])
def test_nothing_crosses_a_start(dev, bad, b, d, L, cuts, at):
    """A non-finite input stays in its channel and its sequence, forward and backward: with a row to 16 waves, 4 and
    one, and rows that share a wave."""
    p = case("f32", b, d, L, 9, h0=False)
    p["starts"] = np.zeros((b, L), np.uint8)
    p["starts"][:, list(cuts)] = 1
    clean = check(p, dev)
    p["x"][1, 2, at] = bad
    t = put(p, dev)
    y, last, ckpt = run_fwd(t, "sigmoid", "unit")
    end = min([c for c in cuts if c > at] + [L])
    first = max([c for c in cuts if c <= at] + [0])
    got = np64(y)
    assert not np.isfinite(got[1, 2, at:end]).any()
    got[1, 2, at:end] = np64(clean[0])[1, 2, at:end]
    assert np.array_equal(got, np64(clean[0]))
    got, want = np64(last), np64(clean[1])
    if end == L:
        got[1, 2] = want[1, 2]
    assert np.array_equal(got, want)
    g = run_bwd(t, ckpt, "sigmoid", "unit")
    for k in ("dx", "dr", "di", "dz"):
        v, c = np64(g[k]), np64(clean[3][k])
        v[1, 2, first:end], c[1, 2, first:end] = 0, 0
        assert np.array_equal(v, c), k
    for k in ("dA", "dr_bias", "di_bias"):
        v, c = np64(g[k]), np64(clean[3][k])
        v[2], c[2] = 0, 0
        assert np.array_equal(v, c), k


@pytest.mark.parametrize("bad", [np.inf, np.nan])
def test_non_finite_values_run_on(dev, bad):
    """Without a start a non-finite x or r makes its channel's outputs non-finite from there on, and no other's."""
    for key in ("x", "r"):
        p = case("f32", 1, 4, 1100, 10, z=False)
        clean = np64(run_fwd(put(p, dev), "sigmoid", "unit")[0])
        if key == "r" and bad == np.inf:
            continue  # an open gate is finite
        p[key][0, 1, 530] = bad
        y = np64(run_fwd(put(p, dev), "sigmoid", "unit")[0])
        assert not np.isfinite(y[0, 1, 530:]).any(), key
        y[0, 1, 530:] = clean[0, 1, 530:]
        assert np.array_equal(y, clean), key


def test_infinite_state_outlives_underflowing_decays(dev):
    """Decays that underflow over a lane's run, or in one step, do not turn an infinite state into NaN."""
    p = case("f32", 1, 3, 1100, 11, z=False, i=False)
    p["A"] = np.array([-60.0, -1e4, -1.0])
    p["x"][0, :, 5] = np.inf
    y = np64(run_fwd(put(p, dev), "softplus", "convex")[0])
    assert np.all(np.isposinf(y[0, :, 5:])) and np.isfinite(y[0, :, :5]).all()


@pytest.mark.parametrize("gate", ["sigmoid", "softplus"])
@pytest.mark.parametrize("weight", ["unit", "convex"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_padding_with_closed_gates(dev, dtype, gate, weight):
    """Steps with r = -inf are the identity: last_state, the sums and the gradients before them are those of the
    shorter sequence."""
    import torch
    L, cut = 1300, 777
    p = case(dtype, 2, 5, L, 12)
    p["r"][1, :, cut:] = -np.inf
    p["dy"][1, :, cut:] = 0
    t = put(p, dev)
    y, last, ckpt = run_fwd(t, gate, weight)
    g = run_bwd(t, ckpt, gate, weight)
    q = {k: (v[1:2, :, :cut] if k in TOK + ("dy",) else v) for k, v in p.items()}
    q["h0"], q["dl"] = p["h0"][1:2], p["dl"][1:2]
    s = put(q, dev)
    y1, last1, ckpt1 = run_fwd(s, gate, weight)
    g1 = run_bwd(s, ckpt1, gate, weight)
    assert torch.equal(last[1], last1[0]) and torch.equal(y[1, :, :cut], y1[0])
    for k in ("dx", "dr", "di", "dz"):
        assert torch.equal(g[k][1, :, :cut], g1[k][0]), k
        assert torch.isfinite(g[k]).all(), k
    assert torch.equal(g["dh0"][1], g1["dh0"][0])
    for k in ("dA", "dr_bias", "di_bias"):
        assert torch.isfinite(g[k]).all(), k


def test_extreme_gates(dev):
    """Gates far open and far closed, decays from 1 - 1e-7 to underflow: finite and as the formula."""
    p = case("f32", 1, 8, 64, 13, z=False)
    p["r"] = np.float32(np.linspace(-120, 120, 8 * 64).reshape(1, 8, 64)).astype(np.float64)
    p["i"] = np.float32(np.linspace(100, -100, 8 * 64).reshape(1, 8, 64)).astype(np.float64)
    p["A"] = np.float32(-np.logspace(-6, 2, 8)).astype(np.float64)
    for gate in ("sigmoid", "softplus"):
        for weight in ("unit", "convex"):
            t = put(p, dev)
            y, last, ckpt = run_fwd(t, gate, weight)
            # pre-activations of 120 carry 20 times the rounding of those of 6
            slack = 20 * 32 * ref.EPS32 * 64
            yr, lr, _ = ref.gated_fwd(p, gate, weight)
            ref.close(np64(y), yr, "f32", slack, "y")
            g = run_bwd(t, ckpt, gate, weight)
            gr = ref.gated_bwd(p, p["dy"], p["dl"], gate, weight)
            for k in ("dx", "dr", "di", "dh0"):
                ref.close(np64(g[k]), gr[k], "f32", 3 * slack, f"{gate} {weight} {k}")


def test_empty_problems(dev):
    import torch
    import selective_state_space_28_amd as ssm
    p = case("f32", 2, 5, 0, 14)
    t = put(p, dev)
    y, last, ckpt = run_fwd(t, "sigmoid", "unit")
    assert y.numel() == 0 and ckpt.shape == (2, 0, 5) and torch.equal(last, t["h0"])
    g = run_bwd(t, ckpt, "sigmoid", "unit")
    assert torch.equal(g["dh0"], t["dl"])
    assert not any(g[k].abs().max().item() for k in ("dA", "dr_bias", "di_bias"))
    t = put(case("f32", 0, 5, 9, 14), dev)
    y, last, ckpt = run_fwd(t, "sigmoid", "unit")
    g = run_bwd(t, ckpt, "sigmoid", "unit")
    assert y.shape == (0, 5, 9) and not g["dA"].abs().max().item()
    assert ssm.ssm_gated_state_update(last, t["x"][:, :, 0].contiguous(), t["r"][:, :, 0].contiguous(),
                                      t["A"]).shape == (0, 5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nothing_is_written_beside_the_outputs(dev, dtype):
    """y of a slice in the middle of a larger buffer, at an odd element: what stands before and behind stays."""
    import torch
    p = case(dtype, 2, 3, 1027, 15, packed=True)
    t = put(p, dev)
    n = t["x"].numel()
    buf = torch.full((n + 39,), 7.0, dtype=t["x"].dtype, device=dev)
    y = run_fwd(t, "sigmoid", "unit", out=buf[19:19 + n].view(t["x"].shape))[0]
    torch.cuda.synchronize()
    assert torch.equal(y, run_fwd(t, "sigmoid", "unit")[0])
    assert bool((buf[:19] == 7).all()) and bool((buf[19 + n:] == 7).all())


def test_offsets_past_32_bits(dev):
    """More than 2^31 elements: the last rows are those of a call on them alone, forward and backward."""
    import torch
    import selective_state_space_28_amd as ssm
    d, L = 33000, 65537
    gen = torch.Generator(device=dev)
    gen.manual_seed(5)
    x = torch.empty((1, d, L), dtype=torch.bfloat16, device=dev)
    r = torch.empty_like(x)
    for k in range(0, d, 3000):
        x[:, k:k + 3000].normal_(generator=gen)
        r[:, k:k + 3000].normal_(generator=gen)
    A = -torch.rand(d, generator=gen, device=dev) - 0.2
    y, last, ckpt = ssm.ssm_gated_scan_fwd(x, r, A, return_last_state=True, return_ckpt=True)
    g = ssm.ssm_gated_scan_bwd(x, r, A, ckpt=ckpt, dy=x)
    xs, rs, As = x[:, -3:].contiguous(), r[:, -3:].contiguous(), A[-3:].contiguous()
    ys, lasts, cks = ssm.ssm_gated_scan_fwd(xs, rs, As, return_last_state=True, return_ckpt=True)
    gs = ssm.ssm_gated_scan_bwd(xs, rs, As, ckpt=cks, dy=xs)
    # another number of rows may split a row over more waves: the same to rounding of bf16
    for u, v in ((y[:, -3:], ys), (g["dx"][:, -3:], gs["dx"]), (g["dr"][:, -3:], gs["dr"])):
        assert (u.float() - v.float()).abs().max().item() <= 2 ** -7 * v.float().abs().max().item()
    assert torch.allclose(last[:, -3:], lasts, rtol=1e-4, atol=1e-4)


@pytest.mark.parametrize("d,L", [(2**27 + 5, 129), (2**26 + 5, 257)])
def test_more_threads_than_a_grid_dimension_has(dev, d, L):
    """2^32 threads and more, of rows that share a wave and of a wave each: rows in the middle and at the end are those
    of a call on them alone, forward and backward."""
    import torch
    import selective_state_space_28_amd as ssm
    if torch.cuda.mem_get_info()[0] < 130 * 2**30:
        pytest.skip("needs 130 GiB of GPU memory")
    gen = torch.Generator(device=dev)
    gen.manual_seed(6)
    x = torch.empty((1, d, L), dtype=torch.bfloat16, device=dev)
    for k in range(0, d, 2**24):
        x[:, k:k + 2**24].normal_(generator=gen)
    A = -torch.rand(d, generator=gen, device=dev) - 0.2
    windows = [slice(at, at + 9) for at in (0, d // 2, d - 9)]
    alone = [(x[:, s].contiguous(), A[s].contiguous()) for s in windows]
    y, last, ckpt = ssm.ssm_gated_scan_fwd(x, x, A, return_last_state=True, return_ckpt=True,
                                           out=torch.full_like(x, float("nan")))
    assert not bool(y[0, :, -1].isnan().any()) and not bool(last.isnan().any())
    small = [ssm.ssm_gated_scan_fwd(xs, xs, As, return_last_state=True, return_ckpt=True) for xs, As in alone]
    for s, (ys, lasts, _) in zip(windows, small):
        assert torch.equal(y[:, s], ys) and torch.equal(last[:, s], lasts)
    del y, last
    g = ssm.ssm_gated_scan_bwd(x, x, A, ckpt=ckpt, dy=x)
    for s, (xs, As), (_, _, cks) in zip(windows, alone, small):
        gs = ssm.ssm_gated_scan_bwd(xs, xs, As, ckpt=cks, dy=xs)
        for name in ("dx", "dr"):
            assert torch.equal(g[name][:, s], gs[name]), name
        for name in ("dA", "dr_bias"):
            assert torch.equal(g[name][s], gs[name]), name
        assert torch.equal(g["dh0"][:, s], gs["dh0"])


# ---- one token ----------------------------------------------------------------------

@pytest.mark.parametrize("gate,weight", [("sigmoid", "unit"), ("softplus", "convex"), ("softplus", "unit")])
@pytest.mark.parametrize("i,z", [(True, True), (False, False)])
@pytest.mark.parametrize("b,d", [(1, 1), (3, 5), (2, 513), (7, 1031), (300, 64), (64, 4096), (50, 5243), (70000, 4)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_step(dev, dtype, b, d, i, z, gate, weight):
    import torch
    import selective_state_space_28_amd as ssm
    p = case(dtype, b, d, 1, 20, i=i, z=z)
    p["starts"] = (np.arange(b) % 3 == 1).astype(np.uint8)[:, None]
    t = put(p, dev)
    tok = [v[:, :, 0].contiguous() if v is not None and v.dim() == 3 else v for v in args(t)]
    starts = t["starts"][:, 0].contiguous()
    yr, lr, _ = ref.gated_fwd(p, gate, weight)
    state = t["h0"].clone()
    after = torch.empty_like(state)
    y = ssm.ssm_gated_state_update(state, *tok, gate=gate, weight=weight, starts=starts, state_out=after)
    assert torch.equal(state, t["h0"]), "the state is kept"
    ref.close(np64(y), yr[:, :, 0], dtype, 64 * ref.EPS32, "y")
    ref.close(np64(after), lr, "f32", 64 * ref.EPS32, "state")
    y2 = ssm.ssm_gated_state_update(state, *tok, gate=gate, weight=weight, starts=starts.bool())
    assert torch.equal(y, y2) and torch.equal(state, after), "in place"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_step_unaligned_and_infinite_state(dev, dtype):
    import torch
    import selective_state_space_28_amd as ssm
    p = case(dtype, 2, 515, 1, 21)
    p["h0"][0, 3] = np.inf
    out = []
    for off in (0, 1):
        t = put(p, dev, off)
        flat = lambda v: v.view(2, 515) if v is not None and v.dim() == 3 else v  # noqa: E731
        st = t["h0"]
        y = ssm.ssm_gated_state_update(st, *[flat(v) for v in args(t)], starts=torch.tensor([0, 1], device=dev).bool())
        out.append((y.clone(), st.clone()))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    assert torch.isinf(out[0][1][0, 3]) and torch.isfinite(out[0][1][1]).all()


def test_steps_continue_a_scan(dev):
    """A prompt through the scan, then tokens one at a time: what the scan of the whole gives."""
    import torch
    import selective_state_space_28_amd as ssm
    p = case("f32", 2, 70, 530, 22)
    t = put(p, dev)
    whole, end, _ = run_fwd(t, "sigmoid", "unit")
    cut = lambda v, s, e: v[:, :, s:e].contiguous() if v is not None and v.dim() == 3 else v  # noqa: E731
    y, st = ssm.ssm_gated_scan_fwd(*[cut(v, 0, 520) for v in args(t)], h0=t["h0"], return_last_state=True)
    for k in range(520, 530):
        tok = [v[:, :, k].contiguous() if v is not None and v.dim() == 3 else v for v in args(t)]
        yk = ssm.ssm_gated_state_update(st, *tok)
        ref.close(np64(yk), np64(whole[:, :, k]), "f32", 64 * ref.EPS32 * ref.memory(p, "sigmoid"), f"token {k}")
    assert torch.allclose(st, end, rtol=1e-4, atol=1e-5)


# ---- refusals -----------------------------------------------------------------------

def test_refusals(dev):
    import torch
    import selective_state_space_28_amd as ssm
    t = put(case("f32", 2, 5, 30, 30), dev)
    x, r, A = t["x"], t["r"], t["A"]
    with pytest.raises(TypeError):
        ssm.ssm_gated_scan_fwd(x.half(), r.half(), A)
    with pytest.raises(TypeError):
        ssm.ssm_gated_scan_fwd(x, r.bfloat16(), A)
    with pytest.raises(ValueError):
        ssm.ssm_gated_scan_fwd(x.transpose(1, 2), r, A)
    with pytest.raises(ValueError):
        ssm.ssm_gated_scan_fwd(x, r, A[:3])
    with pytest.raises(ValueError):
        ssm.ssm_gated_scan_fwd(x, r, A.cpu())
    with pytest.raises(ValueError):
        ssm.ssm_gated_scan_fwd(x[0], r[0], A)
    with pytest.raises(ssm.SsmError, match="ALIAS"):
        ssm.ssm_gated_scan_fwd(x, r, A, out=x)
    y, ckpt = ssm.ssm_gated_scan_fwd(x, r, A, return_ckpt=True)
    with pytest.raises(ValueError):
        ssm.ssm_gated_scan_bwd(x, r, A, ckpt=ckpt[:, :0], dy=y)
    with pytest.raises(ValueError):
        ssm.ssm_gated_scan_bwd(x, r, A, ckpt=ckpt, dy=y[:, :, :20])
    state = torch.zeros(2, 5, device=dev)
    tok = x[:, :, 0].contiguous()
    with pytest.raises(ssm.SsmError, match="ALIAS"):
        ssm.ssm_gated_state_update(state, tok, tok, A, out=tok)
    with pytest.raises(ValueError):
        ssm.ssm_gated_state_update(state, tok, tok, A, starts=torch.zeros(3, dtype=torch.uint8, device=dev))
    with pytest.raises(TypeError):
        ssm.ssm_gated_state_update(state.bfloat16(), tok, tok, A)
