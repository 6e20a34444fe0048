"""The C ABI of the gated recurrence and the layer norm without a GPU: every
declared function is exported, and bad arguments are refused before any HIP
call; the Python wrappers' own checks; and the 64-bit reference of their tests,
pinned by the selective scan's oracle and by differences."""
import ctypes

import numpy as np
import pytest

import oracle
import selective_state_space_28_amd as ssm
from selective_state_space_28_amd._lib import header_functions, load
from tests import layers_ref as ref

OK, NULL, SHAPE, DTYPE, ALIGN, WS, ALIAS, FLAGS = 0, -1, -2, -3, -4, -5, -7, -8
R = 0x1000000


def at(k):
    """Fake device address of the k-th distinct buffer of a call, never dereferenced."""
    return 0x40000000 + k * R


def test_exports_every_declared_symbol():
    gated, norm = header_functions("ssm_gated.h"), header_functions("ssm_norm.h")
    assert set(gated) == {"ssm_gated_scan_ckpt_bytes", "ssm_gated_scan_fwd", "ssm_gated_scan_bwd",
                          "ssm_gated_scan_bwd_workspace_bytes", "ssm_gated_state_update"}
    assert set(norm) == {"ssm_layer_norm_fwd", "ssm_layer_norm_bwd", "ssm_layer_norm_bwd_workspace_bytes"}
    lib = ctypes.CDLL(load()._name)
    for n in gated + norm:
        assert hasattr(lib, n), n


CK = 2 * 4 * 64 * 4  # kept states of (batch 2, dim 64, L 2048)
N = 2 * 64 * 2048 * 2  # bytes of x


def _fwd(**kw):
    a = dict(x=at(0), r=at(1), A=at(2), rb=None, i=None, ib=None, z=None, fl=0, st=None, h0=None, y=at(3),
             last=None, ck=None, ckb=0, batch=2, dim=64, L=2048, dtype=1)
    a.update(kw)
    return load().ssm_gated_scan_fwd(a["x"], a["r"], a["A"], a["rb"], a["i"], a["ib"], a["z"], a["fl"], a["st"],
                                     a["h0"], a["y"], a["last"], a["ck"], a["ckb"], a["batch"], a["dim"],
                                     a["L"], a["dtype"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), DTYPE), (dict(dtype=-1), DTYPE), (dict(fl=4), FLAGS), (dict(fl=-1), FLAGS),
    (dict(batch=-1), SHAPE), (dict(dim=-2), SHAPE), (dict(L=-1), SHAPE), (dict(L=(1 << 31) - 4096), SHAPE),
    (dict(batch=1 << 16, dim=1 << 16), SHAPE),
    (dict(x=None), NULL), (dict(r=None), NULL), (dict(A=None), NULL), (dict(y=None), NULL),
    (dict(x=at(0) + 1), ALIGN), (dict(dtype=0, r=at(1) + 2), ALIGN), (dict(A=at(2) + 2), ALIGN),
    (dict(rb=at(4) + 1), ALIGN), (dict(h0=at(4) + 2), ALIGN), (dict(last=at(4) + 1), ALIGN),
    (dict(ck=at(4) + 1, ckb=CK), ALIGN), (dict(ck=at(4), ckb=CK - 1), WS),
    (dict(y=at(0)), ALIAS), (dict(y=at(1) + N - 2), ALIAS), (dict(i=at(3) + 64), ALIAS), (dict(z=at(3)), ALIAS),
    (dict(last=at(3) + 4), ALIAS), (dict(last=at(2)), ALIAS), (dict(h0=at(4), last=at(4) + 8), ALIAS),
    (dict(ck=at(4), ckb=CK, last=at(4) + CK - 4), ALIAS), (dict(st=at(3) + 128), ALIAS),
    (dict(i=at(5), ib=at(3)), ALIAS),
    (dict(batch=0), OK), (dict(dim=0, x=None), OK), (dict(L=0, x=None, y=None), OK),
])
def test_gated_fwd_validation(kw, code):
    assert _fwd(**kw) == code


def _bwd(**kw):
    a = dict(x=at(0), r=at(1), A=at(2), rb=None, i=None, ib=None, z=None, fl=0, st=None, ck=at(3), ckb=CK,
             dy=at(4), dl=None, dx=at(5), dr=at(6), dA=at(7), drb=None, di=None, dib=None, dz=None, dh0=None,
             batch=2, dim=64, L=2048, dtype=1, ws=at(8), wsb=1 << 16)
    a.update(kw)
    return load().ssm_gated_scan_bwd(a["x"], a["r"], a["A"], a["rb"], a["i"], a["ib"], a["z"], a["fl"], a["st"],
                                     a["ck"], a["ckb"], a["dy"], a["dl"], a["dx"], a["dr"], a["dA"], a["drb"],
                                     a["di"], a["dib"], a["dz"], a["dh0"], a["batch"], a["dim"], a["L"],
                                     a["dtype"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), DTYPE), (dict(fl=8), FLAGS), (dict(dim=-1), SHAPE), (dict(L=1 << 40), SHAPE),
    (dict(ck=None), NULL), (dict(dy=None), NULL), (dict(dx=None), NULL), (dict(dr=None), NULL), (dict(dA=None), NULL),
    (dict(i=at(9)), NULL), (dict(z=at(9)), NULL), (dict(batch=0, dA=None), NULL),
    (dict(dx=at(5) + 1), ALIGN), (dict(dA=at(7) + 2), ALIGN), (dict(dl=at(9) + 1), ALIGN), (dict(ws=at(8) + 4), ALIGN),
    (dict(ckb=CK - 4), WS), (dict(ws=None), WS), (dict(wsb=3 * 2 * 64 * 4 - 1), WS),
    (dict(dx=at(4)), ALIAS), (dict(dr=at(5) + N - 2), ALIAS), (dict(dA=at(2)), ALIAS), (dict(dh0=at(3)), ALIAS),
    (dict(drb=at(7) + 4), ALIAS), (dict(ws=at(5)), ALIAS), (dict(i=at(9), di=at(9)), ALIAS),
    (dict(z=at(9), dz=at(0)), ALIAS), (dict(i=at(9), di=at(10), dib=at(7)), ALIAS),
    (dict(dim=0, dA=None), OK),
])
def test_gated_bwd_validation(kw, code):
    assert _bwd(**kw) == code


def _step(**kw):
    a = dict(s=at(0), x=at(1), r=at(2), A=at(3), rb=None, i=None, ib=None, z=None, fl=0, st=None, y=at(4), so=None,
             batch=4, dim=64, dtype=1)
    a.update(kw)
    return load().ssm_gated_state_update(a["s"], a["x"], a["r"], a["A"], a["rb"], a["i"], a["ib"], a["z"], a["fl"],
                                         a["st"], a["y"], a["so"], a["batch"], a["dim"], a["dtype"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=9), DTYPE), (dict(fl=4), FLAGS), (dict(batch=-1), SHAPE), (dict(dim=(1 << 31) - 1), SHAPE),
    (dict(s=None), NULL), (dict(x=None), NULL), (dict(r=None), NULL), (dict(A=None), NULL), (dict(y=None), NULL),
    (dict(s=at(0) + 2), ALIGN), (dict(y=at(4) + 1), ALIGN), (dict(so=at(5) + 2), ALIGN),
    (dict(y=at(1)), ALIAS), (dict(y=at(0) + 16), ALIAS), (dict(so=at(0) + 4), ALIAS), (dict(so=at(1)), ALIAS),
    (dict(so=at(4)), ALIAS), (dict(batch=0), OK), (dict(dim=0, s=None), OK),
])
def test_gated_step_validation(kw, code):
    assert _step(**kw) == code


def _nf(**kw):
    a = dict(x=at(0), res=None, w=at(1), b=None, eps=1e-5, y=at(2), so=None, m=None, rs=None, batch=4, dim=64, L=32,
             dtype=1)
    a.update(kw)
    return load().ssm_layer_norm_fwd(a["x"], a["res"], a["w"], a["b"], a["eps"], a["y"], a["so"], a["m"], a["rs"],
                                     a["batch"], a["dim"], a["L"], a["dtype"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), DTYPE), (dict(dim=0), SHAPE), (dict(dim=-1), SHAPE), (dict(batch=-1), SHAPE), (dict(L=-1), SHAPE),
    (dict(eps=-1e-6), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(eps=float("inf")), SHAPE),
    (dict(batch=(1 << 31) - 1), SHAPE), (dict(batch=1 << 29, L=7, dim=1), SHAPE), (dict(batch=4, L=1 << 30), SHAPE),
    (dict(x=None), NULL), (dict(w=None), NULL), (dict(y=None), NULL), (dict(res=at(3)), NULL), (dict(so=at(3)), NULL),
    (dict(x=at(0) + 1), ALIGN), (dict(w=at(1) + 2), ALIGN), (dict(m=at(4) + 2), ALIGN),
    (dict(y=at(0)), ALIAS), (dict(y=at(1)), ALIAS), (dict(res=at(3), so=at(3)), ALIAS), (dict(res=at(3), so=at(0)), ALIAS),
    (dict(m=at(4), rs=at(4) + 4), ALIAS), (dict(batch=0), OK), (dict(L=0, x=None), OK),
])
def test_norm_fwd_validation(kw, code):
    assert _nf(**kw) == code


def _nb(**kw):
    a = dict(s=at(0), w=at(1), m=at(2), rs=at(3), dy=at(4), ds=None, dx=at(5), dw=at(6), db=at(7), batch=4, dim=64,
             L=32, dtype=1, ws=at(8), wsb=1 << 20)
    a.update(kw)
    return load().ssm_layer_norm_bwd(a["s"], a["w"], a["m"], a["rs"], a["dy"], a["ds"], a["dx"], a["dw"], a["db"],
                                     a["batch"], a["dim"], a["L"], a["dtype"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), DTYPE), (dict(dim=0), SHAPE), (dict(L=-1), SHAPE),
    (dict(s=None), NULL), (dict(m=None), NULL), (dict(rs=None), NULL), (dict(dy=None), NULL), (dict(dx=None), NULL),
    (dict(dw=None), NULL), (dict(batch=0, dw=None), NULL),
    (dict(dy=at(4) + 1), ALIGN), (dict(dw=at(6) + 1), ALIGN), (dict(ws=at(8) + 8), ALIGN),
    (dict(ws=None), WS), (dict(wsb=16), WS),
    (dict(dx=at(0)), ALIAS), (dict(dx=at(4)), ALIAS), (dict(ds=at(5)), ALIAS), (dict(db=at(6) + 8), ALIAS),
    (dict(ws=at(5)), ALIAS), (dict(dw=at(1)), ALIAS),
])
def test_norm_bwd_validation(kw, code):
    assert _nb(**kw) == code


def test_queries():
    lib = load()
    assert lib.ssm_gated_scan_ckpt_bytes(2, 64, 2048) == CK
    assert lib.ssm_gated_scan_ckpt_bytes(3, 7, 513) == 3 * 2 * 7 * 4
    assert lib.ssm_gated_scan_ckpt_bytes(3, 7, 0) == 0
    assert lib.ssm_gated_scan_ckpt_bytes(-1, 7, 8) == 0
    assert lib.ssm_gated_scan_bwd_workspace_bytes(2, 64, 2048, 1) >= 3 * 2 * 64 * 4
    assert lib.ssm_gated_scan_bwd_workspace_bytes(2, 64, 2048, 5) == 0
    assert lib.ssm_gated_scan_bwd_workspace_bytes(0, 64, 2048, 1) == 0
    assert lib.ssm_layer_norm_bwd_workspace_bytes(4, 64, 32, 1) >= 2 * 64 * 4
    assert lib.ssm_layer_norm_bwd_workspace_bytes(4, 0, 32, 1) == 0
    assert lib.ssm_layer_norm_bwd_workspace_bytes(0, 64, 32, 1) == 0


def test_python_checks_without_gpu():
    import torch
    from selective_state_space_28_amd import layers
    assert layers._rule("sigmoid", "convex") == 0 and layers._rule("softplus", "unit") == 3
    with pytest.raises(ValueError, match="gate"):
        layers._rule("tanh", "unit")
    with pytest.raises(ValueError, match="weight"):
        layers._rule("sigmoid", "none")
    x = torch.zeros(2, 3, 4)
    with pytest.raises(ValueError, match="GPU"):
        ssm.ssm_gated_scan_fwd(x, x, torch.zeros(3))
    with pytest.raises(ValueError, match="GPU"):
        ssm.ssm_layer_norm_fwd(x, torch.zeros(4))
    assert layers._norm_sizes(x, -1) == (6, 4, 1, (2, 3))
    assert layers._norm_sizes(x, 1) == (2, 3, 4, (2, 4))
    assert layers._norm_sizes(x[0], 1) == (3, 4, 1, (3,))
    with pytest.raises(ValueError, match="axis"):
        layers._norm_sizes(x, 0)
    with pytest.raises(ValueError, match="axis"):
        layers._norm_sizes(x, 3)
    dev = x.device
    args = dict(x=x, r=x, A=torch.zeros(3), r_bias=None, i=None, i_bias=None, z=None, starts=None,
                shape=(2, 3, 4), dev=dev)
    layers._check_gates(**args)
    for bad, err in (({"r": x[:, :2]}, ValueError), ({"A": torch.zeros(4)}, ValueError), ({"z": x.double()}, TypeError),
                     ({"i_bias": torch.zeros(3)}, ValueError), ({"starts": torch.zeros(2, 4)}, TypeError),
                     ({"starts": torch.zeros(4, 2, dtype=torch.bool)}, ValueError),
                     ({"i": x.transpose(0, 1).contiguous().transpose(0, 1)}, ValueError)):
        with pytest.raises(err):
            layers._check_gates(**{**args, **bad})


# ---- the reference ------------------------------------------------------------------

def _problem(rng, b=2, d=3, L=7, full=True):
    p = dict(x=rng.standard_normal((b, d, L)), r=rng.standard_normal((b, d, L)), A=-rng.uniform(0.2, 2.0, d),
             r_bias=rng.standard_normal(d) * 0.3, i=None, i_bias=None, z=None, starts=None, h0=None)
    if full:
        p.update(i=rng.standard_normal((b, d, L)), i_bias=rng.standard_normal(d) * 0.3,
                 z=rng.standard_normal((b, d, L)), h0=rng.standard_normal((b, d)),
                 starts=(rng.random((b, L)) < 0.3).astype(np.uint8))
    return p


def test_reference_is_the_selective_scan_of_one_state():
    """softplus gate, convex weight: the zero-order-hold selective scan with one state, B = 1 and C = 1, times -A
    (its input weight is (a - 1)/A)."""
    rng = np.random.default_rng(1)
    p = _problem(rng, L=40, full=False)
    p["h0"] = rng.standard_normal((2, 3))
    y, last, _ = ref.gated_fwd(p, "softplus", "convex")
    one = np.ones((2, 1, 40))
    gain = -p["A"][None, :, None]
    yo, lo = oracle.scan_fwd(p["x"] * gain, p["r"], p["A"][:, None], one, one, None, None, p["r_bias"], True,
                             p["h0"][..., None], nthreads=1, bbar="zoh")
    assert np.allclose(y, yo, rtol=1e-12, atol=1e-13)
    assert np.allclose(last, lo[..., 0], rtol=1e-12, atol=1e-13)


@pytest.mark.parametrize("gate", ["sigmoid", "softplus"])
@pytest.mark.parametrize("weight", ["unit", "convex"])
@pytest.mark.parametrize("full", [True, False])
def test_reference_gradients_by_differences(gate, weight, full):
    """Central differences of the 64-bit forward: the step 1e-5 leaves about 1e-10 of truncation and 1e-11 of rounding
    on values near 1, so 1e-7 is far above both."""
    rng = np.random.default_rng(2)
    p = _problem(rng, full=full)
    dy, dl = rng.standard_normal(p["x"].shape), rng.standard_normal(p["x"].shape[:2])
    if p["h0"] is None:
        p["h0"] = np.zeros((2, 3))

    def loss(q):
        y, last, _ = ref.gated_fwd(q, gate, weight)
        return (y * dy).sum() + (last * dl).sum()

    g = ref.gated_bwd(p, dy, dl, gate, weight)
    for k in ("x", "r", "A", "r_bias", "i", "i_bias", "z", "h0"):
        if p[k] is None:
            continue
        num = np.empty_like(p[k])
        for idx in np.ndindex(p[k].shape):
            up, down = dict(p), dict(p)
            up[k], down[k] = p[k].copy(), p[k].copy()
            up[k][idx] += 1e-5
            down[k][idx] -= 1e-5
            num[idx] = (loss(up) - loss(down)) / 2e-5
        assert np.max(np.abs(num - g["d" + k])) < 1e-7, k


@pytest.mark.parametrize("axis", [-1, 1])
def test_norm_reference_gradients_by_differences(axis):
    rng = np.random.default_rng(3)
    x, dy = rng.standard_normal((2, 4, 5)), rng.standard_normal((2, 4, 5))
    n = x.shape[axis]
    w, b = rng.standard_normal(n), rng.standard_normal(n)

    def loss(x, w, b):
        return (ref.norm_fwd(x, w, b, 1e-5, axis)[0] * dy).sum()

    _, mean, rstd = ref.norm_fwd(x, w, b, 1e-5, axis)
    g = ref.norm_bwd(x, w, mean, rstd, dy, None, axis)
    for k, v in (("dx", x), ("dweight", w), ("dbias", b)):
        num = np.empty_like(v)
        for idx in np.ndindex(v.shape):
            a = dict(x=x, w=w, b=b)
            key = {"dx": "x", "dweight": "w", "dbias": "b"}[k]
            up, down = v.copy(), v.copy()
            up[idx] += 1e-5
            down[idx] -= 1e-5
            num[idx] = (loss(**{**a, key: up}) - loss(**{**a, key: down})) / 2e-5
        assert np.max(np.abs(num - g[k])) < 1e-6, k
