"""The log-depth 64-bit reference (tests/layers_torch_ref.py) is the step-by-step one."""
import numpy as np
import pytest

from tests import layers_ref as ref
from tests import layers_torch_ref as tref


@pytest.mark.parametrize("full", [True, False])
@pytest.mark.parametrize("weight", ["unit", "convex"])
@pytest.mark.parametrize("gate", ["sigmoid", "softplus"])
def test_the_two_references_agree(gate, weight, full):
    """Both in 64 bits over 37 steps of numbers near 1: 1e-13 is some 400 roundings."""
    import torch
    rng = np.random.default_rng(4)
    b, d, L = 2, 3, 37
    tok = lambda: rng.standard_normal((b, d, L))  # noqa: E731
    p = dict(x=tok(), r=tok(), A=-rng.uniform(0.2, 2.0, d), r_bias=None, i=None, i_bias=None, z=None, starts=None, h0=None)
    if full:
        p.update(r_bias=rng.standard_normal(d), i=tok(), i_bias=rng.standard_normal(d), z=tok(),
                 starts=(rng.random((b, L)) < 0.2).astype(np.uint8), h0=rng.standard_normal((b, d)))
    dy, dl = tok(), rng.standard_normal((b, d))
    y, last, states = ref.gated_fwd(p, gate, weight)
    g = ref.gated_bwd(p, dy, dl, gate, weight)
    t = {k: None if v is None else torch.from_numpy(v) for k, v in p.items()}
    y2, last2, before, g2 = tref.gated(t["x"], t["r"], t["A"], t["r_bias"], t["i"], t["i_bias"], t["z"], gate=gate,
                                       weight=weight, starts=t["starts"], h0=t["h0"], dy=torch.from_numpy(dy),
                                       dlast=torch.from_numpy(dl))
    kept = states[:, :, :-1] if p["starts"] is None else np.where(p["starts"][:, None] != 0, 0.0, states[:, :, :-1])
    pairs = [(y, y2), (last, last2), (kept, before)] + [(g[k], g2[k]) for k in g if k != "size" and g[k] is not None]
    pairs += [(g["size"][k], g2["size"][k]) for k in g["size"] if g["size"][k] is not None]
    for u, v in pairs:
        assert np.abs(u - v.numpy()).max() < 1e-13
    for k in ("di", "di_bias", "dz"):
        assert (g[k] is None) == (g2[k] is None)
