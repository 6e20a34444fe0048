"""Linear attention with a decay for each head and the group norm behind it: what is measured of them.

Each case is one call as a training or serving program makes it.  With `own` false `run` computes the operators in
elementary torch operations; with `own` true it calls the entry points of selective_state_space_28_amd.

Linear attention, per batch row and head h of `heads` (q, k and v may have fewer heads, each shared by consecutive ones):

    S_t = exp(g_h) S_{t-1} + k_t v_t^T        S_{t-1} = 0 where a sequence starts at t; S is (dk, dv)
    y_t = scale q_t S_t                       scale = 1 / sqrt(dk)

over (batch, seqlen, heads, width) tensors, the steps of a row behind its length left out (their y and gradients are 0).

The group norm normalises each group of consecutive channels of a token, y = n act(z) or act(n) with
n = (x - mean) rstd weight + bias.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
EPS = 1e-5


# ---- the cases ------------------------------------------------------------------------------------------------------

def _attn(op, name, batch, seqlen, heads, dk, dv, dtype, decay="retention", hq=None, hk=None, hv=None, packed=False,
          padded=False, state=False, fused=False, decay_grad=False):
    return {"op": op, "name": name, "batch": batch, "seqlen": seqlen, "heads": heads, "hq": hq or heads,
            "hk": hk or heads, "hv": hv or heads, "dk": dk, "dv": dv, "dtype": dtype, "decay": decay, "packed": packed,
            "padded": padded, "state": state, "fused": fused, "decay_grad": decay_grad}


def _norm(op, name, tokens, dim, groups, dtype, gate, act, affine=True, fused=False):
    return {"op": op, "name": name, "tokens": tokens, "dim": dim, "groups": groups, "dtype": dtype, "gate": gate,
            "act": act, "affine": affine, "fused": fused}


def listed():
    return [
        # the forward pass of one training step, 40 heads of 128: the widest call
        _attn("attn_fwd", "attn_train_wide", 16, 2048, 40, 128, 128, "bf16"),
        # one long prompt, continued from a state, read from one projection's output: prefill at batch 1
        _attn("attn_fwd", "attn_long_prompt", 1, 65536, 16, 128, 128, "bf16", "slopes", state=True, fused=True),
        # a batch of padded prompts, 80 heads of 64 values on one shared head of 128 keys
        _attn("attn_fwd", "attn_shared_keys", 16, 2048, 80, 128, 64, "bf16", hq=1, hk=1, padded=True, state=True),
        # several short sequences packed into rows of an odd length, odd widths, in float32
        _attn("attn_fwd", "attn_packed_odd", 3, 1777, 10, 50, 100, "f32", "slopes", packed=True, state=True),
        # the backward pass of the wide call at half the batch
        _attn("attn_bwd", "attn_bwd_wide", 8, 2048, 40, 128, 128, "bf16"),
        # a small model trained in float32 on packed documents, its decays learned too
        _attn("attn_bwd", "attn_bwd_packed", 8, 2047, 12, 128, 128, "f32", "slopes", packed=True, state=True,
              decay_grad=True),
        # one token for each of many running requests, a few of them at their first
        _attn("attn_step", "attn_step_many", 256, 1, 40, 128, 128, "bf16", packed=True, state=True),
        # one token of one request: nothing but latency
        _attn("attn_step", "attn_step_one", 1, 1, 12, 128, 128, "f32", "slopes", state=True),
        # the gated norm of the heads' outputs over the tokens of a training batch
        _norm("group_fwd", "group_tokens", 32768, 5120, 40, "bf16", True, "silu"),
        # the same for one token per running request, the gate read from one projection's output
        _norm("group_fwd", "group_step", 256, 5120, 40, "bf16", True, "silu", fused=True),
        # the backward of group_tokens at half the batch
        _norm("group_bwd", "group_bwd_tokens", 16384, 5120, 40, "bf16", True, "silu"),
        # the backward of a norm with an activation and no gate: float32, odd groups
        _norm("group_bwd", "group_bwd_odd", 16376, 1000, 8, "f32", False, "silu"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))


def _shared(rng, heads):
    """A number of heads that divides `heads`."""
    return rng.choice([n for n in range(1, heads + 1) if heads % n == 0]) if rng.random() < 0.3 else heads


def draw(rng):
    op = rng.choice(["attn_fwd", "attn_bwd", "attn_step", "group_fwd", "group_bwd"])
    dtype = rng.choice(["bf16", "f32"])
    if op.startswith("attn"):
        heads = _log_int(rng, 1, 40)
        dk, dv = (rng.choice([16, 64, 80, 128, 256, rng.randint(1, 256)]) for _ in range(2))
        if op == "attn_step":
            seqlen, batch = 1, _log_int(rng, 1, min(256, (1 << 27) // (heads * dk * dv)))
        else:
            most = (1 << 25) // (heads * max(dk, dv))
            seqlen = _log_int(rng, 1, min(32768 if op == "attn_fwd" else 8192, most))
            batch = _log_int(rng, 1, max(1, min(16, most // seqlen)))
        shared = [_shared(rng, heads) for _ in range(3)]
        return _no_name(_attn(op, "", batch, seqlen, heads, dk, dv, dtype, rng.choice(["retention", "slopes"]), *shared,
                              packed=rng.random() < 0.4, padded=op != "attn_step" and rng.random() < 0.3,
                              state=op == "attn_step" or rng.random() < 0.5, fused=rng.random() < 0.3,
                              decay_grad=op == "attn_bwd" and rng.random() < 0.5))
    width = rng.choice([16, 64, 128, 256, _log_int(rng, 1, 2048)])
    groups = _log_int(rng, 1, max(1, 8192 // width))
    tokens = _log_int(rng, 1, min(65536, (1 << 25) // (width * groups)))
    return _no_name(_norm(op, "", tokens, width * groups, groups, dtype, rng.random() < 0.6,
                          rng.choice(["none", "silu", "sigmoid"]), rng.random() < 0.8, rng.random() < 0.3))


def _no_name(case):
    del case["name"]
    return case


def _lengths(case):
    """Lengths of a padded batch's rows: from a whole row down to half of one, the last row empty where there are four."""
    b, L = case["batch"], case["seqlen"]
    n = [L - (i * L) // (2 * b) for i in range(b)]
    if b >= 4:
        n[-1] = 0
    return n


# ---- inputs ---------------------------------------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 1000003 + 29)
    dt = TYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)

    s = {"case": case}
    if case["op"].startswith("group"):
        n, dim, groups = case["tokens"], case["dim"], case["groups"]
        s["x"] = normal(n, dim) + normal(n, 1, scale=0.5)
        s["weight"] = 1.0 + normal(dim, scale=0.1, dtype=torch.float32) if case["affine"] else None
        s["bias"] = normal(dim, scale=0.1, dtype=torch.float32) if case["affine"] else None
        s["z"] = None
        if case["gate"]:  # beside another block of the projection's output, or alone
            s["z"] = normal(n, 2 * dim)[:, dim:] if case["fused"] else normal(n, dim)
        if case["op"] == "group_bwd":  # what the forward pass left, and the gradient that arrives
            wide = s["x"].double().view(n, groups, -1)
            s["mean"] = wide.mean(-1).float()
            s["rstd"] = (wide.var(-1, unbiased=False) + EPS).rsqrt().float()
            s["dy"] = normal(n, dim)
        return s

    b, L, H, dk, dv = (case[k] for k in ("batch", "seqlen", "heads", "dk", "dv"))
    lead = (b,) if case["op"] == "attn_step" else (b, L)
    heads = {"q": (case["hq"], dk), "k": (case["hk"], dk), "v": (case["hv"], dv)}
    if case["fused"]:  # views of one projection's output
        rows = normal(*lead, sum(h * d for h, d in heads.values()))
        at = 0
        for name, (h, d) in heads.items():
            s[name] = rows[..., at:at + h * d].unflatten(-1, (h, d))
            at += h * d
    else:
        for name, (h, d) in heads.items():
            s[name] = normal(*lead, h, d)
    i = torch.arange(H, device="cuda", dtype=torch.float64)
    if case["decay"] == "retention":  # decays of 1 - 2^-5 to 1 - 2^-12 a step
        s["g"] = torch.log1p(-torch.exp2(-5 - 7 * i / max(1, H - 1))).float()
    else:  # slopes of 2^(-8 (i + 1) / H): from a few steps of memory to some 250
        s["g"] = -torch.exp2(-8 * (i + 1) / H).float()
    s["starts"] = s["lengths"] = s["h0"] = None
    if case["packed"]:  # about five sequences to a row; of the running requests, some at their first token
        s["starts"] = (torch.rand(lead, generator=gen, device="cuda") < (0.2 if L == 1 else 5.0 / L)).to(torch.uint8)
    if case["padded"]:
        s["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
    if case["state"]:
        s["h0"] = normal(b, H, dk, dv, dtype=torch.float32)
    if case["op"] == "attn_bwd":
        s["dy"] = normal(b, L, H, dv)
        s["dlast"] = normal(b, H, dk, dv, scale=0.1, dtype=torch.float32) if case["state"] else None
    return s


# ---- one pass -------------------------------------------------------------------------------------------------------

def run(s):
    case = s["case"]
    if own:
        import selective_state_space_28_amd as ssm
        if case["op"] == "group_fwd":
            return ssm.ssm_group_norm_fwd(s["x"], case["groups"], s["weight"], s["bias"], s["z"], act=case["act"],
                                          eps=EPS, return_stats=True)
        if case["op"] == "group_bwd":
            g = ssm.ssm_group_norm_bwd(s["x"], case["groups"], s["weight"], s["bias"], s["z"], act=case["act"],
                                       mean=s["mean"], rstd=s["rstd"], dy=s["dy"])
            return tuple(g[k] for k in ("dx", "dz", "dweight", "dbias"))
        qkv = (s["q"], s["k"], s["v"], s["g"])
        if case["op"] == "attn_step":
            after = torch.empty_like(s["h0"])  # the state before the token is kept, to step back to
            return ssm.ssm_linear_attn_state_update(s["h0"], *qkv, starts=s["starts"], state_out=after), after
        rows = dict(starts=s["starts"], lengths=s["lengths"], h0=s["h0"])
        if case["op"] == "attn_fwd":
            return ssm.ssm_linear_attn_fwd(*qkv, **rows, return_last_state=case["state"])
        g = ssm.ssm_linear_attn_bwd(*qkv, **rows, dy=s["dy"], dlast_state=s["dlast"], decay_grad=case["decay_grad"])
        return tuple(g[k] for k in ("dq", "dk", "dv", "dlog_decay", "dh0"))
    if case["op"] == "group_fwd":
        return _plain_group_fwd(s)
    if case["op"] == "group_bwd":
        return _plain_group_bwd(s)
    if case["op"] == "attn_step":
        return _plain_step(s)
    return _plain_attn(s)


# ---- the plain forms ------------------------------------------------------------------------------------------------

CHUNK = 64


def _spread(t, heads):
    """Shared heads, one for each of `heads`."""
    return t if t.shape[-2] == heads else t.repeat_interleave(heads // t.shape[-2], -2)


def _gathered(t, heads):
    """The gradient of shared heads: the sum over those that share one."""
    n = t.shape[-2]
    return t if n == heads else t.unflatten(-2, (heads, n // heads)).sum(-2)


def _chunks(t, heads, pad):
    """(batch, L, h, d) -> (batch, heads, chunks, CHUNK, d) in 32 bits, zeros behind the last step."""
    t = _spread(t.float(), heads).transpose(1, 2)
    if pad:
        t = torch.cat([t, t.new_zeros(t.shape[0], t.shape[1], pad, t.shape[3])], 2)
    return t.unflatten(2, (-1, CHUNK)).contiguous()


def _whole(t, L):
    return t.flatten(2, 3)[:, :, :L].transpose(1, 2)


def _plain_attn(s):
    """Chunks of 64 steps: within a chunk the masked product, from chunk to chunk the state."""
    case, dt = s["case"], s["q"].dtype
    b, L, H, dk, dv = (case[k] for k in ("batch", "seqlen", "heads", "dk", "dv"))
    dev, scale = s["q"].device, case["dk"] ** -0.5
    n = -(-L // CHUNK)
    pad = n * CHUNK - L
    q, k, v = (_chunks(s[name], H, pad) for name in ("q", "k", "v"))
    pos = torch.arange(n * CHUNK, device=dev)
    lengths = torch.full((b,), L, device=dev) if s["lengths"] is None else s["lengths"].long()
    live = (pos < lengths[:, None]).view(b, 1, n, CHUNK)  # steps behind a row's length decay nothing and add nothing
    q, k, v = (torch.where(live[..., None], t, 0.0) for t in (q, k, v))
    steps = live.long().cumsum(-1)  # steps taken, up to and with each
    cuts = torch.zeros(b, 1, n, CHUNK, dtype=torch.long, device=dev)
    if s["starts"] is not None:
        cuts.view(b, -1)[:, :L] = (s["starts"] != 0).long()
    cuts = (cuts * live).cumsum(-1)  # starts seen, up to and with each
    g = s["g"].double().view(1, H, 1, 1)

    def weight(exponent, kept):  # the exponents are in 64 bits: g times a chunk's steps
        return torch.where(kept, torch.exp(g.view([1, H] + [1] * (exponent.dim() - 2)) * exponent), 0.0).float()

    enter = weight(steps, cuts == 0)  # of the state that enters the chunk, at each step
    leave = weight(steps[..., -1:] - steps, cuts == cuts[..., -1:])  # of each step, in the state that leaves
    through = weight(steps[..., -1:], cuts[..., -1:] == 0)
    apart = steps[..., :, None] - steps[..., None, :]
    tri = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=dev).tril()
    W = weight(apart, tri & (cuts[..., :, None] == cuts[..., None, :]))
    added = (k * leave[..., None]).transpose(-1, -2).contiguous() @ v
    S = torch.zeros(b, H, dk, dv, device=dev) if s["h0"] is None else s["h0"]
    before = torch.empty(b, H, n, dk, dv, device=dev)
    for c in range(n):
        before[:, :, c] = S
        S = through[:, :, c, :, None] * S + added[:, :, c]
    score = scale * (q @ k.transpose(-1, -2).contiguous())
    if case["op"] == "attn_fwd":
        y = (W * score) @ v + scale * enter[..., None] * (q @ before)
        y = _whole(y, L).to(dt).contiguous()
        return (y, S) if case["state"] else y
    dy = torch.where(live[..., None], _chunks(s["dy"], H, pad), 0.0)
    dscore = scale * (dy @ v.transpose(-1, -2).contiguous())
    dq = (W * dscore) @ k + scale * enter[..., None] * (dy @ before.transpose(-1, -2).contiguous())
    added = scale * (q * enter[..., None]).transpose(-1, -2).contiguous() @ dy
    dS = torch.zeros(b, H, dk, dv, device=dev) if s["dlast"] is None else s["dlast"]
    after = torch.empty(b, H, n, dk, dv, device=dev)
    for c in range(n - 1, -1, -1):
        after[:, :, c] = dS
        dS = through[:, :, c, :, None] * dS + added[:, :, c]
    vS = leave[..., None] * (v @ after.transpose(-1, -2).contiguous())
    dkeys = (W * dscore).transpose(-1, -2).contiguous() @ q + vS
    dval = (W * score).transpose(-1, -2).contiguous() @ dy + leave[..., None] * (k @ after)
    dg = None
    if case["decay_grad"]:  # each product times the steps of its decay
        inside = (apart * (W * score * (dy @ v.transpose(-1, -2).contiguous()))).double().sum((0, 2, 3, 4))
        entering = (steps * enter * scale * ((q @ before) * dy).sum(-1)).double().sum((0, 2, 3))
        leaving = ((steps[..., -1:] - steps) * (k * vS).sum(-1)).double().sum((0, 2, 3))
        passing = (steps[..., -1] * through[..., 0] * (before * after).sum((-1, -2))).double().sum((0, 2))
        dg = (inside + entering + leaving + passing).float()
    grads = [_gathered(_whole(t, L), case[h]).to(dt).contiguous() for t, h in ((dq, "hq"), (dkeys, "hk"), (dval, "hv"))]
    return (*grads, dg, dS if case["state"] else None)


def _plain_step(s):
    case = s["case"]
    H = case["heads"]
    q, k, v = (_spread(s[name].float(), H) for name in ("q", "k", "v"))
    decay = torch.exp(s["g"]).view(1, H, 1, 1)
    if s["starts"] is not None:
        decay = torch.where(s["starts"].view(-1, 1, 1, 1) != 0, 0.0, decay)
    S = decay * s["h0"] + k.unsqueeze(-1) * v.unsqueeze(-2)
    y = case["dk"] ** -0.5 * (q.unsqueeze(-1) * S).sum(-2)
    return y.to(s["q"].dtype), S


def _act(case, t):
    """(the activation of t, its derivative)"""
    if case["act"] == "none":
        return t, torch.ones_like(t)
    sg = 1.0 / (1.0 + torch.exp(-t))
    if case["act"] == "sigmoid":
        return sg, sg * (1.0 - sg)
    return t * sg, sg * (1.0 + t * (1.0 - sg))


def _grouped(case, t):
    return t.float().reshape(case["tokens"], case["groups"], -1)


def _plain_affine(s, xhat):
    case = s["case"]
    n = xhat
    if s["weight"] is not None:
        n = n * s["weight"].view(case["groups"], -1)
    if s["bias"] is not None:
        n = n + s["bias"].view(case["groups"], -1)
    return n


def _plain_group_fwd(s):
    case, shape = s["case"], s["x"].shape
    x = _grouped(case, s["x"])
    mean = x.mean(-1, keepdim=True)
    rest = x - mean
    rstd = 1.0 / torch.sqrt((rest * rest).mean(-1, keepdim=True) + EPS)
    n = _plain_affine(s, rest * rstd)
    y = _act(case, n)[0] if s["z"] is None else n * _act(case, _grouped(case, s["z"]))[0]
    return y.reshape(shape).to(s["x"].dtype), mean.squeeze(-1), rstd.squeeze(-1)


def _plain_group_bwd(s):
    case, shape, dt = s["case"], s["x"].shape, s["x"].dtype
    mean, rstd = s["mean"].unsqueeze(-1), s["rstd"].unsqueeze(-1)
    xhat = (_grouped(case, s["x"]) - mean) * rstd
    dy = _grouped(case, s["dy"])
    n = _plain_affine(s, xhat)
    dz = None
    if s["z"] is None:
        dn = dy * _act(case, n)[1]
    else:
        a, slope = _act(case, _grouped(case, s["z"]))
        dn = dy * a
        dz = (dy * n * slope).reshape(shape).to(dt)
    dh = dn if s["weight"] is None else dn * s["weight"].view(case["groups"], -1)
    dx = rstd * (dh - dh.mean(-1, keepdim=True) - xhat * (dh * xhat).mean(-1, keepdim=True))
    dweight = None if s["weight"] is None else (dn * xhat).sum(0).flatten()
    dbias = None if s["bias"] is None else dn.sum(0).flatten()
    return dx.reshape(shape).to(dt), dz, dweight, dbias


# ---- work -----------------------------------------------------------------------------------------------------------

def work(case):
    es = BYTES[case["dtype"]]
    if case["op"].startswith("group"):
        n = case["tokens"] * case["dim"]
        side = 8 * case["tokens"] * case["groups"]
        if case["op"] == "group_fwd":
            return {"bytes": n * es * (3 if case["gate"] else 2) + side + 8 * case["dim"],
                    "flops": n * (13 if case["gate"] else 12)}
        return {"bytes": n * es * (5 if case["gate"] else 3) + side + 16 * case["dim"], "flops": n * 28}
    b, L, H, dk, dv = (case[k] for k in ("batch", "seqlen", "heads", "dk", "dv"))
    steps = sum(_lengths(case)) if case["padded"] else b * L
    qkv = steps * es * ((case["hq"] + case["hk"]) * dk + case["hv"] * dv)
    state = 4 * b * H * dk * dv if case["state"] else 0
    rows = steps if case["packed"] else 0
    inner = steps * H * dk * dv
    if case["op"] != "attn_bwd":  # the state decayed and added to, and read by q
        return {"bytes": qkv + b * L * H * dv * es + 2 * state + rows, "flops": 5 * inner}
    grads = b * L * es * ((case["hq"] + case["hk"]) * dk + case["hv"] * dv)
    # the state and its gradient formed, and three gradients read off them; with the decay's, one product more
    return {"bytes": qkv + steps * H * dv * es + grads + 3 * state + rows,
            "flops": (14 if case["decay_grad"] else 12) * inner}


# ---- the definitions in 64 bits -------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("group"):
        return _exact_group(case, s)
    H, scale = case["heads"], 1.0 / math.sqrt(case["dk"])
    b, L, dk, dv = (case[k] for k in ("batch", "seqlen", "dk", "dv"))
    share = {name: H // case["h" + name] for name in "qkv"}
    dev = s["q"].device

    def at(name, t):  # (batch, heads, d) of step t
        x = s[name] if case["op"] == "attn_step" else s[name][:, t]
        x = x.double()
        return x[:, :, None].expand(-1, -1, share[name], -1).reshape(b, H, -1)

    a = torch.exp(s["g"].double())[None, :, None, None]
    starts = None if s["starts"] is None else (s["starts"].view(b, L) != 0).double()[:, :, None, None, None]
    live = None
    if s["lengths"] is not None:
        live = (torch.arange(L, device=dev) < s["lengths"][:, None]).double()

    def decay(t):  # of the state on its way into step t
        d = a if starts is None else a * (1 - starts[:, t])
        return d if live is None else d * live[:, t, None, None, None] + (1 - live[:, t, None, None, None])

    def only(t, x):  # nothing of a step behind the row's length
        return x if live is None else x * live[:, t].view([b] + [1] * (x.dim() - 1))

    S = torch.zeros(b, H, dk, dv, dtype=torch.float64, device=dev) if s["h0"] is None else s["h0"].double()
    if case["op"] == "attn_step":
        S = S * decay(0)
        S += at("k", 0)[..., None] * at("v", 0)[..., None, :]
        return scale * (S * at("q", 0)[..., None]).sum(-2), S
    if case["op"] == "attn_fwd":
        y = torch.empty(b, L, H, dv, dtype=torch.float64, device=dev)
        S = S.clone()
        for t in range(L):
            S *= decay(t)
            S.addcmul_(only(t, at("k", t))[..., None], at("v", t)[..., None, :])
            y[:, t] = only(t, (S * at("q", t)[..., None]).sum(-2).mul_(scale))
        return (y, S) if case["state"] else y
    dq = torch.empty(b, L, H, dk, dtype=torch.float64, device=dev)
    dkeys, dval = torch.empty_like(dq), torch.empty(b, L, H, dv, dtype=torch.float64, device=dev)
    R = torch.zeros_like(S) if case["decay_grad"] else None  # the state's derivative by g
    dg = torch.zeros(H, dtype=torch.float64, device=dev)
    for t in range(L):
        d = decay(t)
        here = only(t, s["dy"][:, t].double()) * scale
        if R is not None:  # a step left out has decay 1 whatever g is
            R = d * (R + only(t, S))
            dg += ((R * at("q", t)[..., None]).sum(-2) * here).sum((0, 2))
        S = d * S
        S.addcmul_(only(t, at("k", t))[..., None], at("v", t)[..., None, :])
        dq[:, t] = (S * here[..., None, :]).sum(-1)
    dS = torch.zeros_like(S)
    if s["dlast"] is not None:
        dS = s["dlast"].double()
        if R is not None:
            dg += (R * dS).sum((0, 2, 3))
    for t in range(L - 1, -1, -1):
        here = only(t, s["dy"][:, t].double()) * scale
        dS = torch.addcmul(dS, at("q", t)[..., None], here[..., None, :])
        dkeys[:, t] = only(t, (dS * at("v", t)[..., None, :]).sum(-1))
        dval[:, t] = only(t, (dS * at("k", t)[..., None]).sum(-2))
        dS = dS * decay(t)
    grads = [x.view(b, L, H // share[n], share[n], -1).sum(3) for x, n in ((dq, "q"), (dkeys, "k"), (dval, "v"))]
    return (*grads, dg if case["decay_grad"] else None, dS if case["state"] else None)


def _exact_act(kind, t):
    if kind == "none":
        return t, torch.ones_like(t)
    p, m = torch.sigmoid(t), torch.sigmoid(-t)
    return (p, p * m) if kind == "sigmoid" else (t * p, p + t * p * m)


def _exact_group(case, s):
    n, dim, groups = case["tokens"], case["dim"], case["groups"]
    split = (n, groups, dim // groups)
    x = s["x"].double().view(split)
    w = torch.ones(dim, dtype=torch.float64, device=x.device) if s["weight"] is None else s["weight"].double()
    c = torch.zeros_like(w) if s["bias"] is None else s["bias"].double()
    w, c = w.view(split[1:]), c.view(split[1:])
    z = None if s["z"] is None else s["z"].double().reshape(split)
    if case["op"] == "group_fwd":
        var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
        rstd = (var + EPS).rsqrt()
        pre = (x - mean) * rstd * w + c
        y = _exact_act(case["act"], pre)[0] if z is None else pre * _exact_act(case["act"], z)[0]
        return y.view(n, dim), mean[..., 0], rstd[..., 0]
    rstd = s["rstd"].double()[..., None]
    xhat = (x - s["mean"].double()[..., None]) * rstd
    pre = xhat * w + c
    dy = s["dy"].double().view(split)
    dz = None
    if z is None:
        dpre = dy * _exact_act(case["act"], pre)[1]
    else:
        gate, slope = _exact_act(case["act"], z)
        dpre, dz = dy * gate, (dy * pre * slope).view(n, dim)
    d = dpre * w
    size = split[-1]
    dx = (d - d.sum(-1, keepdim=True) / size - xhat * ((d * xhat).sum(-1, keepdim=True) / size)) * rstd
    return (dx.view(n, dim), dz, None if s["weight"] is None else (dpre * xhat).sum(0).view(dim),
            None if s["bias"] is None else dpre.sum(0).view(dim))
