"""Measured calls of the operators on heads and groups: linear attention with
a decay for each head (linear_attention: whole prompts, single tokens and the
backward pass), rotary positions (rotary) and the group norm with an
activation (group_norm), together the parts of a mixer that works in heads.

Each operator has a plain form here, in elementary torch operations in 32
bits (the rotary angles in 64: far positions), and the call of the library's
kernel; ``own`` says which of them ``run`` makes.  ``exact`` evaluates the
definitions in 64 bits, apart from the plain form.

Layouts are channels last: q, k, v and their results [N][T][H][D], carried
states [N][H][Dk][Dv] in fp32, maps and their norms [N][P][C] (P positions of
a frame, or one where every token is normed by itself).
"""
import math

import torch

own = False

DEV = "cuda"
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # 64 streams, one token each: a decode step reads and writes the states once
        dict(name="linear_step", op="linear", dir="fwd", n=64, t=1, h=12, qh=12, kh=12, vh=12, dk=64, dv=64, ragged=0,
             dtype="bf16"),
        # one long prompt: few heads, so the time axis has to be split
        dict(name="linear_prompt", op="linear", dir="fwd", n=1, t=8192, h=16, qh=16, kh=16, vh=16, dk=128, dv=128,
             ragged=0, dtype="bf16"),
        # every position of a 30x52 latent map over 17 frames, clips of unequal length
        dict(name="linear_latent", op="linear", dir="fwd", n=1560, t=17, h=6, qh=6, kh=6, vh=6, dk=64, dv=64, ragged=1,
             dtype="bf16"),
        # training on two prompts of odd length, q and k shared by the heads of four groups
        dict(name="linear_train", op="linear", dir="bwd", n=2, t=2049, h=16, qh=4, kh=4, vh=16, dk=64, dv=128, ragged=0,
             dtype="bf16"),
        # odd heads and widths, sequences of unequal length, k and v shared by all heads, fp32
        dict(name="linear_odd_f32", op="linear", dir="bwd", n=3, t=1023, h=5, qh=5, kh=1, vh=1, dk=50, dv=100, ragged=1,
             dtype="f32"),
        # the positions of a decode step: 64 rows, where only latency counts
        dict(name="rotary_step", op="rotary", dir="fwd", n=64, t=1, qh=12, kh=12, d=64, rot=64, first=0, layout="half",
             scaling="none", ragged=0, dtype="bf16"),
        # a piece of a long context behind its first 100000 tokens, frequencies stretched by parts
        dict(name="rotary_prompt", op="rotary", dir="fwd", n=1, t=8192, qh=16, kh=4, d=128, rot=128, first=0,
             layout="interleaved", scaling="parts", ragged=0, dtype="bf16"),
        # training, half of each odd-width head rotated, sequences of unequal length, fp32
        dict(name="rotary_train_f32", op="rotary", dir="bwd", n=2, t=2049, qh=20, kh=20, d=100, rot=50, first=10,
             layout="half", scaling="linear", ragged=1, dtype="f32"),
        # the norm of each of 16 heads of a long prompt's tokens
        dict(name="group_heads", op="group", dir="fwd", n=8192, p=1, c=2048, g=16, act=0, ragged=0, dtype="bf16"),
        # the norm between two residual blocks of a video decoder: four 360x640 frames of 192 channels
        dict(name="group_decoder", op="group", dir="fwd", n=4, p=230400, c=192, g=32, act=1, ragged=0, dtype="bf16"),
        # training on three 180x320 frames of 384 channels
        dict(name="group_train", op="group", dir="bwd", n=3, p=57600, c=384, g=32, act=1, ragged=0, dtype="bf16"),
        # 17 latent frames of unequal valid parts, odd channels, fp32
        dict(name="group_odd_f32", op="group", dir="bwd", n=17, p=1560, c=515, g=5, act=1, ragged=1, dtype="f32"),
    ]


def _log(rng, lo, hi):
    """A whole number spread evenly over the logarithm of [lo, hi]."""
    v = lo * (hi / lo) ** rng.random()
    return max(lo, min(hi, int(round(v))))


def draw(rng):
    op = rng.choice(["linear", "linear", "rotary", "group"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    way = rng.choice(["fwd", "bwd"])
    ragged = rng.choice([0, 1])
    if op == "linear":
        t = rng.choice([1, _log(rng, 2, 8192), _log(rng, 2, 8192)])
        way = "fwd" if t == 1 else way
        dk, dv = rng.choice([16, 32, 50, 64, 64, 100, 128, 128]), rng.choice([16, 32, 50, 64, 64, 100, 128, 128])
        h = rng.choice([1, 2, 4, 5, 6, 12, 16])
        few = rng.choice([x for x in (1, 2, 4) if h % x == 0])
        qh, kh, vh = rng.choice([(h, h, h), (h, h, h), (few, few, h), (h, few, few)])
        # the plain form keeps T x T numbers a head, the 64-bit one a state for each token
        top = min((1 << 30) // (h * t * t), (1 << 29) // (h * t * dk * dv), (1 << 25) // (h * t * max(dk, dv)), 1560)
        n = _log(rng, 1, max(1, top))
        return dict(op=op, dir=way, n=n, t=t, h=h, qh=qh, kh=kh, vh=vh, dk=dk, dv=dv, ragged=ragged, dtype=dtype)
    if op == "rotary":
        t, d = rng.choice([1, _log(rng, 2, 8192)]), rng.choice([32, 64, 64, 100, 128, 128])
        qh = rng.choice([1, 4, 5, 12, 16])
        kh = rng.choice([x for x in (0, 1, 4, 5, 12, 16) if x <= qh])
        n = _log(rng, 1, max(1, min(1560, (1 << 24) // (t * d * (qh + kh)))))
        rot = rng.choice([d, d, d // 2 // 2 * 2])
        first = rng.choice([0, d - rot])
        return dict(op=op, dir=way, n=n, t=t, qh=qh, kh=kh, d=d, rot=rot, first=first,
                    layout=rng.choice(["half", "interleaved"]), scaling=rng.choice(["none", "linear", "base", "parts"]),
                    ragged=ragged, dtype=dtype)
    g = rng.choice([1, 4, 5, 16, 32])
    c = g * _log(rng, max(1, 32 // g), 2048 // g)
    p = rng.choice([1, _log(rng, 2, 230400)])
    p = max(p, -(-16 * g // c))  # groups of a few elements are all but constant
    n = _log(rng, 1, max(1, min(8192, (1 << 25) // (p * c))))
    return dict(op=op, dir=way, n=n, p=p, c=c, g=g, act=rng.choice([0, 1]), ragged=0 if p == 1 else ragged, dtype=dtype)


def work(case):
    """Each input read once, each output written once; multiplications and
    additions of the formulas, an exponential counted as one.  Linear
    attention is counted as its recurrence over blocks of 64 tokens or fewer,
    the least work of any block size near it."""
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "linear":
        n, t, h, dk, dv = case["n"], case["t"], case["h"], case["dk"], case["dv"]
        q, k, v, o = n * t * case["qh"] * dk, n * t * case["kh"] * dk, n * t * case["vh"] * dv, n * t * h * dv
        state = n * h * dk * dv
        near = min(t, 64)
        one = n * t * h * (4 * dk * dv + (near + 1) * (dk + dv))
        if case["dir"] == "fwd":
            return {"bytes": e * (q + k + v + o) + 8 * state, "flops": one}
        return {"bytes": e * (2 * (q + k + v) + o) + 12 * state + 8 * h, "flops": 3 * one}
    if case["op"] == "rotary":
        el = case["n"] * case["t"] * (case["qh"] + case["kh"])
        return {"bytes": 2 * e * el * case["d"], "flops": 3 * el * case["rot"]}
    n, p, c = case["n"], case["p"], case["c"]
    el = n * p * c
    if case["dir"] == "fwd":
        return {"bytes": e * (2 * el + 2 * c) + 8 * n * case["g"], "flops": el * (7 + 4 * case["act"])}
    return {"bytes": e * (3 * el + 2 * c) + 8 * c + 8 * n * case["g"], "flops": el * (14 + 8 * case["act"])}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _rn(g, shape, dtype, scale=1.0, mean=0.0):
    v = torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)
    return v.mul_(scale).add_(mean).to(dtype)


def _lengths(g, n, t, ragged):
    """Valid tokens of every sequence: None when all are full; else 0, 1, T and others in between."""
    if not ragged:
        return None
    v = torch.randint(0, t + 1, (n,), generator=g, device=DEV, dtype=torch.int32)
    v[0] = t
    if n > 2:
        v[1], v[2] = 0, 1
    return v


def _inputs(case, seed):
    g = _gen(seed)
    dt = _DT[case["dtype"]]
    n = case["n"]
    if case["op"] == "linear":
        t, h, dk, dv = case["t"], case["h"], case["dk"], case["dv"]
        wide = [case["qh"] * dk, case["kh"] * dk, case["vh"] * dv]
        qkv = _rn(g, (n, t, sum(wide)), dt)  # parts of one projection
        parts = qkv.split(wide, -1)
        i = {"q": parts[0].unflatten(-1, (case["qh"], dk)), "k": parts[1].unflatten(-1, (case["kh"], dk)),
             "v": parts[2].unflatten(-1, (case["vh"], dv))}
        # from half forgotten each token to a memory of some 250 tokens, spread over the heads
        at = torch.arange(h, device=DEV, dtype=torch.float64) / max(1, h - 1)
        i["log_decay"] = torch.log1p(-torch.exp2(-1.0 - 7.0 * at)).float()
        i["h_in"] = _rn(g, (n, h, dk, dv), torch.float32, 0.3)
        i["lengths"] = _lengths(g, n, t, case["ragged"])
        if case["dir"] == "bwd":
            i["do"] = _rn(g, (n, t, h, dv), dt)
            i["dh_out"] = _rn(g, (n, h, dk, dv), torch.float32, 0.3)
        return i
    if case["op"] == "rotary":
        t, d = case["t"], case["d"]
        qk = _rn(g, (n, t, (case["qh"] + case["kh"]) * d), dt)  # parts of one projection
        i = {"q": qk[..., :case["qh"] * d].unflatten(-1, (case["qh"], d)), "k": None}
        if case["kh"]:
            i["k"] = qk[..., case["qh"] * d:].unflatten(-1, (case["kh"], d))
        i["offsets"] = torch.randint(100000, 120000, (n,), generator=g, device=DEV, dtype=torch.int32)
        i["lengths"] = _lengths(g, n, t, case["ragged"])
        return i
    p, c = case["p"], case["c"]
    i = {"x": _rn(g, (n, p, c), dt, 1.5, 0.5), "w": _rn(g, (c,), dt, 0.2, 1.0), "b": _rn(g, (c,), dt, 0.2)}
    i["lengths"] = _lengths(g, n, p, case["ragged"])
    if case["dir"] == "bwd":
        i["dy"] = _rn(g, (n, p, c), dt)
        # what the forward pass of a training step left: mean and reciprocal root of each group
        i["stats"] = torch.stack([_group_stats(i["x"][k:k + 1].double(), None if i["lengths"] is None else
                                               i["lengths"][k:k + 1], case["g"])[0] for k in range(n)]).float() \
            if n <= 64 else _group_stats(i["x"].double(), i["lengths"], case["g"]).float()
    return i


def _group_stats(x, lengths, g):
    """[N][G][2]: mean and 1 / sqrt(variance + eps) of each group's valid part; zeros where there is none."""
    n, p, c = x.shape
    v = x.reshape(n, p, g, c // g)
    if lengths is None:
        mean = v.mean((1, 3))
        var = (v - mean[:, None, :, None]).square().mean((1, 3))
        return torch.stack([mean, 1.0 / torch.sqrt(var + EPS)], -1)
    on = (torch.arange(p, device=DEV)[None, :] < lengths[:, None])[..., None, None]
    zero = torch.zeros((), device=DEV, dtype=x.dtype)
    count = (lengths.to(x.dtype) * (c // g))[:, None]
    mean = torch.where(on, v, zero).sum((1, 3)) / count.clamp(min=1)
    var = torch.where(on, v - mean[:, None, :, None], zero).square().sum((1, 3)) / count.clamp(min=1)
    return torch.where(count[..., None] > 0, torch.stack([mean, 1.0 / torch.sqrt(var + EPS)], -1), zero)


_ROTARY = {"none": dict(scaling=None), "linear": dict(scaling="linear", factor=4.0),
           "base": dict(scaling="base", factor=4.0), "parts": dict(scaling="parts", factor=16.0, original=8192)}


def prepare(case, seed):
    i = _inputs(case, seed)
    st = {"case": dict(case), "in": i}
    if not own:
        return st
    import causal_conv3d_video_amd as cc3d

    dt = _DT[case["dtype"]]
    f32 = torch.float32

    def like(t, dtype=None):
        return None if t is None else torch.empty(t.shape, dtype=dtype or t.dtype, device=DEV)

    if case["op"] == "linear":
        plan = cc3d.linear_attention_plan(cc3d.make_linear_attention_desc(
            case["n"], case["t"], case["h"], case["dk"], case["dv"], q_heads=case["qh"], k_heads=case["kh"],
            v_heads=case["vh"], dtype=dt))
        if case["dir"] == "fwd":
            st["out"] = {"o": torch.empty((case["n"], case["t"], case["h"], case["dv"]), dtype=dt, device=DEV),
                         "h_out": like(i["h_in"])}
        else:
            st["out"] = {"dq": like(i["q"]), "dk": like(i["k"]), "dv": like(i["v"]),
                         "dlog_decay": like(i["log_decay"]), "dh_in": like(i["h_in"])}
    elif case["op"] == "rotary":
        plan = cc3d.rotary_plan(cc3d.make_rotary_desc(
            case["n"], case["t"], case["qh"], case["kh"], case["d"], rot=case["rot"], first=case["first"],
            layout=case["layout"], dtype=dt, **_ROTARY[case["scaling"]]))
        st["out"] = {"q_out": like(i["q"]), "k_out": like(i["k"])}
    else:
        plan = cc3d.group_norm_plan(cc3d.make_group_norm_desc(case["n"], case["p"], case["c"], case["g"],
                                                              act="silu" if case["act"] else None, eps=EPS, dtype=dt))
        if case["dir"] == "fwd":
            st["out"] = {"y": like(i["x"]), "stats": torch.empty((case["n"], case["g"], 2), dtype=f32, device=DEV)}
        else:
            st["out"] = {"dx": like(i["x"]), "dw": like(i["w"], f32), "db": like(i["b"], f32)}
    st["plan"] = plan
    nbytes = plan.info["backward_workspace_bytes" if case["dir"] == "bwd" else "workspace_bytes"]
    st["workspace"] = torch.empty(nbytes, dtype=torch.uint8, device=DEV) if nbytes else None
    return st


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(state):
    case, i = state["case"], state["in"]
    if own:
        return _run_own(state, case, i)
    if case["op"] == "linear":
        out = _linear_plain(i, case) if case["dir"] == "fwd" else _linear_plain_bwd(i, case)
    elif case["op"] == "rotary":
        out = _rotary_plain(i, case)
    else:
        out = _group_plain(i, case) if case["dir"] == "fwd" else _group_plain_bwd(i, case)
    return {k: v for k, v in out.items() if v is not None}


def _run_own(state, case, i):
    import causal_conv3d_video_amd as cc3d

    o, plan, ws, ln = state["out"], state["plan"], state["workspace"], i["lengths"]
    if case["op"] == "linear":
        if case["dir"] == "fwd":
            cc3d.linear_attention_forward(plan, i["q"], i["k"], i["v"], o["o"], log_decay=i["log_decay"],
                                          h_in=i["h_in"], h_out=o["h_out"], lengths=ln, workspace=ws)
        else:
            cc3d.linear_attention_backward(plan, i["q"], i["k"], i["v"], i["do"], log_decay=i["log_decay"],
                                           h_in=i["h_in"], dh_out=i["dh_out"], lengths=ln, workspace=ws, **o)
    elif case["op"] == "rotary":
        if case["dir"] == "fwd":
            cc3d.rotary_forward(plan, i["q"], i["k"], o["q_out"], o["k_out"], offsets=i["offsets"], lengths=ln)
        else:
            cc3d.rotary_backward(plan, i["q"], i["k"], o["q_out"], o["k_out"], offsets=i["offsets"], lengths=ln)
    elif case["dir"] == "fwd":
        cc3d.group_norm_forward(plan, i["x"], o["y"], w=i["w"], b=i["b"], stats=o["stats"], lengths=ln, workspace=ws)
    else:
        cc3d.group_norm_backward(plan, i["x"], i["dy"], w=i["w"], b=i["b"], stats=i["stats"], lengths=ln, workspace=ws,
                                 **o)
    return {k: v for k, v in o.items() if v is not None}


# --------------------------------------------------------------------------
# plain forms, in 32 bits
# --------------------------------------------------------------------------

def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _keep(v, x):
    return x if v is None else torch.where(v, x, torch.zeros((), device=DEV, dtype=x.dtype))


def _spread(x, h, valid):
    """[N][T][H'][D] -> [N][H][T][D] in fp32, each head repeated for those that share it, zero after the valid tokens."""
    x = _keep(valid, x.float())
    return x.repeat_interleave(h // x.shape[2], 2).transpose(1, 2).contiguous()


def _join_heads(x, heads):
    """[N][H][T][D] -> [N][T][heads][D]: the sum over the heads that share one."""
    n, h, t, d = x.shape
    return x.reshape(n, heads, h // heads, t, d).sum(2).transpose(1, 2)


def _linear_parts(i, case):
    n, t, h = case["n"], case["t"], case["h"]
    ln = i["lengths"]
    ln = torch.full((n,), t, device=DEV, dtype=torch.int32) if ln is None else ln
    valid = None if i["lengths"] is None else (torch.arange(t, device=DEV)[None, :] < ln[:, None])[..., None, None]
    q, k, v = (_spread(i[x], h, valid) for x in ("q", "k", "v"))
    at = torch.arange(t, device=DEV, dtype=torch.float32)
    apart = at[:, None] - at[None, :]
    g = i["log_decay"][:, None, None]
    zero = torch.zeros((), device=DEV)
    fade = torch.where(apart >= 0, torch.exp(g * apart.clamp(min=0)), zero)  # [H][T][T]
    lead = torch.exp(g * (at + 1)[:, None])                                  # [H][T][1]: from the state that came in
    left = ln.float()[:, None] - 1 - at[None, :]                             # tokens that follow inside the sequence
    tail = torch.where(left[:, None] >= 0, torch.exp(i["log_decay"][None, :, None] * left.clamp(min=0)[:, None]), zero)[..., None]
    whole = torch.exp(i["log_decay"][None, :] * ln.float()[:, None])[..., None, None]
    return ln, valid, q, k, v, at, apart, fade, lead, left, tail, whole


def _linear_plain(i, case):
    dt = _DT[case["dtype"]]
    ln, valid, q, k, v, at, apart, fade, lead, left, tail, whole = _linear_parts(i, case)
    score = (q @ k.transpose(2, 3).contiguous()) * fade
    o = (score @ v + (q * lead) @ i["h_in"]) * case["dk"] ** -0.5
    h_out = i["h_in"] * whole + (k * tail).transpose(2, 3).contiguous() @ v
    return {"o": _keep(valid, o.transpose(1, 2)).to(dt).contiguous(), "h_out": h_out}


def _linear_plain_bwd(i, case):
    dt = _DT[case["dtype"]]
    ln, valid, q, k, v, at, apart, fade, lead, left, tail, whole = _linear_parts(i, case)
    do = _spread(i["do"], case["h"], valid) * case["dk"] ** -0.5
    score, dscore = q @ k.transpose(2, 3).contiguous(), do @ v.transpose(2, 3).contiguous()
    # the decay: every pair by its distance, the state that came in, and the one that is left
    into = (q * lead) @ i["h_in"]
    dlog = (score * dscore * fade * apart).sum((0, 2, 3)) + ((into * do).sum(3) * (at + 1)).sum((0, 2))
    dscore = dscore * fade
    score = score * fade
    back = i["dh_out"].transpose(2, 3).contiguous()
    dq = dscore @ k + (do @ i["h_in"].transpose(2, 3).contiguous()) * lead
    away = (v * tail) @ back
    dk = dscore.transpose(2, 3).contiguous() @ q + away
    dv = score.transpose(2, 3).contiguous() @ do + (k * tail) @ i["dh_out"]
    dh_in = (q * lead).transpose(2, 3).contiguous() @ do + i["dh_out"] * whole
    dlog = dlog + ((away * k).sum(3) * left[:, None]).sum((0, 2))
    dlog = dlog + ((i["dh_out"] * i["h_in"] * whole).sum((2, 3)) * ln.float()[:, None]).sum(0)
    return {"dq": _join_heads(dq, case["qh"]).to(dt).contiguous(), "dk": _join_heads(dk, case["kh"]).to(dt).contiguous(),
            "dv": _join_heads(dv, case["vh"]).to(dt).contiguous(), "dlog_decay": dlog, "dh_in": dh_in}


def _frequencies(case):
    """Angle per position of each pair, in 64 bits, and the results' amplitude."""
    rot, theta = case["rot"], 10000.0
    s = _ROTARY[case["scaling"]]
    at = torch.arange(rot // 2, device=DEV, dtype=torch.float64) * 2 / rot
    if case["scaling"] == "base":
        theta = theta * s["factor"] ** (rot / (rot - 2))
    f = torch.exp(at * -math.log(theta))
    if case["scaling"] == "linear":
        f = f / s["factor"]
    if case["scaling"] == "parts":
        turns = s["original"] * f / (2 * math.pi)
        own_part = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        return f * own_part + f / s["factor"] * (1 - own_part), 0.1 * math.log(s["factor"]) + 1
    return f, 1.0


def _rotary_plain(i, case):
    t, rot, first, dt = case["t"], case["rot"], case["first"], _DT[case["dtype"]]
    f, amplitude = _frequencies(case)
    pos = i["offsets"][:, None].double() + torch.arange(t, device=DEV, dtype=torch.float64)
    angle = pos[..., None] * f
    c = (torch.cos(angle) * amplitude).float()[:, :, None]
    s = (torch.sin(angle) * amplitude).float()[:, :, None]
    if case["dir"] == "bwd":
        s = -s
    valid = None
    if i["lengths"] is not None:
        valid = (torch.arange(t, device=DEV)[None, :] < i["lengths"][:, None])[..., None, None]

    def turn(x):
        if x is None:
            return None
        x = _keep(valid, x.float())
        part = x[..., first:first + rot]
        if case["layout"] == "half":
            a, b = part[..., :rot // 2], part[..., rot // 2:]
            part = torch.cat([a * c - b * s, a * s + b * c], -1)
        else:
            a, b = part[..., 0::2], part[..., 1::2]
            part = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
        return torch.cat([x[..., :first], part, x[..., first + rot:]], -1).to(dt)

    return {"q_out": turn(i["q"]), "k_out": turn(i["k"])}


def _group_parts(i, case, stats):
    n, p, c, g = case["n"], case["p"], case["c"], case["g"]
    valid = None
    if i["lengths"] is not None:
        valid = (torch.arange(p, device=DEV)[None, :] < i["lengths"][:, None])[..., None]
    x = _keep(valid, i["x"].float())
    mean, rs = (stats[..., k].repeat_interleave(c // g, 1)[:, None] for k in (0, 1))
    xn = _keep(valid, (x - mean) * rs)
    return valid, xn, rs, xn * i["w"].float() + i["b"].float()


def _group_plain(i, case):
    stats = _group_stats(i["x"].float(), i["lengths"], case["g"])
    valid, _, _, y = _group_parts(i, case, stats)
    if case["act"]:
        y = y * _sigmoid(y)
    return {"y": _keep(valid, y).to(_DT[case["dtype"]]), "stats": stats}


def _group_plain_bwd(i, case):
    n, p, c, g = case["n"], case["p"], case["c"], case["g"]
    valid, xn, rs, pre = _group_parts(i, case, i["stats"])
    d = i["dy"].float()
    if case["act"]:
        s = _sigmoid(pre)
        d = d * s * (1.0 + pre * (1.0 - s))
    d = _keep(valid, d)
    dw, db = (d * xn).sum((0, 1)), d.sum((0, 1))
    d = d * i["w"].float()
    count = float(p * (c // g)) if valid is None else (i["lengths"].float() * (c // g)).clamp(min=1)[:, None]
    m1 = (d.reshape(n, p, g, -1).sum((1, 3)) / count).repeat_interleave(c // g, 1)[:, None]
    m2 = ((d * xn).reshape(n, p, g, -1).sum((1, 3)) / count).repeat_interleave(c // g, 1)[:, None]
    return {"dx": _keep(valid, (d - m1 - xn * m2) * rs).to(_DT[case["dtype"]]), "dw": dw, "db": db}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    i = {k: (v.double() if v is not None and v.is_floating_point() else v) for k, v in _inputs(case, seed).items()}
    out = {"linear": _linear_exact, "rotary": _rotary_exact, "group": _group_exact}[case["op"]](i, case)
    return {k: v for k, v in out.items() if v is not None}


def _linear_exact(i, case):
    """The recurrence token by token, and its gradient walked back."""
    n, t, h, scale = case["n"], case["t"], case["h"], case["dk"] ** -0.5
    back = case["dir"] == "bwd"
    ln = i["lengths"] if i["lengths"] is not None else torch.full((n,), t, device=DEV, dtype=torch.int32)
    lam = torch.exp(i["log_decay"])[None, :, None, None]
    of = {x: torch.arange(h, device=DEV) // (h // i[x].shape[2]) for x in ("q", "k", "v")}
    s, kept = i["h_in"], [i["h_in"]]
    o = torch.zeros((n, t, h, case["dv"]), device=DEV, dtype=torch.float64)
    for p in range(t):
        on = (p < ln)[:, None, None, None]
        new = lam * s + i["k"][:, p][:, of["k"]][..., None] * i["v"][:, p][:, of["v"]][:, :, None]
        s = torch.where(on, new, s)
        if back:
            kept.append(s)
        else:
            o[:, p] = torch.where(on[..., 0], (i["q"][:, p][:, of["q"]][..., None] * s).sum(2) * scale, 0.0)
    if not back:
        return {"o": o, "h_out": s}
    out = {"d" + x: torch.zeros_like(i[x]) for x in ("q", "k", "v")}
    dlog = torch.zeros((h,), device=DEV, dtype=torch.float64)
    gs = i["dh_out"].clone()
    for p in range(t - 1, -1, -1):
        on = (p < ln)[:, None, None]
        do = torch.where(on, i["do"][:, p], 0.0) * scale
        q, k, v = (i[x][:, p][:, of[x]] for x in ("q", "k", "v"))
        gs = gs + torch.where(on[..., None], q[..., None] * do[:, :, None], 0.0)
        dq = (kept[p + 1] * do[:, :, None]).sum(3)
        dk, dv = (gs * v[:, :, None]).sum(3), (gs * k[..., None]).sum(2)
        for name, x in (("q", dq), ("k", dk), ("v", dv)):
            out["d" + name][:, p].index_add_(1, of[name], torch.where(on, x, 0.0))
        dlog += torch.where(on[..., 0], (gs * kept[p] * lam).sum((2, 3)), 0.0).sum(0)
        gs = torch.where(on[..., None], gs * lam, gs)
    return {**out, "dlog_decay": dlog, "dh_in": gs}


def _rotary_exact(i, case):
    """Every pair as a complex number times one of the angle."""
    rot, first = case["rot"], case["first"]
    s = _ROTARY[case["scaling"]]
    f, amplitude = [], 1.0
    for j in range(rot // 2):
        theta = 10000.0
        if case["scaling"] == "base":
            theta *= s["factor"] ** (rot / (rot - 2))
        v = theta ** (-2.0 * j / rot)
        if case["scaling"] == "linear":
            v /= s["factor"]
        if case["scaling"] == "parts":
            amplitude = 1 + 0.1 * math.log(s["factor"])
            keep = min(1.0, max(0.0, (s["original"] * v / (2 * math.pi) - 1.0) / 31.0))
            v = (1 - keep) * v / s["factor"] + keep * v
        f.append(v)
    angle = (i["offsets"][:, None] + torch.arange(case["t"], device=DEV)).double()[..., None] * \
        torch.tensor(f, device=DEV, dtype=torch.float64)
    factor = torch.polar(torch.full_like(angle, amplitude), -angle if case["dir"] == "bwd" else angle)[:, :, None]
    out = {}
    for name in ("q", "k"):
        x = i[name]
        if x is None:
            continue
        y = x.clone()
        part = y[..., first:first + rot]
        lo, hi = (part[..., :rot // 2], part[..., rot // 2:]) if case["layout"] == "half" else (part[..., 0::2], part[..., 1::2])
        z = torch.complex(lo.contiguous(), hi.contiguous()) * factor
        lo.copy_(z.real)
        hi.copy_(z.imag)
        if i["lengths"] is not None:
            y[torch.arange(case["t"], device=DEV)[None, :] >= i["lengths"][:, None]] = 0
        out[name + "_out"] = y
    return out


def _group_exact(i, case):
    """One sequence or frame after another where they are large, all at once where they are small."""
    n, p, c, g = case["n"], case["p"], case["c"], case["g"]
    back = case["dir"] == "bwd"
    y = torch.zeros_like(i["x"])
    stats = torch.zeros((n, g, 2), device=DEV, dtype=torch.float64)
    dw, db = torch.zeros_like(i["w"]), torch.zeros_like(i["b"])
    for lo in range(0, n, n if n > 64 and i["lengths"] is None else 1):
        hi = n if n > 64 and i["lengths"] is None else lo + 1
        m = p if i["lengths"] is None else int(i["lengths"][lo])
        if m == 0:
            continue
        x = i["x"][lo:hi, :m].unflatten(-1, (g, c // g))
        if back:
            mean, rs = i["stats"][lo:hi, None, :, None, 0], i["stats"][lo:hi, None, :, None, 1]
        else:
            var, mean = torch.var_mean(x, (1, 3), unbiased=False, keepdim=True)
            rs = (var + EPS) ** -0.5
            stats[lo:hi] = torch.stack([mean[:, 0, :, 0], rs[:, 0, :, 0]], -1)
        xn = (x - mean) * rs
        w, b = i["w"].reshape(g, -1), i["b"].reshape(g, -1)
        pre = xn * w + b
        sg = torch.sigmoid(pre)
        if not back:
            y[lo:hi, :m] = (pre * sg if case["act"] else pre).flatten(-2)
            continue
        d = i["dy"][lo:hi, :m].unflatten(-1, (g, c // g))
        if case["act"]:
            d = d * (sg + pre * sg * (1 - sg))
        dw += (d * xn).sum((0, 1)).flatten()
        db += d.sum((0, 1)).flatten()
        d = d * w
        y[lo:hi, :m] = (rs * (d - d.mean((1, 3), keepdim=True) - xn * (d * xn).mean((1, 3), keepdim=True))).flatten(-2)
    return {"dx": y, "dw": dw, "db": db} if back else {"y": y, "stats": stats}
