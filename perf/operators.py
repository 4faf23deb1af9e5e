"""Measured calls of the streaming state-space operators: the short cached
causal convolution (causal_conv1d), the selective state space scan
(selective_scan) and the block join (norm_join: the norm after a block, its
gate, the residual scale and sum, and the norm and activation before the next
block).

Each operator has a plain form here, in elementary torch operations in 32
bits, and the call of the library's kernel; ``own`` says which of them
``run`` makes.  ``exact`` evaluates the definitions in 64 bits, position by
position, apart from the plain form.

Layouts are channels last: activations [N][T][C], B and C of the scan
[N][T][G][S], states [N][C][S] in fp32, convolution taps [K][C].
"""
import torch

own = False

DEV = "cuda"
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # 64 streams, one token each: the short convolution of a decode step, where only latency counts
        dict(name="conv1d_step", op="conv1d", dir="fwd", n=64, t=1, c=768, k=4, wide=2, act=1, ragged=0, dtype="bf16"),
        # every position of a 60x104 latent map over 17 frames, clips of unequal length, fp32
        dict(name="conv1d_latent_f32", op="conv1d", dir="fwd", n=6240, t=17, c=384, k=3, wide=1, act=1, ragged=1,
             dtype="f32"),
        # training on two long prompts; the input is one half of a wider projection
        dict(name="conv1d_train", op="conv1d", dir="bwd", n=2, t=8193, c=2048, k=4, wide=2, act=1, ragged=0,
             dtype="bf16"),
        # 256 streams, one token each: read and write the states once
        dict(name="scan_step", op="scan", dir="fwd", n=256, t=1, c=768, s=16, g=1, ragged=0, dtype="bf16"),
        # one long prompt: too few channels to fill the card, the time axis has to be split
        dict(name="scan_prompt", op="scan", dir="fwd", n=1, t=8192, c=2048, s=16, g=1, ragged=0, dtype="bf16"),
        # every position of a 30x52 latent map over 17 frames, clips of unequal length
        dict(name="scan_latent", op="scan", dir="fwd", n=1560, t=17, c=768, s=16, g=1, ragged=1, dtype="bf16"),
        # a wide state in four groups, odd lengths and a channel count that no vector width divides, fp32
        dict(name="scan_wide_f32", op="scan", dir="fwd", n=3, t=1023, c=500, s=64, g=4, ragged=1, dtype="f32"),
        # training on two prompts of odd length
        dict(name="scan_train", op="scan", dir="bwd", n=2, t=2049, c=2048, s=16, g=2, ragged=0, dtype="bf16"),
        # the block join of a decode step: 64 rows, where only latency counts
        dict(name="join_step", op="join", dir="fwd", r=64, c=768, post="rms", pre="rms", act=0, gate=1, gate_act=1,
             dtype="bf16"),
        # the join between two residual blocks of the video decoder: four 360x640 frames of 192 channels
        dict(name="join_decoder", op="join", dir="fwd", r=921600, c=192, post="rms", pre="rms", act=1, gate=0,
             gate_act=0, dtype="bf16"),
        # training on two long prompts, each element gated
        dict(name="join_train", op="join", dir="bwd", r=16386, c=2048, post="rms", pre="rms", act=0, gate=1, gate_act=1,
             dtype="bf16"),
        # one gate row shared by the 1560 positions of each latent frame, odd channels, mean-centred norms, fp32
        dict(name="join_shared_gate_f32", op="join", dir="bwd", r=26520, c=515, post="layer", pre="layer", act=1,
             gate=1560, gate_act=0, dtype="f32"),
    ]


def _log(rng, lo, hi):
    """A whole number spread evenly over the logarithm of [lo, hi]."""
    v = lo * (hi / lo) ** rng.random()
    return max(lo, min(hi, int(round(v))))


def draw(rng):
    op = rng.choice(["conv1d", "scan", "join"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    way = rng.choice(["fwd", "bwd"])
    if op == "conv1d":
        c, t = _log(rng, 32, 2048), rng.choice([1, _log(rng, 2, 8193)])
        n = _log(rng, 1, max(1, min(6240, (1 << 25) // (c * t))))
        return dict(op=op, dir="fwd" if t == 1 else way, n=n, t=t, c=c, k=rng.choice([2, 3, 4]),
                    wide=rng.choice([1, 2]), act=rng.choice([0, 1]), ragged=rng.choice([0, 1]), dtype=dtype)
    if op == "scan":
        g = rng.choice([1, 1, 2, 4])
        c, s, t = g * _log(rng, 32 // g, 2048 // g), rng.choice([4, 8, 16, 16, 24, 64]), \
            rng.choice([1, _log(rng, 2, 8192)])
        top = (1 << 28) if way == "fwd" else (1 << 27)
        n = _log(rng, 1, max(1, min(1560, top // (c * s * t))))
        return dict(op=op, dir="fwd" if t == 1 else way, n=n, t=t, c=c, s=s, g=g, ragged=rng.choice([0, 1]),
                    dtype=dtype)
    c = _log(rng, 64, 4096)
    r = _log(rng, 1, min(921600, (1 << 25) // c))
    gate = rng.choice([0, 1, 1 + r // rng.choice([2, 5, 17])])
    kinds = rng.choice([("rms", "rms"), ("rms", "rms"), ("layer", "layer"), ("none", "rms"), ("rms", "none")])
    return dict(op=op, dir=way, r=r, c=c, post=kinds[0], pre=kinds[1], act=rng.choice([0, 1]) if kinds[1] != "none" else 0,
                gate=gate, gate_act=rng.choice([0, 1]), dtype=dtype)


def work(case):
    """Each input read once, each output written once; multiplications and
    additions of the formulas, an exponential counted as one."""
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "conv1d":
        n, t, c, k = case["n"], case["t"], case["c"], case["k"]
        el = n * t * c
        if case["dir"] == "fwd":
            return {"bytes": e * (2 * el + 2 * n * (k - 1) * c + (k + 1) * c), "flops": el * (2 * k + 1 + 4 * case["act"])}
        return {"bytes": e * (3 * el + 3 * n * (k - 1) * c + (k + 1) * c) + 4 * (k + 1) * c,
                "flops": el * (6 * k + 2 + 8 * case["act"])}
    if case["op"] == "scan":
        n, t, c, s, g = case["n"], case["t"], case["c"], case["s"], case["g"]
        el, bc, st = n * t * c, 2 * n * t * g * s, n * c * s
        if case["dir"] == "fwd":
            return {"bytes": e * (4 * el + bc) + 4 * (2 * st + c * s + 2 * c), "flops": el * (7 * s + 12)}
        return {"bytes": e * (7 * el + 2 * bc) + 4 * (3 * st + 2 * c * s + 4 * c), "flops": el * (21 * s + 30)}
    r, c = case["r"], case["c"]
    gates = 0 if case["gate"] == 0 else (r + case["gate"] - 1) // case["gate"]
    np_ = 1 + (case["post"] != "none") + (case["pre"] != "none")
    if case["dir"] == "fwd":
        outs = 1 + (case["pre"] != "none")
        return {"bytes": e * ((2 + outs) * r * c + gates * c + np_ * c), "flops": r * c * 16}
    ins = 3 + (case["pre"] != "none")
    return {"bytes": e * ((ins + 2) * r * c + 2 * gates * c + np_ * c) + 4 * np_ * c, "flops": r * c * 40}


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


def _lengths(g, case):
    """Valid tokens of every sequence: None when all are full; else 0, 1, T and others in between."""
    n, t = case["n"], case["t"]
    if not case["ragged"]:
        return None
    v = torch.randint(0, t + 1, (n,), generator=g, device=DEV, dtype=torch.int32)
    v[0] = t
    if n > 2:
        v[1], v[2] = 0, 1
    return v


def _inputs(case, seed):
    g = _gen(seed)
    dt = _DT[case["dtype"]]
    if case["op"] == "conv1d":
        n, t, c, k = case["n"], case["t"], case["c"], case["k"]
        i = {"w": _rn(g, (k, c), dt, k ** -0.5), "b": _rn(g, (c,), dt, 0.1)}
        i["x"] = _rn(g, (n, t, c * case["wide"]), dt)[..., :c]  # one part of a wider projection
        i["cache_in"] = _rn(g, (n, k - 1, c), dt)
        i["lengths"] = _lengths(g, case)
        if case["dir"] == "bwd":
            i["dy"] = _rn(g, (n, t, c), dt)
            i["dcache_out"] = _rn(g, (n, k - 1, c), dt)
        return i
    if case["op"] == "scan":
        n, t, c, s, gr = case["n"], case["t"], case["c"], case["s"], case["g"]
        i = {"u": _rn(g, (n, t, c), dt)}
        # step sizes between about 0.001 and 0.1 after the softplus, as trained biases leave them
        i["dt"] = _rn(g, (n, t, c), dt, 0.5)
        lo, hi = -6.9, -2.25
        i["dt_bias"] = torch.rand(c, generator=g, device=DEV).mul_(hi - lo).add_(lo)
        i["a"] = -(torch.arange(1, s + 1, device=DEV, dtype=torch.float32)[None, :]
                   * (0.5 + torch.rand((c, 1), generator=g, device=DEV)))
        bc = _rn(g, (n, t, 2 * gr * s), dt)  # B and C are parts of one projection
        i["b"] = bc[..., :gr * s].unflatten(-1, (gr, s))
        i["c"] = bc[..., gr * s:].unflatten(-1, (gr, s))
        i["d"] = _rn(g, (c,), torch.float32, 0.1, 1.0)
        i["z"] = _rn(g, (n, t, 2 * c), dt)[..., c:]  # the other half of the wider projection
        i["h_in"] = _rn(g, (n, c, s), torch.float32, 0.3)
        i["lengths"] = _lengths(g, case)
        if case["dir"] == "bwd":
            i["dy"] = _rn(g, (n, t, c), dt)
            i["dh_out"] = _rn(g, (n, c, s), torch.float32, 0.3)
        return i
    r, c = case["r"], case["c"]
    i = {"residual": _rn(g, (r, c), dt, 2.0), "y": _rn(g, (r, c), dt)}
    i["scale"] = _rn(g, (c,), dt, 0.1, 0.5)
    for side in ("post", "pre"):
        kind = case[side]
        i[side + "_w"] = _rn(g, (c,), dt, 0.2, 1.0) if kind != "none" else None
        i[side + "_b"] = _rn(g, (c,), dt, 0.2) if kind == "layer" else None
    i["gate"] = None
    if case["gate"]:
        i["gate"] = _rn(g, ((r + case["gate"] - 1) // case["gate"], c), dt)
    if case["dir"] == "bwd":
        i["dx_out"] = _rn(g, (r, c), dt)
        i["dh"] = _rn(g, (r, c), dt) if case["pre"] != "none" else None
    return i


EPS = 1e-6


def prepare(case, seed):
    i = _inputs(case, seed)
    st = {"case": dict(case), "in": i}
    if not own:
        return st
    import causal_conv3d_video_amd as cc3d

    dt = _DT[case["dtype"]]
    act = "silu" if case.get("act") else None

    def like(t, dtype=None):
        return None if t is None else torch.empty(t.shape, dtype=dtype or t.dtype, device=DEV)

    def space(nbytes):
        return torch.empty(nbytes, dtype=torch.uint8, device=DEV) if nbytes else None

    f32 = torch.float32
    if case["op"] == "conv1d":
        plan = cc3d.causal_conv1d_plan(cc3d.make_conv1d_desc(case["n"], case["t"], case["c"], case["k"], act=act, dtype=dt))
        if case["dir"] == "fwd":
            st["out"] = {"y": like(i["x"]), "cache_out": like(i["cache_in"])}
        else:
            st["out"] = {"dx": like(i["x"]), "dw": like(i["w"], f32), "db": like(i["b"], f32),
                         "dcache_in": like(i["cache_in"])}
    elif case["op"] == "scan":
        plan = cc3d.selective_scan_plan(cc3d.make_scan_desc(case["n"], case["t"], case["c"], case["s"], groups=case["g"],
                                                            softplus=True, dtype=dt))
        if case["dir"] == "fwd":
            st["out"] = {"y": like(i["u"]), "h_out": like(i["h_in"])}
        else:
            st["out"] = {"du": like(i["u"]), "ddt": like(i["dt"]), "da": like(i["a"]), "db": like(i["b"]),
                         "dc": like(i["c"]), "dd": like(i["d"]), "dz": like(i["z"]), "ddt_bias": like(i["dt_bias"]),
                         "dh_in": like(i["h_in"])}
    else:
        kinds = {"none": None, "rms": "rms", "layer": "layer"}
        plan = cc3d.norm_join_plan(cc3d.make_join_desc(
            case["r"], case["c"], post=kinds[case["post"]], pre=kinds[case["pre"]], act=act,
            gate_act="silu" if case["gate_act"] else None, gate_rows=max(1, case["gate"]), eps=EPS, dtype=dt))
        if case["dir"] == "fwd":
            st["out"] = {"x_out": like(i["residual"]),
                         "h_out": like(i["residual"]) if case["pre"] != "none" else None}
        else:
            st["out"] = {"dresidual": like(i["residual"]), "dy": like(i["y"]), "dgate": like(i["gate"]),
                         "dscale": like(i["scale"], f32),
                         **{"d" + p: like(i[p], f32) for p in ("post_w", "post_b", "pre_w", "pre_b")}}
    st["plan"] = plan
    st["workspace"] = space(plan.info["backward_workspace_bytes" if case["dir"] == "bwd" else "workspace_bytes"])
    return st


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(state):
    case, i = state["case"], state["in"]
    if own:
        return _run_own(state, case, i)
    if case["op"] == "conv1d":
        out = _conv1d_plain(i, case) if case["dir"] == "fwd" else _conv1d_plain_bwd(i, case)
    elif case["op"] == "scan":
        out = _scan_plain(i, case) if case["dir"] == "fwd" else _scan_plain_bwd(i, case)
    else:
        out = _join_plain(i, case) if case["dir"] == "fwd" else _join_plain_bwd(i, case)
    return {k: v for k, v in out.items() if v is not None}


def _run_own(state, case, i):
    import causal_conv3d_video_amd as cc3d

    o, plan, ws = state["out"], state["plan"], state["workspace"]
    if case["op"] == "conv1d":
        if case["dir"] == "fwd":
            cc3d.causal_conv1d_forward(plan, i["x"], i["w"], i["b"], o["y"], cache_in=i["cache_in"],
                                       cache_out=o["cache_out"], lengths=i["lengths"])
        else:
            cc3d.causal_conv1d_backward(plan, i["x"], i["w"], i["b"], i["dy"], dx=o["dx"], dw=o["dw"], db=o["db"],
                                        cache_in=i["cache_in"], dcache_out=i["dcache_out"], dcache_in=o["dcache_in"],
                                        lengths=i["lengths"], workspace=ws)
    elif case["op"] == "scan":
        if case["dir"] == "fwd":
            cc3d.selective_scan_forward(plan, i["u"], i["dt"], i["a"], i["b"], i["c"], o["y"], d=i["d"], z=i["z"],
                                        dt_bias=i["dt_bias"], h_in=i["h_in"], h_out=o["h_out"], lengths=i["lengths"],
                                        workspace=ws)
        else:
            cc3d.selective_scan_backward(plan, i["u"], i["dt"], i["a"], i["b"], i["c"], i["dy"], d=i["d"], z=i["z"],
                                         dt_bias=i["dt_bias"], h_in=i["h_in"], dh_out=i["dh_out"],
                                         lengths=i["lengths"], workspace=ws, **o)
    else:
        p = {k: i[k] for k in ("gate", "scale", "post_w", "post_b", "pre_w", "pre_b")}
        if case["dir"] == "fwd":
            cc3d.norm_join_forward(plan, i["y"], i["residual"], x_out=o["x_out"], h_out=o["h_out"], **p)
        else:
            cc3d.norm_join_backward(plan, i["y"], i["residual"], dx_out=i["dx_out"], dh=i["dh"], workspace=ws, **p, **o)
    return {k: v for k, v in o.items() if v is not None}


# --------------------------------------------------------------------------
# plain forms, in 32 bits
# --------------------------------------------------------------------------

def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _softplus(v):
    return torch.where(v > 20.0, v, torch.log1p(torch.exp(torch.clamp(v, max=20.0))))


def _valid(lengths, n, t):
    """[N][T][1] truth values: the token is inside its sequence; None when all are."""
    if lengths is None:
        return None
    return (torch.arange(t, device=DEV)[None, :] < lengths[:, None])[..., None]


def _keep(v, x):
    return x if v is None else torch.where(v, x, torch.zeros((), device=DEV, dtype=x.dtype))


def _tail(z, lengths, t, k):
    """The last K - 1 tokens of the joined sequence [cache; x] cut at each length."""
    if lengths is None:
        return z[:, t:t + k - 1]
    at = lengths[:, None].long() + torch.arange(k - 1, device=DEV)[None, :]
    return torch.gather(z, 1, at[..., None].expand(-1, -1, z.shape[2]))


def _conv1d_pre(i, case):
    n, t, k = case["n"], case["t"], case["k"]
    v = _valid(i["lengths"], n, t)
    x = _keep(v, i["x"].float())
    z = torch.cat([i["cache_in"].float(), x], 1)
    w = i["w"].float()
    pre = i["b"].float()
    for j in range(k):
        pre = pre + w[j] * z[:, j:j + t]
    return v, z, w, pre


def _conv1d_plain(i, case):
    t, k, dt = case["t"], case["k"], _DT[case["dtype"]]
    v, z, _, pre = _conv1d_pre(i, case)
    y = pre * _sigmoid(pre) if case["act"] else pre
    return {"y": _keep(v, y).to(dt), "cache_out": _tail(z, i["lengths"], t, k).to(dt).contiguous()}


def _conv1d_plain_bwd(i, case):
    t, k, dt = case["t"], case["k"], _DT[case["dtype"]]
    v, z, w, pre = _conv1d_pre(i, case)
    dp = i["dy"].float()
    if case["act"]:
        s = _sigmoid(pre)
        dp = dp * s * (1.0 + pre * (1.0 - s))
    dp = _keep(v, dp)
    dz = torch.zeros_like(z)
    dw = torch.empty_like(w)
    for j in range(k):
        dz[:, j:j + t] += w[j] * dp
        dw[j] = (dp * z[:, j:j + t]).sum((0, 1))
    dco = i["dcache_out"].float()
    if i["lengths"] is None:
        dz[:, t:t + k - 1] += dco
    else:
        at = i["lengths"][:, None].long() + torch.arange(k - 1, device=DEV)[None, :]
        dz.scatter_add_(1, at[..., None].expand(-1, -1, z.shape[2]), dco)
    return {"dx": dz[:, k - 1:].to(dt), "dw": dw, "db": dp.sum((0, 1)), "dcache_in": dz[:, :k - 1].to(dt)}


def _linear_scan(a, b, t):
    """h[t] = a[t] * h[t - 1] + b[t] along axis 1 from h = 0, by doubling: pairs (decay, value) of spans of 1, 2, 4, ...
    tokens are joined.  Overwrites a and b and returns b."""
    step = 1
    while step < t:
        b[:, step:] = b[:, step:] + a[:, step:] * b[:, :t - step]
        a[:, step:] = a[:, step:] * a[:, :t - step]
        step *= 2
    return b


def _scan_parts(i, case):
    n, t, c, g = case["n"], case["t"], case["c"], case["g"]
    v = _valid(i["lengths"], n, t)
    u = _keep(v, i["u"].float())
    raw = i["dt"].float() + i["dt_bias"]
    delta = _keep(v, _softplus(raw))
    vb = None if v is None else v[..., None]
    wide = c // g
    bb = _keep(vb, i["b"].float()).repeat_interleave(wide, 2)  # [N][T][C][S]
    cc = _keep(vb, i["c"].float()).repeat_interleave(wide, 2)
    z = _keep(v, i["z"].float())
    decay = torch.exp(delta[..., None] * i["a"])
    inc = (delta * u)[..., None] * bb
    inc[:, 0] += decay[:, 0] * i["h_in"]
    h = _linear_scan(decay.clone(), inc, t)
    return v, u, raw, delta, bb, cc, z, decay, h


def _scan_plain(i, case):
    dt = _DT[case["dtype"]]
    v, u, _, _, _, cc, z, _, h = _scan_parts(i, case)
    y = ((h * cc).sum(-1) + i["d"] * u) * (z * _sigmoid(z))
    return {"y": _keep(v, y).to(dt), "h_out": h[:, -1].contiguous()}


def _scan_plain_bwd(i, case):
    n, t, c, s, g = case["n"], case["t"], case["c"], case["s"], case["g"]
    dt = _DT[case["dtype"]]
    v, u, raw, delta, bb, cc, z, decay, h = _scan_parts(i, case)
    sg = _sigmoid(z)
    dout = _keep(v, i["dy"].float())
    y0 = (h * cc).sum(-1) + i["d"] * u
    dz = dout * y0 * (sg * (1.0 + z * (1.0 - sg)))
    gy = dout * (z * sg)
    # gradient of the states, from the last token backwards
    gh = gy[..., None] * cc
    gh[:, -1] += i["dh_out"]
    follow = torch.ones_like(decay)
    follow[:, :-1] = decay[:, 1:]
    gh = _linear_scan(follow.flip(1), gh.flip(1), t).flip(1)
    before = torch.cat([i["h_in"][:, None], h[:, :-1]], 1)
    carried = gh * decay * before
    gb = (gh * bb).sum(-1)
    ddelta = (carried * i["a"]).sum(-1) + u * gb
    ddt = _keep(v, ddelta * torch.where(raw > 20.0, torch.ones_like(raw), _sigmoid(raw)))
    da = (carried * delta[..., None]).sum((0, 1))
    db = (gh * (delta * u)[..., None]).reshape(n, t, g, c // g, s).sum(3)
    dc = (h * gy[..., None]).reshape(n, t, g, c // g, s).sum(3)
    if v is not None:
        db, dc = _keep(v[..., None], db), _keep(v[..., None], dc)
    return {"du": (delta * gb + i["d"] * gy).to(dt), "ddt": ddt.to(dt), "da": da, "db": db.to(dt), "dc": dc.to(dt),
            "dd": (gy * u).sum((0, 1)), "dz": dz.to(dt), "ddt_bias": ddt.sum((0, 1)), "dh_in": gh[:, 0] * decay[:, 0]}


def _norm_plain(x, kind, w, b):
    """The norm of every row, and what its gradient needs: the normalised row and the reciprocal root."""
    if kind == "none":
        return x, None, None
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    rs = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    xn = x * rs
    out = xn * w.float()
    return (out if b is None else out + b.float()), xn, rs


def _norm_plain_bwd(dout, kind, w, xn, rs):
    if kind == "none":
        return dout
    d = dout * w.float()
    d = d - xn * (d * xn).mean(-1, keepdim=True)
    if kind == "layer":
        d = d - d.mean(-1, keepdim=True)
    return d * rs


def _gate_plain(i, case):
    if i["gate"] is None:
        return None, None, None
    gt = i["gate"].float()
    s = _sigmoid(gt)
    val = gt * s if case["gate_act"] else gt
    slope = s * (1.0 + gt * (1.0 - s)) if case["gate_act"] else torch.ones_like(gt)
    if case["gate"] == 1:
        return val, slope, None
    at = torch.arange(case["r"], device=DEV) // case["gate"]
    return val[at], slope, at


def _join_parts(i, case):
    n1, xn1, rs1 = _norm_plain(i["y"].float(), case["post"], i["post_w"], i["post_b"])
    val, slope, at = _gate_plain(i, case)
    f = i["scale"].float() if val is None else val * i["scale"].float()
    x = i["residual"].float() + n1 * f
    return n1, xn1, rs1, val, slope, at, f, x


def _join_plain(i, case):
    dt = _DT[case["dtype"]]
    x = _join_parts(i, case)[-1]
    if case["pre"] == "none":
        return {"x_out": x.to(dt), "h_out": None}
    h, _, _ = _norm_plain(x, case["pre"], i["pre_w"], i["pre_b"])
    if case["act"]:
        h = h * _sigmoid(h)
    return {"x_out": x.to(dt), "h_out": h.to(dt)}


def _join_plain_bwd(i, case):
    dt = _DT[case["dtype"]]
    n1, xn1, rs1, val, slope, at, f, x = _join_parts(i, case)
    dx = i["dx_out"].float()
    dpre_w = dpre_b = dpost_w = dpost_b = dgate = None
    if case["pre"] != "none":
        h, xn2, rs2 = _norm_plain(x, case["pre"], i["pre_w"], i["pre_b"])
        dh = i["dh"].float()
        if case["act"]:
            s = _sigmoid(h)
            dh = dh * s * (1.0 + h * (1.0 - s))
        dpre_w = (dh * xn2).sum(0)
        dpre_b = dh.sum(0) if i["pre_b"] is not None else None
        dx = dx + _norm_plain_bwd(dh, case["pre"], i["pre_w"], xn2, rs2)
    along = dx * n1
    dscale = (along if val is None else along * val).sum(0)
    if val is not None:
        dgate = along * i["scale"].float()
        if at is not None:
            dgate = torch.zeros(i["gate"].shape, device=DEV).index_add_(0, at, dgate)
        dgate = (dgate * slope).to(dt)
    dn = dx * f
    if case["post"] != "none":
        dpost_w = (dn * xn1).sum(0)
        dpost_b = dn.sum(0) if i["post_b"] is not None else None
    dy = _norm_plain_bwd(dn, case["post"], i["post_w"], xn1, rs1)
    return {"dresidual": dx.to(dt), "dy": dy.to(dt), "dgate": dgate, "dscale": dscale, "dpost_w": dpost_w,
            "dpost_b": dpost_b, "dpre_w": dpre_w, "dpre_b": dpre_b}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    i = {k: (v.double() if v is not None and v.is_floating_point() else v) for k, v in _inputs(case, seed).items()}
    out = {"conv1d": _conv1d_exact, "scan": _scan_exact, "join": _join_exact}[case["op"]](i, case)
    return {k: v for k, v in out.items() if v is not None}


def _conv1d_exact(i, case):
    """Token by token over a window that slides along each sequence; the gradient is pushed back the same way."""
    n, t, c, k = case["n"], case["t"], case["c"], case["k"]
    ln = i["lengths"] if i["lengths"] is not None else torch.full((n,), t, device=DEV, dtype=torch.int32)
    seq = torch.zeros((n, t + k - 1, c), device=DEV, dtype=torch.float64)
    seq[:, :k - 1] = i["cache_in"]
    seq[:, k - 1:] = torch.where((torch.arange(t, device=DEV)[None, :] < ln[:, None])[..., None], i["x"], 0.0)
    if case["dir"] == "fwd":
        y = torch.zeros((n, t, c), device=DEV, dtype=torch.float64)
        tail = torch.empty_like(i["cache_in"])
        for p in range(t):
            v = i["b"] + (seq[:, p:p + k] * i["w"]).sum(1)
            v = v * torch.sigmoid(v) if case["act"] else v
            y[:, p] = torch.where((p < ln)[:, None], v, 0.0)
        rows = torch.arange(n, device=DEV)
        for j in range(k - 1):
            tail[:, j] = seq[rows, (ln + j).long()]
        return {"y": y, "cache_out": tail}
    dseq = torch.zeros_like(seq)
    dw, db = torch.zeros_like(i["w"]), torch.zeros_like(i["b"])
    rows = torch.arange(n, device=DEV)
    for j in range(k - 1):
        dseq[rows, (ln + j).long()] += i["dcache_out"][:, j]
    for p in range(t):
        win = seq[:, p:p + k]
        v = i["b"] + (win * i["w"]).sum(1)
        dv = i["dy"][:, p]
        if case["act"]:
            sg = torch.sigmoid(v)
            dv = dv * (sg + v * sg * (1 - sg))
        dv = torch.where((p < ln)[:, None], dv, 0.0)
        dseq[:, p:p + k] += dv[:, None] * i["w"]
        dw += (dv[:, None] * win).sum(0)
        db += dv.sum(0)
    return {"dx": dseq[:, k - 1:], "dw": dw, "db": db, "dcache_in": dseq[:, :k - 1]}


def _scan_exact(i, case):
    """The recurrence token by token."""
    n, t, c, s, g = case["n"], case["t"], case["c"], case["s"], case["g"]
    ln = i["lengths"] if i["lengths"] is not None else torch.full((n,), t, device=DEV, dtype=torch.int32)
    grp = torch.arange(c, device=DEV) // (c // g)
    back = case["dir"] == "bwd"
    h = i["h_in"]
    kept = [h]
    y = torch.zeros((n, t, c), device=DEV, dtype=torch.float64)
    for p in range(t):
        on = (p < ln)[:, None]
        delta = torch.nn.functional.softplus(i["dt"][:, p] + i["dt_bias"])
        new = torch.exp(delta[..., None] * i["a"]) * h + (delta * i["u"][:, p])[..., None] * i["b"][:, p][:, grp]
        h = torch.where(on[..., None], new, h)
        if back:
            kept.append(h)
        else:
            v = (h * i["c"][:, p][:, grp]).sum(-1) + i["d"] * i["u"][:, p]
            zz = i["z"][:, p]
            y[:, p] = torch.where(on, v * zz * torch.sigmoid(zz), 0.0)
    if not back:
        return {"y": y, "h_out": h}
    o = {k: torch.zeros(i[k[1:]].shape, device=DEV, dtype=torch.float64)
         for k in ("du", "ddt", "da", "db", "dc", "dd", "dz", "ddt_bias")}
    gh = i["dh_out"].clone()
    for p in range(t - 1, -1, -1):
        on = (p < ln)[:, None]
        u, zz, dy = i["u"][:, p], i["z"][:, p], torch.where(on, i["dy"][:, p], 0.0)
        raw = i["dt"][:, p] + i["dt_bias"]
        delta = torch.nn.functional.softplus(raw)
        bb, cc = i["b"][:, p][:, grp], i["c"][:, p][:, grp]
        sg = torch.sigmoid(zz)
        o["dz"][:, p] = torch.where(on, dy * ((kept[p + 1] * cc).sum(-1) + i["d"] * u) * (sg + zz * sg * (1 - sg)), 0.0)
        gy = torch.where(on, dy * zz * sg, 0.0)
        gh = gh + gy[..., None] * cc
        decay = torch.exp(delta[..., None] * i["a"])
        through = torch.where(on[..., None], gh * decay * kept[p], 0.0)
        gb = (gh * bb).sum(-1)
        dr = torch.where(on, ((through * i["a"]).sum(-1) + u * gb) * torch.sigmoid(raw), 0.0)
        o["du"][:, p] = torch.where(on, delta * gb + i["d"] * gy, 0.0)
        o["ddt"][:, p] = dr
        o["ddt_bias"] += dr.sum(0)
        o["dd"] += (gy * torch.where(on, u, 0.0)).sum(0)
        o["da"] += (through * delta[..., None]).sum(0)
        o["db"][:, p] = torch.where(on[..., None], gh * (delta * u)[..., None], 0.0).reshape(n, g, c // g, s).sum(2)
        o["dc"][:, p] = torch.where(on[..., None], kept[p + 1] * gy[..., None], 0.0).reshape(n, g, c // g, s).sum(2)
        gh = torch.where(on[..., None], gh * decay, gh)
    o["dh_in"] = gh
    return o


def _join_exact(i, case):
    """Written as a function of its inputs in pieces of whole gate groups; gradients by torch's differentiation of it."""
    names = ["residual", "y", "gate", "scale", "post_w", "post_b", "pre_w", "pre_b"]
    back = case["dir"] == "bwd"
    leaf = {k: (i[k].detach().requires_grad_(back) if i[k] is not None else None) for k in names}

    def norm(v, kind, w, b):
        if kind == "layer":
            v = (v - v.mean(-1, keepdim=True)) / (v.var(-1, unbiased=False, keepdim=True) + EPS).sqrt()
        elif kind == "rms":
            v = v / ((v ** 2).mean(-1, keepdim=True) + EPS).sqrt()
        if w is not None:
            v = v * w
        return v if b is None else v + b

    span = max(1, (1 << 24) // case["c"])
    whole = max(1, case["gate"])
    span = max(whole, span // whole * whole)
    parts = {"x_out": [], "h_out": []}
    with torch.set_grad_enabled(back):
        for lo in range(0, case["r"], span):
            hi = min(case["r"], lo + span)
            m = norm(leaf["y"][lo:hi], case["post"], leaf["post_w"], leaf["post_b"]) * leaf["scale"]
            if leaf["gate"] is not None:
                gt = leaf["gate"][torch.arange(lo, hi, device=DEV) // whole]
                m = m * (gt * torch.sigmoid(gt) if case["gate_act"] else gt)
            x = leaf["residual"][lo:hi] + m
            total = None
            h = None
            if case["pre"] != "none":
                h = norm(x, case["pre"], leaf["pre_w"], leaf["pre_b"])
                h = h * torch.sigmoid(h) if case["act"] else h
            if back:
                total = (x * i["dx_out"][lo:hi]).sum()
                if h is not None:
                    total = total + (h * i["dh"][lo:hi]).sum()
                total.backward()
            else:
                parts["x_out"].append(x)
                if h is not None:
                    parts["h_out"].append(h)
    if not back:
        return {k: torch.cat(v) if v else None for k, v in parts.items()}
    order = ["residual", "y", "gate", "scale", "post_w", "post_b", "pre_w", "pre_b"]
    return {"d" + k: (leaf[k].grad if leaf[k] is not None else None) for k in order}
