"""causal_conv1d, selective_scan and norm_join on the GPU against their plain
64-bit forms (seq_oracle), forward and backward: every type, odd sizes,
strided views, lengths of zero and one, absent optional tensors, NaN in the
tokens after a sequence's valid ones and around the outputs; streamed calls
against one call, repeated calls bit for bit, another stream, a replayed
graph, and gradients against differences of the 64-bit forward form.

Bounds (seq_oracle.assert_close): depth * 2**-24 of the sum of the absolute
values of a result's terms.  Depths, in roundings:
  conv1d forward: K multiply-adds and the bias, twice through the activation's
    slope, and the activation itself (its exponential's argument is rounded at
    |v| <= 8: 16; reciprocal and products: 8): 2 (K + 2) + 32.
  conv1d backward: the slope of the activation carries the argument's error
    (at most half of (K + 2) roundings of a sum of up to 16): 8 (K + 2) + 64;
    dw and db add N T terms.
  scan forward: delta carries up to 64 roundings (1 + exp rounded, at exp
    >= 0.018) into an exponent of at most 8 that matters: 512; four a token;
    the sums over states; the activation: 4 T + 2 S + 640.
  scan backward: the states and their gradient both: twice that, the sums over
    states, tokens and channels: 2 (4 T + 2 S + 640) + N T + C.
  join: rows' sums are trees of at most 32, the norms' conditions are in the
    magnitudes: 256 forward, 1024 backward, and the rows for summed gradients.
"""
import pytest
import torch

import causal_conv3d_video_amd as cc3d
import seq_oracle as so

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F64 = torch.float64
NAN = float("nan")
BF, F32 = torch.bfloat16, torch.float32


def rn(g, *shape, dtype=F32, scale=1.0, mean=0.0):
    """A seeded tensor rounded to dtype, on the CPU."""
    return (torch.randn(*shape, generator=g, dtype=F32) * scale + mean).to(dtype)


def d64(t):
    return None if t is None else t.to(F64)


def dev(t):
    return None if t is None else t.to(DEV)


class Wide:
    """A view of the given shape inside a larger NaN-filled buffer: `pad`
    elements before and after every row and one spare row; `untouched` says
    that nothing around the view was written."""

    def __init__(self, shape, dtype, pad, fill=None):
        n, t, c = shape
        self.buf = torch.full((n, t + 1, c + 2 * pad), NAN, dtype=dtype, device=DEV)
        self.v = self.buf[:, :t, pad:pad + c]
        self.pad, self.t, self.c = pad, t, c
        if fill is not None:
            self.v.copy_(fill)

    def untouched(self):
        b = self.buf.clone()
        b[:, :self.t, self.pad:self.pad + self.c] = NAN
        return bool(torch.isnan(b).all())


def lengths_of(kind, n, t):
    if not kind:
        return None
    v = [(i * 7 + 3) % (t + 1) for i in range(n)]
    for i, x in enumerate((t, 0, 1)):
        if i < n:
            v[i] = min(x, t)
    if n > 3:
        v[3] = t + 5  # longer than the call: clamped
    return v


def poison(x, lengths):
    """NaN in the tokens after the valid ones."""
    x = x.clone()
    for i, ln in enumerate(lengths or []):
        x[i, ln:] = NAN
    return x


def space(plan, backward=False):
    nb = plan.info["backward_workspace_bytes" if backward else "workspace_bytes"]
    return torch.full((nb,), 255, dtype=torch.uint8, device=DEV) if nb else None  # NaN words


def nan(*shape, dtype=F32):
    return torch.full(shape, NAN, dtype=dtype, device=DEV)


# ------------------------------------------------------------------ conv1d

CONV = [
    # n, t, c, k, act, dtype, ragged, pad, cache, bias
    (1, 1, 1, 1, "silu", F32, False, 0, True, True),
    (64, 1, 768, 4, "silu", BF, False, 8, True, True),
    (3, 1, 40, 4, None, BF, True, 0, True, False),
    (2, 2, 7, 4, "silu", F32, False, 3, True, True),
    (4, 9, 24, 3, "silu", BF, True, 0, True, True),
    (5, 33, 96, 4, "silu", BF, True, 8, False, True),
    (2, 65, 520, 2, None, F32, False, 0, True, True),
    (3, 130, 37, 3, "silu", BF, True, 1, True, True),
    (1, 257, 8, 8, "silu", F32, True, 4, True, True),
    (2, 70, 16, 5, "silu", BF, False, 8, True, False),
    (4, 40, 12, 6, None, F32, True, 0, False, False),
    (2, 31, 9, 7, "silu", BF, True, 0, True, True),
]


@pytest.mark.parametrize("n,t,c,k,act,dtype,ragged,pad,cache,bias", CONV)
def test_conv1d_forward_and_backward(cuda_device, n, t, c, k, act, dtype, ragged, pad, cache, bias):
    g = torch.Generator().manual_seed(1000 + n * t + c + k)
    ln = lengths_of(ragged, n, t)
    x, w = rn(g, n, t, c, dtype=dtype), rn(g, k, c, dtype=dtype, scale=k ** -0.5)
    b = rn(g, c, dtype=dtype) if bias else None
    cin = rn(g, n, k - 1, c, dtype=dtype) if cache else None
    dy, dtail = rn(g, n, t, c, dtype=dtype), rn(g, n, k - 1, c, dtype=dtype)
    lt = None if ln is None else torch.tensor(ln, dtype=torch.int32, device=DEV)
    plan = cc3d.causal_conv1d_plan(cc3d.make_conv1d_desc(n, t, c, k, act=act, dtype=dtype))

    xw = Wide((n, t, c), dtype, pad, poison(x, ln))
    yw = Wide((n, t, c), dtype, pad)
    co = nan(n, k - 1, c, dtype=dtype)
    cc3d.causal_conv1d_forward(plan, xw.v, dev(w), dev(b), yw.v, cache_in=dev(cin), cache_out=co, lengths=lt)
    a = (d64(x), d64(w), d64(b), act == "silu", d64(cin), ln)
    y, tail, _ = so.conv1d(*a)
    ym = so.conv1d(*a, mag=True)[0]
    so.assert_close(yw.v, y, ym, 2 * (k + 2) + 32, "y")
    assert yw.untouched()
    assert torch.equal(co.cpu().to(F64), tail)  # copied, not computed

    dyw = Wide((n, t, c), dtype, pad, poison(dy, ln))
    dxw = Wide((n, t, c), dtype, pad)
    dw, db, dci = nan(k, c), nan(c), nan(n, k - 1, c, dtype=dtype)
    cc3d.causal_conv1d_backward(plan, xw.v, dev(w), dev(b), dyw.v, dx=dxw.v, dw=dw, db=db if bias else db,
                                cache_in=dev(cin), dcache_out=dev(dtail), dcache_in=dci, lengths=lt,
                                workspace=space(plan, True))
    ga = (d64(x), d64(w), d64(b), act == "silu", d64(dy), d64(cin), d64(dtail), ln)
    ref, mag = so.conv1d_grad(*ga), so.conv1d_grad(*ga, mag=True)
    depth = 8 * (k + 2) + 64
    for name, got, r, m, dp in zip(("dx", "dw", "db", "dcache_in"), (dxw.v, dw, db, dci), ref, mag,
                                   (depth, depth + n * t, depth + n * t, depth)):
        so.assert_close(got, r, m, dp, name)
    assert dxw.untouched()


def test_conv1d_streamed_calls_equal_one_call_bit_for_bit(cuda_device):
    g = torch.Generator().manual_seed(3)
    n, t, c, k = 3, 23, 96, 4
    x, w, b = dev(rn(g, n, t, c, dtype=BF)), dev(rn(g, k, c, dtype=BF)), dev(rn(g, c, dtype=BF))

    def call(xs, cache):
        plan = cc3d.causal_conv1d_plan(cc3d.make_conv1d_desc(n, xs.shape[1], c, k, act="silu"))
        y, co = nan(n, xs.shape[1], c, dtype=BF), nan(n, k - 1, c, dtype=BF)
        cc3d.causal_conv1d_forward(plan, xs, w, b, y, cache_in=cache, cache_out=co)
        return y, co

    whole, end = call(x, None)
    cache, parts, at = None, [], 0
    for step in (1, 1, 2, 5, 1, 13):
        y, cache = call(x[:, at:at + step], cache)
        parts.append(y)
        at += step
    assert torch.equal(torch.cat(parts, 1), whole) and torch.equal(cache, end)


# -------------------------------------------------------------------- scan

SCAN = [
    # n, t, c, s, g, dtype, ragged, pad, softplus, opts (which of d, z, bias, h are there)
    (1, 1, 1, 1, 1, F32, False, 0, True, "dzbh"),
    (5, 1, 96, 16, 1, BF, False, 8, True, "dzbh"),
    (3, 1, 70, 3, 2, BF, True, 0, True, "dzbh"),
    (4, 1, 40, 64, 4, F32, True, 1, True, "h"),
    (2, 2, 65, 4, 1, F32, False, 0, True, "dzbh"),
    (3, 9, 24, 8, 3, BF, True, 0, True, "dzbh"),
    (4, 17, 130, 16, 2, BF, True, 4, True, "dzbh"),
    (2, 33, 64, 16, 1, F32, False, 0, False, "dz"),
    (1, 300, 70, 16, 1, BF, False, 1, True, "dzbh"),
    (4, 131, 36, 16, 2, F32, True, 0, True, "zbh"),
    (2, 130, 20, 64, 4, F32, True, 0, True, "dzbh"),
    (2, 77, 33, 24, 1, BF, True, 0, True, "dbh"),
    (1, 200, 10, 5, 5, F32, False, 3, True, ""),
    (70, 6, 40, 12, 1, BF, True, 0, True, "dzbh"),
    (2, 65, 9, 40, 3, BF, True, 0, False, "dzbh"),
]


def scan_inputs(n, t, c, s, g_, dtype, softplus, opts, seed):
    g = torch.Generator().manual_seed(seed)
    i = dict(u=rn(g, n, t, c, dtype=dtype), b=rn(g, n, t, g_, s, dtype=dtype), c=rn(g, n, t, g_, s, dtype=dtype),
             dt=rn(g, n, t, c, dtype=dtype, scale=0.7, mean=0.0 if softplus else 0.4),
             a=-(torch.rand(c, s, generator=g) * 3 + 0.1))
    if not softplus:
        i["dt"] = i["dt"].abs()
    i["d"] = rn(g, c) if "d" in opts else None
    i["z"] = rn(g, n, t, c, dtype=dtype) if "z" in opts else None
    i["dt_bias"] = rn(g, c, mean=-1.5) if "b" in opts and softplus else None
    i["h_in"] = rn(g, n, c, s) if "h" in opts else None
    i["dy"] = rn(g, n, t, c, dtype=dtype)
    i["dh_out"] = rn(g, n, c, s) if "h" in opts else None
    return i


@pytest.mark.parametrize("n,t,c,s,g,dtype,ragged,pad,softplus,opts", SCAN)
def test_scan_forward_and_backward(cuda_device, n, t, c, s, g, dtype, ragged, pad, softplus, opts):
    i = scan_inputs(n, t, c, s, g, dtype, softplus, opts, 2000 + n * t + c * s)
    ln = lengths_of(ragged, n, t)
    lt = None if ln is None else torch.tensor(ln, dtype=torch.int32, device=DEV)
    plan = cc3d.selective_scan_plan(cc3d.make_scan_desc(n, t, c, s, groups=g, softplus=softplus, dtype=dtype))

    def wide(x, width=c):
        return None if x is None else Wide((n, t, width), dtype, pad, poison(x.reshape(n, t, width), ln)).v

    gu = dict(dt_bias=dev(i["dt_bias"]), d=dev(i["d"]), h_in=dev(i["h_in"]), z=wide(i["z"]), lengths=lt)
    ins = (wide(i["u"]), wide(i["dt"]), dev(i["a"]), wide(i["b"], g * s), wide(i["c"], g * s))
    yw, ho = Wide((n, t, c), dtype, pad), nan(n, c, s)
    cc3d.selective_scan_forward(plan, *ins, yw.v, h_out=ho, workspace=space(plan), **gu)

    o = [d64(i[k]) for k in ("u", "dt", "a", "b", "c", "d", "z", "dt_bias", "h_in")] + [ln, softplus]
    y, h, _ = so.scan(*o)
    ym, hm, _ = so.scan(*o, mag=True)
    depth = 4 * t + 2 * s + 640
    so.assert_close(yw.v, y, ym, depth, "y")
    so.assert_close(ho, h, hm, depth, "h_out")
    assert yw.untouched()

    outs = {k: Wide((n, t, c), dtype, pad) for k in ("du", "ddt") + (("dz",) if i["z"] is not None else ())}
    outs.update({k: Wide((n, t, g * s), dtype, pad) for k in ("db", "dc")})
    got = {k: v.v for k, v in outs.items()}
    got.update(da=nan(c, s), dh_in=nan(n, c, s))
    if i["d"] is not None:
        got["dd"] = nan(c)
    if i["dt_bias"] is not None:
        got["ddt_bias"] = nan(c)
    dyw = wide(i["dy"])
    cc3d.selective_scan_backward(plan, *ins, dyw, dh_out=dev(i["dh_out"]), workspace=space(plan, True), **gu, **got)
    ga = [d64(i[k]) for k in ("u", "dt", "a", "b", "c", "dy", "d", "z", "dt_bias", "h_in", "dh_out")] + [ln, softplus]
    ref, mag = so.scan_grad(*ga), so.scan_grad(*ga, mag=True)
    for name, v in got.items():
        so.assert_close(v, ref[name].reshape(v.shape), mag[name].reshape(v.shape), 2 * depth + n * t + c, name)
    for name, v in outs.items():
        assert v.untouched(), name


def test_scan_streamed_steps_follow_one_call_and_reuse_the_state(cuda_device):
    """A prompt, then single tokens with h_out = h_in, against one call over all of it."""
    n, t, c, s, head = 4, 21, 96, 16, 13
    i = scan_inputs(n, t, c, s, 2, F32, True, "dzbh", 77)
    fixed = dict(d=dev(i["d"]), dt_bias=dev(i["dt_bias"]))
    seq = {k: dev(i[k]) for k in ("u", "dt", "b", "c", "z")}
    h = dev(i["h_in"]).clone()

    def call(lo, hi, h_out):
        plan = cc3d.selective_scan_plan(cc3d.make_scan_desc(n, hi - lo, c, s, groups=2, dtype=F32))
        p = {k: v[:, lo:hi] for k, v in seq.items()}
        y = nan(n, hi - lo, c)
        cc3d.selective_scan_forward(plan, p["u"], p["dt"], dev(i["a"]), p["b"], p["c"], y, z=p["z"], h_in=h,
                                    h_out=h_out, workspace=space(plan), **fixed)
        return y

    end = nan(n, c, s)
    call(0, t, end)
    ys = [call(0, head, h)] + [call(q, q + 1, h) for q in range(head, t)]
    o = [d64(i[k]) for k in ("u", "dt", "a", "b", "c", "d", "z", "dt_bias", "h_in")]
    y, hr, _ = so.scan(*o)
    ym, hm, _ = so.scan(*o, mag=True)
    depth = 4 * t + 2 * s + 640
    so.assert_close(torch.cat(ys, 1), y, ym, depth, "y")
    so.assert_close(h, hr, hm, depth, "h")
    so.assert_close(end, hr, hm, depth, "h of one call")


def test_scan_decays_to_zero_and_keeps_large_steps_finite(cuda_device):
    """Steps so large that every decay underflows, and steps of zero: exp(-inf) = 0 and exp(0) = 1 exactly."""
    n, t, c, s = 2, 70, 64, 16
    i = scan_inputs(n, t, c, s, 1, F32, False, "h", 78)
    i["dt"][0] = 300.0
    i["dt"][1] = 0.0
    plan = cc3d.selective_scan_plan(cc3d.make_scan_desc(n, t, c, s, softplus=False, dtype=F32))
    y, h = nan(n, t, c), nan(n, c, s)
    cc3d.selective_scan_forward(plan, *[dev(i[k]) for k in ("u", "dt", "a", "b", "c")], y, h_in=dev(i["h_in"]), h_out=h,
                                workspace=space(plan))
    want = 300.0 * d64(i["u"][0, -1])[:, None] * d64(i["b"][0, -1, 0])
    # exp(300 A), A <= -0.1, leaves at most e**-30 of a state of a few hundred
    so.assert_close(h[0], want, want.abs() + 1e-6, 640, "h")
    assert torch.equal(h[1].cpu(), i["h_in"][1])


# -------------------------------------------------------------------- join

JOIN = [
    # r, c, post, pre, act, gate_rows (0: no gate), gate_act, scale, weights, biases, dtype, pad
    (1, 1, "rms", "rms", None, 1, "silu", True, True, False, F32, 0),
    (64, 768, "rms", "rms", None, 1, "silu", True, True, False, BF, 8),
    (37, 96, "rms", "rms", "silu", 0, None, True, True, True, BF, 0),
    (300, 192, "rms", "rms", "silu", 0, None, True, True, False, BF, 8),
    (50, 384, "layer", "layer", None, 7, None, True, True, True, BF, 0),
    (61, 515, "layer", "layer", "silu", 13, "silu", True, True, True, F32, 1),
    (2050, 40, "rms", "layer", None, 3, "silu", False, True, True, F32, 0),
    (1600, 33, None, "rms", "silu", 2, None, True, True, False, BF, 0),
    (33, 2048, "rms", "rms", None, 1, None, True, True, False, BF, 0),
    (9, 4096, "rms", None, None, 5, "silu", True, True, False, F32, 8),
    (5, 8192, "layer", "rms", "silu", 1, "silu", True, True, True, BF, 0),
    (4, 8191, "rms", "layer", None, 4, None, False, False, False, BF, 0),
    (130, 8, None, None, None, 1, "silu", True, False, False, F32, 0),
    (21, 100, "layer", "rms", None, 100, "silu", True, False, True, F32, 2),
]


def join_case(r, c, post, pre, gate_rows, scale, weights, biases, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    gates = 0 if not gate_rows else (r + gate_rows - 1) // gate_rows
    i = dict(y=rn(g, r, c, dtype=dtype), res=rn(g, r, c, dtype=dtype, scale=2.0))
    i["y"][0] = 0  # a row of zeros: the norm's root is that of eps
    i["gate"] = rn(g, gates, c, dtype=dtype) if gates else None
    i["scale"] = rn(g, c, dtype=dtype, scale=0.5) if scale else None
    for side, kind in (("post", post), ("pre", pre)):
        i[side + "_w"] = rn(g, c, dtype=dtype, mean=1.0, scale=0.3) if kind and weights else None
        i[side + "_b"] = rn(g, c, dtype=dtype, scale=0.3) if kind and biases else None
    i["dx_out"], i["dh"] = rn(g, r, c, dtype=dtype), (rn(g, r, c, dtype=dtype) if pre else None)
    return i


def rows_view(x, dtype, pad, r=None, c=None):
    """Rows inside a wider NaN-filled buffer."""
    if x is None and r is None:
        return None
    r, c = (r, c) if x is None else x.shape
    w = Wide((1, r, c), dtype, pad, None if x is None else x[None])
    return w


@pytest.mark.parametrize("r,c,post,pre,act,gate_rows,gate_act,scale,weights,biases,dtype,pad", JOIN)
def test_join_forward_and_backward(cuda_device, r, c, post, pre, act, gate_rows, gate_act, scale, weights, biases,
                                   dtype, pad):
    i = join_case(r, c, post, pre, gate_rows, scale, weights, biases, dtype, 3000 + r + c)
    eps = 1e-5
    plan = cc3d.norm_join_plan(cc3d.make_join_desc(r, c, post=post, pre=pre, act=act, gate_act=gate_act,
                                                   gate_rows=max(1, gate_rows), eps=eps, dtype=dtype))

    def view(x):
        return None if x is None else rows_view(x, dtype, pad).v[0]

    yv, rv, gv = view(i["y"]), view(i["res"]), view(i["gate"])
    par = {k: dev(i[k]) for k in ("scale", "post_w", "post_b", "pre_w", "pre_b")}
    xo = rows_view(None, dtype, pad, r, c)
    ho = rows_view(None, dtype, pad, r, c) if pre else None
    cc3d.norm_join_forward(plan, yv, rv, x_out=xo.v[0], h_out=ho.v[0] if ho else None, gate=gv, **par)
    opts = dict(post=post, pre=pre, act=act == "silu", eps=eps, gate_act=gate_act == "silu",
                gate_rows=max(1, gate_rows), **{k: d64(i[k]) for k in ("gate",) + tuple(par)})
    x, h, (xm, hm) = so.join(d64(i["y"]), d64(i["res"]), **opts)
    so.assert_close(xo.v[0], x, xm, 256, "x_out")
    assert xo.untouched()
    if pre:
        so.assert_close(ho.v[0], h, hm, 256, "h_out")
        assert ho.untouched()

    big = {k: rows_view(None, dtype, pad, *(i["gate"].shape if k == "dgate" else (r, c)))
           for k in ("dy", "dresidual") + (("dgate",) if gate_rows else ())}
    got = {k: v.v[0] for k, v in big.items()}
    got.update({"d" + k: nan(c) for k in par if par[k] is not None})
    cc3d.norm_join_backward(plan, yv, rv, dx_out=view(i["dx_out"]), dh=view(i["dh"]), gate=gv, workspace=space(plan, True),
                            **par, **got)
    ref, mag = so.join_grad(d64(i["y"]), d64(i["res"]), d64(i["dx_out"]), d64(i["dh"]), **opts)
    for k, v in got.items():
        so.assert_close(v, ref[k], mag[k], 1024 + (r if v.dim() == 1 else max(1, gate_rows)), k)
    for k, v in big.items():
        assert v.untouched(), k


@pytest.mark.parametrize("dtype,c", [(BF, 96), (F32, 50)])
def test_join_of_a_first_norm_and_without_a_residual(cuda_device, dtype, c):
    g = torch.Generator().manual_seed(41)
    r = 19
    x, w, dh = rn(g, r, c, dtype=dtype), rn(g, c, dtype=dtype), rn(g, r, c, dtype=dtype)
    plan = cc3d.norm_join_plan(cc3d.make_join_desc(r, c, post=None, pre="rms", act="silu", dtype=dtype))
    opts = dict(post=None, pre="rms", act=True, eps=1e-6, pre_w=d64(w))
    for y, res in ((None, x), (x, None)):
        ho = nan(r, c, dtype=dtype)
        cc3d.norm_join_forward(plan, dev(y), dev(res), h_out=ho, pre_w=dev(w))
        _, h, (_, hm) = so.join(d64(y), d64(res), **opts)
        so.assert_close(ho, h, hm, 256, "h_out")
        name = "dresidual" if y is None else "dy"
        got, dw = nan(r, c, dtype=dtype), nan(c)
        cc3d.norm_join_backward(plan, dev(y), dev(res), dh=dev(dh), pre_w=dev(w), dpre_w=dw, workspace=space(plan, True),
                                **{name: got})
        ref, mag = so.join_grad(d64(y), d64(res), None, d64(dh), **opts)
        so.assert_close(got, ref[name], mag[name], 1024, name)
        so.assert_close(dw, ref["dpre_w"], mag["dpre_w"], 1024 + r, "dpre_w")


def test_join_rows_do_not_reach_each_other(cuda_device):
    """Infinities and NaN in one row stay in that row."""
    g = torch.Generator().manual_seed(43)
    r, c = 70, 96
    y, res = rn(g, r, c, dtype=BF), rn(g, r, c, dtype=BF)
    plan = cc3d.norm_join_plan(cc3d.make_join_desc(r, c, post="layer", pre="rms"))
    clean = nan(r, c, dtype=BF)
    cc3d.norm_join_forward(plan, dev(y), dev(res), h_out=clean)
    y[3, 5], y[40] = float("inf"), NAN
    got = nan(r, c, dtype=BF)
    cc3d.norm_join_forward(plan, dev(y), dev(res), h_out=got)
    keep = torch.ones(r, dtype=torch.bool)
    keep[3] = keep[40] = False
    assert torch.equal(got.cpu()[keep], clean.cpu()[keep])
    assert bool(torch.isnan(got.cpu()[~keep]).any(1).all())


# ------------------------------------------------- gradients by differences

def _along(f, x, v, e):
    return float(f(x + e * v) - f(x - e * v)) / (2 * e)


def test_gpu_gradients_match_differences_of_the_64_bit_forward(cuda_device):
    """<gradient of the kernel, v> against (f(x + e v) - f(x - e v)) / 2e, f in
    float64 with e = 1e-5 (truncation and rounding below 1e-8); the kernel's
    own roundings are bounded as above, here by 4000 * 2**-24 of the sum of
    |gradient * v|, with 1e-6 for the differences."""
    n, t, c, s = 2, 70, 12, 5
    i = scan_inputs(n, t, c, s, 2, F32, True, "dzbh", 91)
    plan = cc3d.selective_scan_plan(cc3d.make_scan_desc(n, t, c, s, groups=2, dtype=F32))
    names = dict(u="du", dt="ddt", a="da", b="db", c="dc", d="dd", z="dz", dt_bias="ddt_bias", h_in="dh_in")
    got = {v: nan(*i[k].shape) for k, v in names.items()}
    j = {k: dev(v) for k, v in i.items()}
    cc3d.selective_scan_backward(plan, j["u"], j["dt"], j["a"], j["b"], j["c"], j["dy"], d=j["d"], z=j["z"],
                                 dt_bias=j["dt_bias"], h_in=j["h_in"], dh_out=j["dh_out"], workspace=space(plan, True),
                                 **got)
    base = {k: d64(v) for k, v in i.items()}
    order = ("u", "dt", "a", "b", "c", "d", "z", "dt_bias", "h_in")
    g = torch.Generator().manual_seed(92)
    mag = so.scan_grad(*[base[k] for k in ("u", "dt", "a", "b", "c", "dy", "d", "z", "dt_bias", "h_in", "dh_out")],
                       mag=True)
    for k, name in names.items():
        v = torch.randn(base[k].shape, generator=g, dtype=F64)

        def f(x):
            y, h, _ = so.scan(*[x if q == k else base[q] for q in order])
            return (y * base["dy"]).sum() + (h * base["dh_out"]).sum()

        have = float((got[name].cpu().to(F64) * v).sum())
        want = _along(f, base[k], v, 1e-5)
        assert abs(have - want) <= 4000 * so.EPS32 * float((mag[name] * v.abs()).sum()) + 1e-6 * max(1.0, abs(want)), \
            (name, have, want)


# ------------------------------------------------ streams, graphs, repeats

def _everything(seed):
    """One call of each operator each way on fresh buffers; returns (function that launches them, outputs)."""
    g = torch.Generator().manual_seed(seed)
    n, t, c, s, k = 2, 150, 72, 16, 4
    i = {q: dev(v) for q, v in scan_inputs(n, t, c, s, 2, BF, True, "dzbh", seed).items()}
    w, b = dev(rn(g, k, c, dtype=BF)), dev(rn(g, c, dtype=BF))
    cp = cc3d.causal_conv1d_plan(cc3d.make_conv1d_desc(n, t, c, k, act="silu"))
    sp = cc3d.selective_scan_plan(cc3d.make_scan_desc(n, t, c, s, groups=2))
    jp = cc3d.norm_join_plan(cc3d.make_join_desc(n * t, c, gate_rows=t, gate_act="silu"))
    gate, one = dev(rn(g, n, c, dtype=BF)), dev(rn(g, c, dtype=BF))
    o = dict(xc=nan(n, t, c, dtype=BF), y=nan(n, t, c, dtype=BF), h=nan(n, c, s), xo=nan(n, t, c, dtype=BF),
             ho=nan(n, t, c, dtype=BF), dx=nan(n, t, c, dtype=BF), dw=nan(k, c), db_=nan(c),
             du=nan(n, t, c, dtype=BF), ddt=nan(n, t, c, dtype=BF), da=nan(c, s), db=nan(n, t, 2, s, dtype=BF),
             dc=nan(n, t, 2, s, dtype=BF), dgate=nan(n, c, dtype=BF), dscale=nan(c), dres=nan(n, t, c, dtype=BF),
             dyj=nan(n, t, c, dtype=BF))
    ws = [space(cp, True), space(sp), space(sp, True), space(jp, True)]

    def launch(stream=None):
        cc3d.causal_conv1d_forward(cp, i["u"], w, b, o["xc"], stream=stream)
        cc3d.selective_scan_forward(sp, o["xc"], i["dt"], i["a"], i["b"], i["c"], o["y"], z=i["z"], d=i["d"],
                                    dt_bias=i["dt_bias"], h_in=i["h_in"], h_out=o["h"], workspace=ws[1], stream=stream)
        cc3d.norm_join_forward(jp, o["y"], i["u"], x_out=o["xo"], h_out=o["ho"], gate=gate, scale=one, stream=stream)
        cc3d.norm_join_backward(jp, o["y"], i["u"], dx_out=i["dy"], dh=o["ho"], gate=gate, scale=one, dgate=o["dgate"],
                                dscale=o["dscale"], dresidual=o["dres"], dy=o["dyj"], workspace=ws[3], stream=stream)
        cc3d.selective_scan_backward(sp, o["xc"], i["dt"], i["a"], i["b"], i["c"], o["dyj"], z=i["z"], d=i["d"],
                                     dt_bias=i["dt_bias"], h_in=i["h_in"], du=o["du"], ddt=o["ddt"], da=o["da"],
                                     db=o["db"], dc=o["dc"], workspace=ws[2], stream=stream)
        cc3d.causal_conv1d_backward(cp, i["u"], w, b, o["du"], dx=o["dx"], dw=o["dw"], db=o["db_"], workspace=ws[0],
                                    stream=stream)

    return launch, o, i


def test_repeated_calls_and_another_stream_give_the_same_bits(cuda_device):
    launch, o, _ = _everything(55)
    launch()
    torch.cuda.synchronize()
    first = {k: v.clone() for k, v in o.items()}
    assert all(bool(torch.isfinite(v.float()).all()) for v in first.values())
    side = torch.cuda.Stream()
    for stream in (None, side, side):
        for v in o.values():
            v.fill_(NAN)
        torch.cuda.synchronize()
        launch(stream)
        torch.cuda.synchronize()
        for k, v in o.items():
            assert torch.equal(v, first[k]), k


def test_a_replayed_graph_equals_eager_calls(cuda_device):
    launch, o, i = _everything(56)
    launch()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        launch()
    for step in range(3):
        i["u"].mul_(0.9)
        for v in o.values():
            v.fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        replayed = {k: v.clone() for k, v in o.items()}
        for v in o.values():
            v.fill_(NAN)
        launch()
        torch.cuda.synchronize()
        for k, v in o.items():
            assert torch.equal(v, replayed[k]), (step, k)


def test_offsets_past_32_bits(cuda_device):
    """Rows more than 2**31 elements apart: the last sequence of a strided view of a 6 GiB buffer."""
    n, t, c, k, s = 2, 3, 16, 4, 4
    g = torch.Generator().manual_seed(61)
    big = torch.empty(3 * (1 << 30), dtype=BF, device=DEV)
    step = big.numel() - 4 * c * t

    def far(x):
        v = big.as_strided((n, t, c), (step, c, 1), 0)
        v.copy_(x)
        return v

    x, w = rn(g, n, t, c, dtype=BF), rn(g, k, c, dtype=BF)
    plan = cc3d.causal_conv1d_plan(cc3d.make_conv1d_desc(n, t, c, k))
    y = nan(n, t, c, dtype=BF)
    cc3d.causal_conv1d_forward(plan, far(x), dev(w), None, y)
    a = (d64(x), d64(w), None, False)
    so.assert_close(y, so.conv1d(*a)[0], so.conv1d(*a, mag=True)[0], 2 * (k + 2) + 32, "y")
    i = scan_inputs(n, t, c, s, 1, BF, True, "h", 62)
    sp = cc3d.selective_scan_plan(cc3d.make_scan_desc(n, t, c, s))
    cc3d.selective_scan_forward(sp, far(i["u"]), *[dev(i[q]) for q in ("dt", "a", "b", "c")], y, h_in=dev(i["h_in"]))
    so_ = [d64(i[q]) for q in ("u", "dt", "a", "b", "c")] + [None, None, None, d64(i["h_in"])]
    so.assert_close(y, so.scan(*so_)[0], so.scan(*so_, mag=True)[0], 4 * t + 2 * s + 640, "scan y")
    rows = big.as_strided((2, c), (step, 1), 0)
    rows.copy_(x[:, 0])
    jp = cc3d.norm_join_plan(cc3d.make_join_desc(2, c, post="rms", pre=None))
    xo = nan(2, c, dtype=BF)
    cc3d.norm_join_forward(jp, rows, dev(x[:, 1]), x_out=xo)
    ref, _, (m, _) = so.join(d64(x[:, 0]), d64(x[:, 1]), post="rms", pre=None, act=False, eps=1e-6)
    so.assert_close(xo, ref, m, 256, "x_out")
