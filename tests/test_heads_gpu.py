"""linear_attention, rotary and group_norm on the GPU against their plain
64-bit forms (heads_oracle), forward and backward: every type, odd sizes,
shared heads, strided views, lengths of zero and one, absent optional tensors,
NaN in the tokens after a sequence's valid ones and around the outputs.

Bounds.  Linear attention (heads_oracle.linear_bound): a term's roundings of
2^-24 are linear_depth; with bf16 tensors the products of q and k, and the
state that meets q, are rounded to bf16 once (half a step: 2^-8 of the terms);
states and the decay's gradient are not.  The backward depth is twice the
forward one, and sums over shared heads and sequences add their number.
Rotary: an angle is rounded to a half turn's 2^-25, 3.2 of which move a sine by
as much, sine and cosine and their factor by some units more, two products and
a sum: 16 roundings of the pair's terms.
Group norm: units (heads_oracle.group) of 2^-24, times the roundings of a sum:
a thread's rows one after another, then trees: 64 + rows.
"""
import pytest
import torch

import causal_conv3d_video_amd as cc3d
import heads_oracle as ho
from test_seq_gpu import NAN, dev, lengths_of, nan, rn, space

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F64 = torch.float64
BF, F32 = torch.bfloat16, torch.float32


def d64(t):
    return None if t is None else t.to(F64)


def poison(x, lengths):
    x = x.clone()
    for i, ln in enumerate(lengths or []):
        x[i, max(ln, 0):] = NAN
    return x


class Wide:
    """A view of the given shape inside a larger NaN-filled buffer, with `pad`
    elements before and after every token and a spare token; ``untouched``
    says that nothing around the view was written."""

    def __init__(self, shape, dtype, pad, fill=None):
        n, t, rest = shape[0], shape[1], shape[2:]
        c = 1
        for s in rest:
            c *= s
        self.buf = torch.full((n, t + 1, c + 2 * pad), NAN, dtype=dtype, device=DEV)
        self.inner = self.buf[:, :t, pad:pad + c]
        self.v = self.inner.unflatten(-1, rest) if len(rest) > 1 else self.inner
        if fill is not None:
            self.v.copy_(fill)

    def untouched(self):
        b = self.buf.clone()
        n, t, c = self.inner.shape
        pad = (b.shape[2] - c) // 2
        b[:, :t, pad:pad + c] = NAN
        return bool(torch.isnan(b).all())


def near(got, want, bound, what):
    got, want, bound = got.detach().to(F64).cpu(), want.detach(), bound.detach()
    assert bool(torch.isfinite(got).all()), what
    over = (got - want).abs() - bound
    at = int(over.argmax())
    assert float(over.max()) <= 0, "%s: off by %.3e, allowed %.3e (value %.3e), at %d of %s" % (
        what, float((got - want).abs().reshape(-1)[at]), float(bound.reshape(-1)[at]), float(want.reshape(-1)[at]), at,
        tuple(want.shape))


# ------------------------------------------------------ linear attention

LINEAR = [
    # n, t, heads, (q, k, v heads), dk, dv, dtype, ragged, pad, state, decay
    (1, 1, 1, (1, 1, 1), 1, 1, F32, 0, 0, True, "some"),
    (3, 1, 4, (4, 4, 4), 64, 64, BF, 0, 8, True, "some"),
    (5, 1, 6, (2, 2, 6), 50, 100, BF, 1, 3, True, "some"),
    (2, 1, 3, (3, 1, 1), 128, 256, F32, 1, 0, False, None),
    (2, 1, 2, (2, 2, 2), 7, 3, F32, 0, 1, True, "none and all"),
    (1, 2, 2, (2, 2, 2), 16, 16, BF, 0, 0, True, "some"),
    (2, 3, 1, (1, 1, 1), 5, 9, F32, 0, 1, True, "some"),
    (4, 17, 3, (3, 3, 3), 64, 64, BF, 1, 8, True, "some"),
    (4, 63, 2, (2, 2, 2), 33, 65, F32, 1, 0, True, "some"),
    (2, 64, 4, (2, 2, 4), 64, 128, BF, 0, 0, False, "some"),
    (2, 65, 4, (4, 2, 2), 128, 64, BF, 0, 8, True, "none and all"),
    (4, 130, 3, (1, 1, 3), 100, 50, BF, 1, 5, True, "some"),
    (4, 200, 2, (2, 1, 1), 40, 24, F32, 1, 4, True, "some"),
    (1, 129, 1, (1, 1, 1), 256, 256, BF, 0, 0, True, "some"),
    (1, 130, 1, (1, 1, 1), 130, 200, F32, 0, 0, True, "some"),
    (2, 300, 2, (2, 2, 2), 64, 64, F32, 0, 0, True, None),
    (1, 515, 5, (5, 1, 1), 50, 100, F32, 0, 2, True, "some"),
    (3, 700, 2, (1, 2, 2), 128, 128, BF, 1, 0, True, "some"),
    (2, 130, 2, (2, 1, 2), 128, 128, F32, 1, 0, True, "some"),
    (1, 90, 3, (3, 3, 3), 70, 125, F32, 0, 1, True, "some"),
    (2, 100, 2, (2, 2, 1), 256, 40, F32, 1, 0, True, "some"),
    (2, 90, 1, (1, 1, 1), 200, 100, BF, 1, 0, True, "some"),
    (33, 70, 8, (2, 8, 8), 128, 128, BF, 1, 0, True, "some"),  # more heads than compute units
]


def linear_case(case, seed):
    n, t, h, shared, dk, dv, dtype, ragged, pad, state, decay = case
    g = torch.Generator().manual_seed(seed)
    ln = lengths_of(ragged, n, t)
    i = {"q": rn(g, n, t, shared[0], dk, dtype=dtype), "k": rn(g, n, t, shared[1], dk, dtype=dtype),
         "v": rn(g, n, t, shared[2], dv, dtype=dtype), "do": rn(g, n, t, h, dv, dtype=dtype)}
    i["h_in"] = rn(g, n, h, dk, dv, scale=0.3) if state else None
    i["dh_out"] = rn(g, n, h, dk, dv, scale=0.3) if state else None
    i["log_decay"] = None
    if decay:
        i["log_decay"] = torch.log1p(-torch.exp2(-1.0 - 7.0 * torch.arange(h, dtype=F64) / max(1, h - 1))).float()
    if decay == "none and all":
        i["log_decay"][0] = 0.0
        i["log_decay"][-1] = float("-inf")
    plan = cc3d.linear_attention_plan(cc3d.make_linear_attention_desc(n, t, h, dk, dv, *shared, dtype=dtype))
    dec = torch.zeros(h, dtype=F64) if i["log_decay"] is None else d64(i["log_decay"])
    return i, ln, plan, dec, float(plan.desc.scale)


def views(i, names, ln, dtype, pad):
    return {x: Wide(i[x].shape, dtype, pad, dev(poison(i[x], ln))).v for x in names}


@pytest.mark.parametrize("case", LINEAR, ids=lambda c: "-".join(map(str, c)).replace("torch.", ""))
def test_linear_forward(cuda_device, case):
    n, t, h, shared, dk, dv, dtype, ragged, pad, state, decay = case
    i, ln, plan, dec, scale = linear_case(case, 11)
    args = [d64(i[x]) for x in ("q", "k", "v")] + [dec, scale, d64(i["h_in"]), ln, h]
    want, last = ho.linear(*args)
    mag, mag_last = ho.linear(*args, mag=True)
    v = views(i, ("q", "k", "v"), ln, dtype, pad)
    o = Wide((n, t, h, dv), dtype, pad)
    h_out = nan(n, h, dk, dv)
    lengths = None if ln is None else torch.tensor(ln, dtype=torch.int32, device=DEV)
    cc3d.linear_attention_forward(plan, v["q"], v["k"], v["v"], o.v, log_decay=dev(i["log_decay"]), h_in=dev(i["h_in"]),
                                  h_out=h_out, lengths=lengths, workspace=space(plan))
    torch.cuda.synchronize()
    depth, bf = ho.linear_depth(t, dk, dv), dtype == BF
    near(o.v, want, ho.linear_bound(mag, want, dtype, depth, 2.0 ** -8 if bf and t > 1 else 0.0), "o")
    near(h_out, last, ho.linear_bound(mag_last, last, F32, depth, 0.0), "h_out")
    assert o.untouched()
    for k, m in enumerate(ln or []):
        assert not o.v[k, max(m, 0):].any()


@pytest.mark.parametrize("case", LINEAR, ids=lambda c: "-".join(map(str, c)).replace("torch.", ""))
def test_linear_backward(cuda_device, case):
    n, t, h, shared, dk, dv, dtype, ragged, pad, state, decay = case
    i, ln, plan, dec, scale = linear_case(case, 12)
    args = [d64(i[x]) for x in ("q", "k", "v")] + [dec, scale] + [d64(i[x]) for x in ("do", "h_in", "dh_out")] + [ln, h]
    want, mag = ho.linear_grad(*args), ho.linear_grad(*args, mag=True)
    v = views(i, ("q", "k", "v", "do"), ln, dtype, pad)
    o = {x: Wide(i[x[1:]].shape, dtype, pad) for x in ("dq", "dk", "dv")}
    dh_in, dlog = nan(n, h, dk, dv), nan(h)
    lengths = None if ln is None else torch.tensor(ln, dtype=torch.int32, device=DEV)
    cc3d.linear_attention_backward(
        plan, v["q"], v["k"], v["v"], v["do"], log_decay=dev(i["log_decay"]), h_in=dev(i["h_in"]), dh_out=dev(i["dh_out"]),
        dq=o["dq"].v, dk=o["dk"].v, dv=o["dv"].v, dlog_decay=dlog if decay else None, dh_in=dh_in, lengths=lengths,
        workspace=space(plan, True))
    torch.cuda.synchronize()
    depth, bf = 2 * ho.linear_depth(t, dk, dv) + h, dtype == BF
    for x in ("dq", "dk", "dv"):
        near(o[x].v, want[x], ho.linear_bound(mag[x], want[x], dtype, depth, 2.0 ** -8 if bf else 0.0), x)
        assert o[x].untouched(), x
        for k, m in enumerate(ln or []):
            assert not o[x].v[k, max(m, 0):].any(), x
    near(dh_in, want["dh_in"], ho.linear_bound(mag["dh_in"], want["dh_in"], F32, depth, 0.0), "dh_in")
    if decay:
        near(dlog, want["dlog_decay"], ho.linear_bound(mag["dlog_decay"], want["dlog_decay"], F32, depth + n * t, 0.0), "dlog_decay")


# ---------------------------------------------------------------- rotary

ROTARY = [
    # n, t, q heads, k heads, d, rot, first, layout, dtype, ragged, pad, settings
    (1, 1, 1, 0, 2, 2, 0, "half", F32, 0, 0, {}),
    (64, 1, 12, 12, 64, 64, 0, "half", BF, 0, 8, {}),
    (3, 7, 4, 1, 128, 128, 0, "interleaved", BF, 1, 8, dict(scaling="parts", factor=16.0, original=4096)),
    (2, 33, 3, 3, 100, 50, 10, "half", F32, 1, 3, dict(scaling="linear", factor=4.0)),
    (2, 9, 5, 2, 48, 16, 24, "interleaved", BF, 0, 0, dict(scaling="base", factor=8.0)),
    (4, 40, 2, 2, 96, 32, 32, "half", F32, 1, 4, {}),
    (2, 300, 16, 4, 64, 64, 0, "interleaved", F32, 0, 0, dict(theta=500000.0)),
    (5, 3, 1, 1, 7, 4, 3, "interleaved", BF, 1, 1, dict(amplitude=1.5)),
    (2, 5, 3, 0, 256, 256, 0, "half", BF, 0, 0, {}),
    (2, 5, 3, 1, 300, 256, 40, "half", F32, 0, 0, {}),
]


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("where", ["start", "far", "given"])
@pytest.mark.parametrize("case", ROTARY, ids=lambda c: "-".join(map(str, c[:11])).replace("torch.", ""))
def test_rotary(cuda_device, case, where, back):
    n, t, hq, hk, d, rot, first, layout, dtype, ragged, pad, kw = case
    g = torch.Generator().manual_seed(21)
    ln = lengths_of(ragged, n, t)
    x = {"q": rn(g, n, t, hq, d, dtype=dtype), "k": rn(g, n, t, max(hk, 1), d, dtype=dtype)}
    off, pos = None, None
    if where == "far":
        off = torch.randint(-5, 1 << 30, (n,), generator=g, dtype=torch.int32)
        off[0] = 2 ** 31 - 1  # positions of further tokens pass 32 bits
    if where == "given":
        pos = torch.randint(-100, 200000, (n, t), generator=g, dtype=torch.int32)
    at = pos.long() if pos is not None else torch.arange(t)[None] + (0 if off is None else off.long()[:, None]) + torch.zeros(
        n, 1, dtype=torch.long)
    desc = cc3d.make_rotary_desc(n, t, hq, hk, d, rot=rot, first=first, layout=layout, dtype=dtype, **kw)
    plan = cc3d.rotary_plan(desc)
    f = ho.frequencies(rot, **{k: v for k, v in kw.items() if k != "amplitude"})
    v = {k: Wide(u.shape, dtype, pad, dev(poison(u, ln))).v for k, u in x.items()}
    o = {k: Wide(u.shape, dtype, pad) for k, u in x.items()}
    lengths = None if ln is None else torch.tensor(ln, dtype=torch.int32, device=DEV)
    call = cc3d.rotary_backward if back else cc3d.rotary_forward
    call(plan, v["q"], v["k"] if hk else None, o["q"].v, o["k"].v if hk else None, positions=dev(pos), offsets=dev(off),
         lengths=lengths)
    torch.cuda.synchronize()
    for k in ("q", "k")[:1 + (hk > 0)]:
        args = (d64(x[k]), at, f, first, layout, desc.amplitude)
        want = ho.rotary(*args, back=back, lengths=ln)
        mag = ho.rotary(*args, lengths=ln, mag=True)
        # an angle of up to 2^31 positions holds 2^-53 of its turns: 2^31 2^-53 2 pi 2 = 6e-6
        far = 6e-6 if where == "far" else 0.0
        near(o[k].v, want, (16 * ho.EPS32 + far) * mag + ho.HALF_STEP[dtype] * want.abs(), k)
        assert o[k].untouched()
        same = [c for c in range(d) if not first <= c < first + rot]
        for i, m in enumerate(ho.lens(ln, n, t)):
            assert torch.equal(o[k].v[i, :m][..., same].cpu(), x[k][i, :m][..., same])
            assert not o[k].v[i, m:].any()
        if not hk:
            break


# ------------------------------------------------------------ group norm

GROUP = [
    # n, p, c, groups, act, dtype, ragged, pad, weight, bias
    (1, 1, 8, 1, "silu", F32, 0, 0, True, True),
    (64, 1, 768, 12, None, BF, 0, 8, True, True),
    (1030, 1, 192, 3, "silu", BF, 0, 0, True, False),
    (9, 2, 24, 3, "silu", F32, 1, 8, False, True),
    (7, 4, 2048, 16, None, BF, 1, 0, True, True),
    (5, 30, 192, 32, "silu", BF, 1, 8, True, True),
    (3, 33, 192, 32, "silu", BF, 1, 0, True, True),
    (4, 20, 37, 37, None, F32, 1, 3, True, True),
    (4, 300, 37, 1, "silu", F32, 1, 3, True, True),
    (2, 1000, 5, 5, "silu", F32, 1, 1, True, True),
    (3, 1560, 515, 5, "silu", F32, 1, 0, True, True),
    (2, 2000, 384, 32, "silu", BF, 0, 8, True, True),
    (3, 777, 256, 4, None, BF, 1, 0, False, False),
    (2, 17, 8192, 8, "silu", BF, 1, 0, True, True),
    (2, 3, 8188, 4, None, F32, 0, 0, True, True),
    (2, 40, 4096, 4096, "silu", F32, 0, 0, True, True),
    (1, 20000, 96, 8, "silu", BF, 0, 0, True, True),
    (6, 9, 3, 1, None, F32, 1, 2, True, True),
    (2, 2000, 7, 7, "silu", BF, 1, 0, True, True),
]
EPS = 1e-5


def group_case(case, seed):
    n, p, c, groups, act, dtype, ragged, pad, weight, bias = case
    g = torch.Generator().manual_seed(seed)
    ln = lengths_of(ragged, n, p)
    i = {"x": rn(g, n, p, c, dtype=dtype, scale=1.5, mean=0.5), "dy": rn(g, n, p, c, dtype=dtype),
         "w": rn(g, c, dtype=dtype, scale=0.2, mean=1.0) if weight else None,
         "b": rn(g, c, dtype=dtype, scale=0.2) if bias else None}
    plan = cc3d.group_norm_plan(cc3d.make_group_norm_desc(n, p, c, groups, act=act, eps=EPS, dtype=dtype))
    lengths = None if ln is None else torch.tensor(ln, dtype=torch.int32, device=DEV)
    return i, ln, plan, lengths


def group_near(got, want, unit, dtype, rows, what):
    b = (64 + rows) * ho.EPS32 * unit
    near(got, want, b + ho.HALF_STEP[dtype] * (want.abs() + b), what)


@pytest.mark.parametrize("case", GROUP, ids=lambda c: "-".join(map(str, c)).replace("torch.", ""))
def test_group_forward(cuda_device, case):
    n, p, c, groups, act, dtype, ragged, pad, weight, bias = case
    i, ln, plan, lengths = group_case(case, 31)
    want = ho.group(d64(i["x"]), groups, d64(i["w"]), d64(i["b"]), bool(act), EPS, ln)
    x, y = Wide((n, p, c), dtype, pad, dev(poison(i["x"], ln))), Wide((n, p, c), dtype, pad)
    stats = nan(n, groups, 2)
    for st in (stats, None):
        y.v.fill_(NAN)
        cc3d.group_norm_forward(plan, x.v, y.v, w=dev(i["w"]), b=dev(i["b"]), stats=st, lengths=lengths, workspace=space(plan))
        torch.cuda.synchronize()
        group_near(y.v, want["y"], want["y_unit"], dtype, p, "y")
        assert y.untouched()
    group_near(stats, want["stats"], want["stats_unit"], F32, p, "stats")
    for k, m in enumerate(ln or []):
        assert not y.v[k, max(m, 0):].any()


@pytest.mark.parametrize("case", GROUP, ids=lambda c: "-".join(map(str, c)).replace("torch.", ""))
def test_group_backward(cuda_device, case):
    n, p, c, groups, act, dtype, ragged, pad, weight, bias = case
    i, ln, plan, lengths = group_case(case, 32)
    want = ho.group(d64(i["x"]), groups, d64(i["w"]), d64(i["b"]), bool(act), EPS, ln, d64(i["dy"]))
    stats = ho.group(d64(i["x"]), groups, None, None, False, EPS, ln)["stats"].float()
    x, dy = (Wide((n, p, c), dtype, pad, dev(poison(i[k], ln))) for k in ("x", "dy"))
    for st in (dev(stats), None):
        dx, dw, db = Wide((n, p, c), dtype, pad), nan(c), nan(c)
        cc3d.group_norm_backward(plan, x.v, dy.v, w=dev(i["w"]), b=dev(i["b"]), stats=st, dx=dx.v, dw=dw if weight else None,
                                 db=db if bias else None, lengths=lengths, workspace=space(plan, True))
        torch.cuda.synchronize()
        group_near(dx.v, want["dx"], want["dx_unit"], dtype, p, "dx")
        assert dx.untouched()
        if weight:
            group_near(dw, want["dw"], want["dw_unit"], F32, p + n, "dw")
        if bias:
            group_near(db, want["db"], want["db_unit"], F32, p + n, "db")
    for k, m in enumerate(ln or []):
        assert not dx.v[k, max(m, 0):].any()
