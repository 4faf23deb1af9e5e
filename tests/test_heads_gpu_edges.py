"""linear_attention, rotary and group_norm at their edges: results left out,
infinities and NaN beside values that they do not reach, states in place,
streamed calls, repeated and replayed calls, another stream, offsets past 32
bits, far means, and the three one after another."""
import pytest
import torch

import causal_conv3d_video_amd as cc3d
import heads_oracle as ho
from test_heads_gpu import BF, DEV, EPS, F32, F64, Wide, d64, group_near, near
from test_seq_gpu import NAN, dev, nan, rn, space

pytestmark = pytest.mark.gpu
INF = float("inf")


def bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == BF else torch.int32)


def same(a, b, what=""):
    assert torch.equal(bits(a), bits(b)), what


class Linear:
    """A case of one call with everything in it, on the GPU."""

    def __init__(self, n, t, h, dk, dv, dtype=BF, shared=None, seed=5, ragged=None, **kw):
        shared = shared or (h, h, h)
        g = torch.Generator().manual_seed(seed)
        self.plan = cc3d.linear_attention_plan(cc3d.make_linear_attention_desc(n, t, h, dk, dv, *shared, dtype=dtype, **kw))
        self.i = {"q": rn(g, n, t, shared[0], dk, dtype=dtype), "k": rn(g, n, t, shared[1], dk, dtype=dtype),
                  "v": rn(g, n, t, shared[2], dv, dtype=dtype), "do": rn(g, n, t, h, dv, dtype=dtype),
                  "h_in": rn(g, n, h, dk, dv, scale=0.3), "dh_out": rn(g, n, h, dk, dv, scale=0.3),
                  "log_decay": -torch.rand(h, generator=g) * 0.2}
        self.i = {k: dev(v) for k, v in self.i.items()}
        self.lengths = None if ragged is None else torch.tensor(ragged, dtype=torch.int32, device=DEV)
        self.shape, self.dtype = (n, t, h, dk, dv), dtype
        self.space, self.back_space = space(self.plan), space(self.plan, True)

    def forward(self, stream=None, **over):
        i = {**self.i, **over}
        n, t, h, dk, dv = self.shape
        o, h_out = nan(n, t, h, dv, dtype=self.dtype), nan(n, h, dk, dv)
        cc3d.linear_attention_forward(self.plan, i["q"], i["k"], i["v"], o, log_decay=i["log_decay"], h_in=i["h_in"],
                                      h_out=h_out, lengths=self.lengths, workspace=self.space, stream=stream)
        return {"o": o, "h_out": h_out}

    def backward(self, ask=("dq", "dk", "dv", "dlog_decay", "dh_in"), stream=None, **over):
        i = {**self.i, **over}
        out = {x: nan(*self.i[x[1:]].shape, dtype=self.i[x[1:]].dtype) for x in ask}
        cc3d.linear_attention_backward(self.plan, i["q"], i["k"], i["v"], i["do"], log_decay=i["log_decay"], h_in=i["h_in"],
                                       dh_out=i["dh_out"], lengths=self.lengths, workspace=self.back_space, stream=stream, **out)
        return out


@pytest.mark.parametrize("shared", [None, (1, 2, 2)])
@pytest.mark.parametrize("t", [1, 70, 400])
def test_gradients_left_out(cuda_device, t, shared):
    c = Linear(2, t, 2, 24, 40, shared=shared)
    full = c.backward()
    for ask in (("dq",), ("dk",), ("dv",), ("dh_in",), ("dlog_decay",), ("dq", "dh_in"), ("dlog_decay", "dv"), ("dk", "dlog_decay")):
        got = c.backward(ask)
        torch.cuda.synchronize()
        for k, v in got.items():
            assert bool(torch.isfinite(v).all()), (ask, k)
            # (with the decay's gradient dq and dk are taken from the state in more bits)
            if "dlog_decay" in ask or k in ("dv", "dh_in"):
                same(v, full[k], (ask, k))
            else:
                assert float((v - full[k]).abs().max()) <= 2.0 ** -6 * float(full[k].abs().max()), (ask, k)
    for missing in ("h_in", "dh_out"):
        got = c.backward(**{missing: None})
        want = c.backward(**{missing: torch.zeros_like(c.i[missing])})
        torch.cuda.synchronize()
        for k in got:
            same(got[k], want[k], (missing, k))
    assert cc3d.linear_attention_forward(c.plan, c.i["q"], c.i["k"], c.i["v"], nan(2, t, 2, 40, dtype=BF),
                                         workspace=c.space) is None


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("t,at", [(1, 0), (20, 7), (100, 37), (130, 64), (300, 299)])
@pytest.mark.parametrize("what", ["q", "k", "v"])
def test_values_that_are_no_numbers_reach_no_earlier_token(cuda_device, t, at, what, dtype):
    """An infinity and a NaN in one token of one head: earlier tokens, other heads and other sequences keep their bits, its
    own results and (of k and v) later ones are no numbers where the formula says so."""
    c = Linear(2, t, 2, 24, 40, dtype=dtype)
    clean = c.forward()
    for bad in (INF, NAN):
        x = c.i[what].clone()
        x[1, at, 0, 3] = bad
        got = c.forward(**{what: x})
        torch.cuda.synchronize()
        same(got["o"][0], clean["o"][0])
        same(got["o"][1, :, 1], clean["o"][1, :, 1])
        same(got["o"][1, :at], clean["o"][1, :at])
        same(got["h_out"][0], clean["h_out"][0])
        same(got["h_out"][1, 1], clean["h_out"][1, 1])
        if what == "q":
            same(got["h_out"], clean["h_out"])
            same(got["o"][1, at + 1:], clean["o"][1, at + 1:])
            assert not bool(torch.isfinite(got["o"][1, at, 0]).any())
        elif what == "v":  # one column of the state
            assert not bool(torch.isfinite(got["o"][1, at:, 0, 3]).any())
            assert bool(torch.isfinite(got["o"][1, :, 0, 4:]).all())
            same(got["h_out"][1, 0, :, 4:], clean["h_out"][1, 0, :, 4:])
        else:              # one row of it, that every column meets
            assert not bool(torch.isfinite(got["o"][1, at:, 0]).any())
            same(got["h_out"][1, 0, 4:], clean["h_out"][1, 0, 4:])
            assert not bool(torch.isfinite(got["h_out"][1, 0, 3]).any())


@pytest.mark.parametrize("t,at", [(20, 7), (100, 37), (130, 64), (300, 1)])
def test_values_that_are_no_numbers_in_the_backward_pass(cuda_device, t, at):
    """do of one token is met by dk and dv of it and earlier tokens, v and k by dq of it and later ones."""
    ask = ("dq", "dk", "dv")
    c = Linear(1, t, 2, 24, 40)
    clean = c.backward(ask)
    for bad in (INF, NAN):
        do = c.i["do"].clone()
        do[0, at, 0, 3] = bad
        got = c.backward(ask, do=do)
        torch.cuda.synchronize()
        for x in ("dk", "dv"):
            same(got[x][0, at + 1:], clean[x][0, at + 1:], x)
            same(got[x][0, :, 1], clean[x][0, :, 1], x)
        rest = [p for p in range(t) if p != at]
        same(got["dq"][0, rest], clean["dq"][0, rest])
        for what in ("k", "v"):
            x = c.i[what].clone()
            x[0, at, 0, 3] = bad
            got = c.backward(ask, **{what: x})
            torch.cuda.synchronize()
            same(got["dq"][0, :at], clean["dq"][0, :at])
            same(got["dq"][0, :, 1], clean["dq"][0, :, 1])


@pytest.mark.parametrize("t", [1, 20, 90, 2000])
def test_state_in_place(cuda_device, t):
    c = Linear(2, t, 2, 64, 64)
    want = c.forward()
    state, o = c.i["h_in"].clone(), torch.empty_like(want["o"])
    cc3d.linear_attention_forward(c.plan, c.i["q"], c.i["k"], c.i["v"], o, log_decay=c.i["log_decay"], h_in=state, h_out=state,
                                  workspace=c.space)
    torch.cuda.synchronize()
    same(o, want["o"])
    same(state, want["h_out"])


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (50, 40)])
@pytest.mark.parametrize("ragged", [[1, 2900, 65, 0], [3000, 64, 130, 1]])
def test_state_in_place_of_short_sequences_in_a_long_call(cuda_device, ragged, dk, dv):
    """The time axis is split, and its last parts have no tokens: their state goes where the first part's came from."""
    c = Linear(4, 3000, 4, dk, dv, ragged=ragged)
    assert c.plan.info["chunks"] > 3
    want = c.forward()
    for _ in range(5):
        state, o = c.i["h_in"].clone(), nan(4, 3000, 4, dv, dtype=BF)
        cc3d.linear_attention_forward(c.plan, c.i["q"], c.i["k"], c.i["v"], o, log_decay=c.i["log_decay"], h_in=state, h_out=state,
                                      lengths=c.lengths, workspace=c.space)
        torch.cuda.synchronize()
        same(o, want["o"])
        same(state, want["h_out"])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_one_buffer_holds_q_k_and_v(cuda_device, dtype):
    """q, k and v as parts of one projection's rows, rotary in place there, and their gradients as parts of another."""
    n, t, h, d = 2, 150, 4, 32
    c = Linear(n, t, h, d, d, dtype=dtype)
    plan = cc3d.rotary_plan(cc3d.make_rotary_desc(n, t, h, h, d, dtype=dtype))
    qo, ko = nan(n, t, h, d, dtype=dtype), nan(n, t, h, d, dtype=dtype)
    cc3d.rotary_forward(plan, c.i["q"], c.i["k"], qo, ko)
    want, back = c.forward(q=qo, k=ko), c.backward(q=qo, k=ko)
    rows = torch.cat([c.i[x].reshape(n, t, h * d) for x in ("q", "k", "v")], 2)
    q, k, v = (rows[..., h * d * i:h * d * (i + 1)] for i in range(3))
    cc3d.rotary_forward(plan, q, k, q, k)
    got = c.forward(q=q, k=k, v=v)
    grads = nan(n, t, 3 * h * d, dtype=dtype)
    dq, dk, dv = (grads[..., h * d * i:h * d * (i + 1)] for i in range(3))
    dlog, dh = nan(h), nan(n, h, d, d)
    cc3d.linear_attention_backward(c.plan, q, k, v, c.i["do"], log_decay=c.i["log_decay"], h_in=c.i["h_in"], dh_out=c.i["dh_out"],
                                   dq=dq, dk=dk, dv=dv, dlog_decay=dlog, dh_in=dh, workspace=c.back_space)
    torch.cuda.synchronize()
    for x in ("o", "h_out"):
        same(got[x], want[x], x)
    for x, g in (("dq", dq), ("dk", dk), ("dv", dv)):
        same(g.unflatten(-1, (h, d)), back[x], x)
    same(dlog, back["dlog_decay"])
    same(dh, back["dh_in"])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_streamed_chunks_follow_one_call(cuda_device, dtype):
    """Chunks of 1, 5, 64, 130 and 1 tokens against one call over 201: each is within its own bound of the 64-bit form."""
    sizes = [1, 5, 64, 130, 1]
    t = sum(sizes)
    c = Linear(2, t, 3, 40, 24, dtype=dtype)
    i = c.i
    args = [d64(i[x].cpu()) for x in ("q", "k", "v", "log_decay")] + [float(c.plan.desc.scale), d64(i["h_in"].cpu()), None, 3]
    want, last = ho.linear(*args)
    mag, mag_last = ho.linear(*args, mag=True)
    state, parts, at = i["h_in"].clone(), [], 0
    for m in sizes:
        plan = cc3d.linear_attention_plan(cc3d.make_linear_attention_desc(2, m, 3, 40, 24, dtype=dtype))
        q, k, v = (i[x][:, at:at + m] for x in ("q", "k", "v"))
        o = nan(2, m, 3, 24, dtype=dtype)
        cc3d.linear_attention_forward(plan, q, k, v, o, log_decay=i["log_decay"], h_in=state, h_out=state, workspace=space(plan))
        parts.append(o)
        at += m
    torch.cuda.synchronize()
    depth, bf = ho.linear_depth(t, 40, 24) + 8 * len(sizes), dtype == BF
    near(torch.cat(parts, 1), want, ho.linear_bound(mag, want, dtype, depth, 2.0 ** -8 if bf else 0.0), "o")
    near(state, last, ho.linear_bound(mag_last, last, F32, depth, 2.0 ** -16 if bf else 0.0), "state")


def everything(seed):
    """Calls of every operator with its workspaces, as one function, and its outputs."""
    c = Linear(2, 333, 4, 64, 64, shared=(2, 2, 4), seed=seed, ragged=[333, 100])
    short = Linear(3, 9, 2, 64, 128, seed=seed + 1)
    g = torch.Generator().manual_seed(seed + 2)
    x, dy = dev(rn(g, 3, 900, 192, dtype=BF)), dev(rn(g, 3, 900, 192, dtype=BF))
    w, b = dev(rn(g, 192, dtype=BF)), dev(rn(g, 192, dtype=BF))
    gp = cc3d.group_norm_plan(cc3d.make_group_norm_desc(3, 900, 192, 32, act="silu"))
    tok = cc3d.group_norm_plan(cc3d.make_group_norm_desc(2700, 1, 192, 3))
    gs, gb, ts, tb = space(gp), space(gp, True), space(tok), space(tok, True)
    rp = cc3d.rotary_plan(cc3d.make_rotary_desc(2, 333, 2, 2, 64))
    rq, rk = torch.empty_like(c.i["q"]), torch.empty_like(c.i["k"])
    off = torch.tensor([7, 100000], dtype=torch.int32, device=DEV)
    o = {"o": nan(2, 333, 4, 64, dtype=BF), "h": nan(2, 4, 64, 64), "so": nan(3, 9, 2, 128, dtype=BF), "sh": nan(3, 2, 64, 128),
         "dq": nan(2, 333, 2, 64, dtype=BF), "dk": nan(2, 333, 2, 64, dtype=BF), "dv": nan(2, 333, 4, 64, dtype=BF),
         "dlog_decay": nan(4), "dh_in": nan(2, 4, 64, 64), "y": torch.empty_like(x), "stats": nan(3, 32, 2),
         "dx": torch.empty_like(x), "dw": nan(192), "db": nan(192), "ty": torch.empty_like(x), "tdx": torch.empty_like(x),
         "tdw": nan(192), "rq": rq, "rk": rk}

    def run(stream=None):
        i = c.i
        cc3d.rotary_forward(rp, i["q"], i["k"], rq, rk, offsets=off, stream=stream)
        cc3d.linear_attention_forward(c.plan, rq, rk, i["v"], o["o"], log_decay=i["log_decay"], h_in=i["h_in"], h_out=o["h"],
                                      lengths=c.lengths, workspace=c.space, stream=stream)
        cc3d.linear_attention_backward(c.plan, rq, rk, i["v"], i["do"], log_decay=i["log_decay"], h_in=i["h_in"],
                                       dh_out=i["dh_out"], lengths=c.lengths, workspace=c.back_space, stream=stream,
                                       **{k: o[k] for k in ("dq", "dk", "dv", "dlog_decay", "dh_in")})
        s = short.i
        cc3d.linear_attention_forward(short.plan, s["q"], s["k"], s["v"], o["so"], log_decay=s["log_decay"], h_in=s["h_in"],
                                      h_out=o["sh"], stream=stream)
        cc3d.group_norm_forward(gp, x, o["y"], w=w, b=b, stats=o["stats"], workspace=gs, stream=stream)
        cc3d.group_norm_backward(gp, x, dy, w=w, b=b, stats=o["stats"], dx=o["dx"], dw=o["dw"], db=o["db"], workspace=gb,
                                 stream=stream)
        flat = (2700, 1, 192)
        cc3d.group_norm_forward(tok, x.reshape(flat), o["ty"].view(flat), w=w, b=b, workspace=ts, stream=stream)
        cc3d.group_norm_backward(tok, x.reshape(flat), dy.reshape(flat), w=w, b=b, dx=o["tdx"].view(flat), dw=o["tdw"],
                                 workspace=tb, stream=stream)

    return run, o


def test_repeated_calls_and_another_stream_give_the_same_bits(cuda_device):
    run, o = everything(50)
    run()
    torch.cuda.synchronize()
    first = {k: v.clone() for k, v in o.items()}
    assert all(bool(torch.isfinite(v).all()) for v in first.values())
    other = torch.cuda.Stream()
    for stream in (None, other, other.cuda_stream):
        for v in o.values():
            v.fill_(NAN)
        torch.cuda.synchronize()
        run(stream)
        torch.cuda.synchronize()
        for k, v in o.items():
            same(v, first[k], k)


def test_replayed_graphs(cuda_device):
    """Two graphs of the same calls on the same workspaces, replayed in turn with eager calls and fills between them."""
    run, o = everything(60)
    run()
    torch.cuda.synchronize()
    first = {k: v.clone() for k, v in o.items()}
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        graphs.append(graph)
    for turn in range(4):
        for v in o.values():
            v.fill_(NAN)
        graphs[turn % 2].replay()
        torch.cuda.synchronize()
        for k, v in o.items():
            same(v, first[k], (turn, k))
        run()
        torch.cuda.synchronize()
        for k, v in o.items():
            same(v, first[k], (turn, k))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot,first", [(64, 64, 0), (64, 32, 16), (100, 50, 10), (7, 4, 2), (1000, 256, 100)])
def test_rotary_in_place(cuda_device, d, rot, first, layout):
    g = torch.Generator().manual_seed(70)
    plan = cc3d.rotary_plan(cc3d.make_rotary_desc(2, 11, 9, 3, d, rot=rot, first=first, layout=layout))
    wide = dev(rn(g, 2, 11, 12 * d, dtype=BF))
    q, k = wide[..., :9 * d], wide[..., 9 * d:]  # parts of one projection
    want = [torch.empty(v.shape, dtype=BF, device=DEV) for v in (q, k)]
    lengths = torch.tensor([11, 4], dtype=torch.int32, device=DEV)
    cc3d.rotary_forward(plan, q, k, *want, lengths=lengths)
    cc3d.rotary_forward(plan, q, k, q, k, lengths=lengths)
    torch.cuda.synchronize()
    same(q, want[0])
    same(k, want[1])


def test_rotary_axes(cuda_device):
    """Positions along three axes of a latent, each turning its part of a head: three calls, in place."""
    g = torch.Generator().manual_seed(71)
    t, h, d = 24, 2, 48
    x = rn(g, 1, t, h, d)
    got = dev(x)
    want, at = d64(x), torch.arange(t)
    for first, pos in ((0, at // 12), (16, at // 4 % 3), (32, at % 4)):
        plan = cc3d.rotary_plan(cc3d.make_rotary_desc(1, t, h, 0, d, rot=16, first=first, dtype=F32))
        cc3d.rotary_forward(plan, got, None, got, None, positions=dev(pos[None].int()))
        want = ho.rotary(want, pos[None], ho.frequencies(16), first, "half")
    torch.cuda.synchronize()
    # sixteen roundings of two terms of up to the largest value
    assert float((got.cpu().double() - want).abs().max()) <= 32 * ho.EPS32 * float(x.abs().max())


@pytest.mark.parametrize("p", [1, 20, 3000])
@pytest.mark.parametrize("c,groups", [(192, 32), (64, 4), (37, 1)])
def test_group_norm_far_from_zero(cuda_device, p, c, groups):
    """Means of a thousand standard deviations: the bound grows with max|x| rstd and no faster."""
    g = torch.Generator().manual_seed(80)
    x = rn(g, 3, p, c, mean=1000.0)
    x[1] -= 2000.0
    plan = cc3d.group_norm_plan(cc3d.make_group_norm_desc(3, p, c, groups, eps=EPS, dtype=F32))
    want = ho.group(d64(x), groups, None, None, False, EPS)
    y, stats = nan(3, p, c), nan(3, groups, 2)
    cc3d.group_norm_forward(plan, dev(x), y, stats=stats, workspace=space(plan))
    torch.cuda.synchronize()
    group_near(y, want["y"], want["y_unit"], F32, p, "y")
    group_near(stats, want["stats"], want["stats_unit"], F32, p, "stats")


@pytest.mark.parametrize("p", [1, 20, 3000])
@pytest.mark.parametrize("bad", [INF, NAN])
def test_group_norm_keeps_strange_values_in_their_group(cuda_device, p, bad):
    g = torch.Generator().manual_seed(81)
    x, dy = dev(rn(g, 3, p, 64, dtype=BF)), dev(rn(g, 3, p, 64, dtype=BF))
    w, b = dev(rn(g, 64, dtype=BF)), dev(rn(g, 64, dtype=BF))
    plan = cc3d.group_norm_plan(cc3d.make_group_norm_desc(3, p, 64, 4, act="silu"))

    def run(x, dy):
        y, stats, dx, dw = torch.empty_like(x), nan(3, 4, 2), torch.empty_like(x), nan(64)
        cc3d.group_norm_forward(plan, x, y, w=w, b=b, stats=stats, workspace=space(plan))
        cc3d.group_norm_backward(plan, x, dy, w=w, b=b, dx=dx, dw=dw, workspace=space(plan, True))
        torch.cuda.synchronize()
        return y, stats, dx, dw

    clean = run(x, dy)
    z = x.clone()
    z[1, p // 2, 20] = bad
    got = run(z, dy)
    other = [c for c in range(64) if not 16 <= c < 32]
    for k in (0, 2):
        same(got[k][[0, 2]], clean[k][[0, 2]])
        same(got[k][1][:, other], clean[k][1][:, other])
        assert not bool(torch.isfinite(got[k][1, :, 16:32]).any())
    same(got[1][:, [0, 2, 3]], clean[1][:, [0, 2, 3]])
    assert not bool(torch.isfinite(got[1][1, 1, 0]))
    same(got[3][other], clean[3][other])
    z = dy.clone()
    z[1, p // 2, 20] = bad
    got = run(x, z)
    same(got[2][[0, 2]], clean[2][[0, 2]])
    same(got[2][1][:, other], clean[2][1][:, other])
    same(got[3][[c for c in range(64) if c != 20]], clean[3][[c for c in range(64) if c != 20]])


def test_offsets_past_32_bits(cuda_device):
    """Sequences more than 2^31 elements apart, and in one buffer of more than 2^32 bytes."""
    apart = (1 << 31) + 4096
    buf = torch.zeros(apart + 200 * 256, dtype=BF, device=DEV)
    g = torch.Generator().manual_seed(90)
    x = rn(g, 2, 200, 256, dtype=BF)
    far = torch.as_strided(buf, (2, 200, 256), (apart, 256, 1))
    far.copy_(dev(x))
    plan = cc3d.linear_attention_plan(cc3d.make_linear_attention_desc(2, 200, 4, 64, 64))
    q = far.unflatten(-1, (4, 64))
    o, want = nan(2, 200, 4, 64, dtype=BF), nan(2, 200, 4, 64, dtype=BF)
    cc3d.linear_attention_forward(plan, q, q, q, o, workspace=space(plan))
    d = dev(x).unflatten(-1, (4, 64))
    cc3d.linear_attention_forward(plan, d, d, d, want, workspace=space(plan))
    torch.cuda.synchronize()
    same(o, want)
    gq, wq = nan(2, 200, 4, 64, dtype=BF), nan(2, 200, 4, 64, dtype=BF)
    cc3d.linear_attention_backward(plan, q, q, q, q, dq=gq, workspace=space(plan, True))
    cc3d.linear_attention_backward(plan, d, d, d, d, dq=wq, workspace=space(plan, True))
    torch.cuda.synchronize()
    same(gq, wq)
    gp = cc3d.group_norm_plan(cc3d.make_group_norm_desc(2, 200, 256, 8, act="silu"))
    y, wy = torch.empty_like(dev(x)), torch.empty_like(dev(x))
    cc3d.group_norm_forward(gp, far, y, workspace=space(gp))
    cc3d.group_norm_forward(gp, dev(x), wy, workspace=space(gp))
    torch.cuda.synchronize()
    same(y, wy)
    rp = cc3d.rotary_plan(cc3d.make_rotary_desc(2, 200, 4, 0, 64))
    cc3d.rotary_forward(rp, dev(x), None, wy, None)
    cc3d.rotary_forward(rp, far, None, far, None)
    torch.cuda.synchronize()
    same(far, wy)
    del buf, far, q
    torch.cuda.empty_cache()


def test_states_past_32_bits(cuda_device):
    """More than 2^32 bytes of states: 2100 sequences of 8 heads of 256 by 256, one token."""
    n = 2100
    c = cc3d.linear_attention_plan(cc3d.make_linear_attention_desc(n, 1, 8, 256, 256, dtype=F32))
    g = torch.Generator(device=DEV).manual_seed(91)
    q, k, v = (torch.randn(n, 1, 8, 256, generator=g, device=DEV) for _ in range(3))
    state = torch.randn(n, 8, 256, 256, generator=g, device=DEV)
    tail, o = state[-1].clone(), nan(n, 1, 8, 256)
    cc3d.linear_attention_forward(c, q, k, v, o, h_in=state, h_out=state)
    torch.cuda.synchronize()
    want = tail.double() + k[-1, 0].double()[..., None] * v[-1, 0].double()[:, None]
    assert float((state[-1].double() - want).abs().max()) <= 4 * ho.EPS32 * float(want.abs().max())
    out = (q[-1, 0].double()[..., None] * want).sum(1) / 16
    assert float((o[-1, 0].double() - out).abs().max()) <= 512 * ho.EPS32 * float((q[-1, 0].double().abs()[..., None] * want.abs()).sum(1).max()) / 16
    del state
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_growing_states(cuda_device, dtype):
    """Decays above one: states grow as the recurrence's do."""
    c = Linear(1, 150, 2, 16, 16, dtype=dtype)
    i = dict(c.i)
    grow = torch.tensor([0.05, 0.3], device=DEV)
    got = c.forward(log_decay=grow)
    torch.cuda.synchronize()
    args = [d64(i[x].cpu()) for x in ("q", "k", "v")] + [d64(grow.cpu()), float(c.plan.desc.scale), d64(i["h_in"].cpu()), None, 2]
    want, last = ho.linear(*args)
    mag, mag_last = ho.linear(*args, mag=True)
    depth, bf = ho.linear_depth(150, 16, 16), dtype == BF
    near(got["o"], want, ho.linear_bound(mag, want, dtype, depth, 2.0 ** -8 if bf else 0.0), "o")
    near(got["h_out"], last, ho.linear_bound(mag_last, last, F32, depth, 2.0 ** -16 if bf else 0.0), "h_out")
