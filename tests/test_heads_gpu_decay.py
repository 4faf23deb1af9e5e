"""linear_attention's decay on the GPU where nothing covers it: old states that
fade strongly beside little or nothing that is added.

Bounds.  A state that only fades is rounded once a block and once a segment,
by half a step of 2^-24, and its factor once or twice.  Calls of up to 32
tokens may take them one after another: a factor each, off by its exponent's
rounding (|g| log2(e) / 2 steps of 2^-24, times ln 2) and the exponential's one
or two units, and a rounding of the product: old_depth.
"""
import pytest
import torch

import causal_conv3d_video_amd as cc3d
import heads_oracle as ho
from test_heads_gpu import BF, DEV, F32, d64, near
from test_heads_gpu_edges import INF, Linear, same
from test_seq_gpu import dev, nan, space

pytestmark = pytest.mark.gpu


def old_depth(t, g):
    return 12 + t / 32 + min(t, 32) * (3 + float(g.abs().max()))


def positive(gen, *shape):
    return dev(0.5 + torch.rand(*shape, generator=gen))


# exp(g t) from 1e-4 to 1e-20 and beyond
FADES = [(1, -14.0), (1, -1.0), (2, -7.0), (9, -1.5), (20, -0.9), (40, -0.4), (64, -0.2), (64, -0.25), (64, -0.3), (100, -0.2),
         (100, -0.3), (130, -0.1), (64, -0.001), (1000, -0.02), (3000, -0.005), (3000, -0.012)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("t,g", FADES)
@pytest.mark.parametrize("dk,dv", [(16, 16), (50, 100), (128, 128), (256, 40)])
def test_old_states_fade_to_their_last_bits(cuda_device, dk, dv, t, g, dtype):
    """h_out from h_in with nothing added, dh_in from dh_out with nothing asked of the tokens, and the decay's gradient of
    both, whole calls and (few heads, many tokens) split ones."""
    gen = torch.Generator().manual_seed(100)
    c = Linear(2, t, 2, dk, dv, dtype=dtype)
    decay = torch.tensor([g, 0.7 * g])
    h, dh = positive(gen, 2, 2, dk, dv), positive(gen, 2, 2, dk, dv)
    f = torch.exp(d64(decay) * t)[None, :, None, None]
    for none in ("k", "v"):
        got = c.forward(**{none: torch.zeros_like(c.i[none]), "h_in": h, "log_decay": dev(decay)})
        torch.cuda.synchronize()
        want = d64(h).cpu() * f
        near(got["h_out"], want, old_depth(t, decay) * ho.EPS32 * want, "h_out")
    zero = {"do": torch.zeros_like(c.i["do"]), "k": torch.zeros_like(c.i["k"])}
    got = c.backward(("dh_in", "dlog_decay"), h_in=h, dh_out=dh, log_decay=dev(decay), **zero)
    torch.cuda.synchronize()
    want = d64(dh).cpu() * f
    near(got["dh_in"], want, old_depth(t, decay) * ho.EPS32 * want, "dh_in")
    # sum over tokens of <dh f[t-1-i], f f[i] h>: all terms are positive; sums of dk dv products along 16 terms a tile
    # of a lane's columns and then in 64 bits, the factors of both states
    want = t * (f * d64(h).cpu() * d64(dh).cpu()).sum((0, 2, 3))
    near(got["dlog_decay"], want, (2 * old_depth(t, decay) + max(dk, dv) + 8) * ho.EPS32 * want, "dlog_decay")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_streamed_fades_follow_one_call(cuda_device, dtype):
    """Single tokens and one call over all of them fade a state alike."""
    gen = torch.Generator().manual_seed(101)
    t, h, d = 90, 2, 32
    decay = torch.tensor([-0.3, -0.21])
    state = positive(gen, 1, h, d, d)
    want = d64(state).cpu() * torch.exp(d64(decay) * t)[None, :, None, None]
    zero = torch.zeros(1, t, h, d, dtype=dtype, device=DEV)
    o, h_out = nan(1, t, h, d, dtype=dtype), nan(1, h, d, d)
    plan = cc3d.linear_attention_plan(cc3d.make_linear_attention_desc(1, t, h, d, d, dtype=dtype))
    cc3d.linear_attention_forward(plan, zero, zero, zero, o, log_decay=dev(decay), h_in=state, h_out=h_out, workspace=space(plan))
    one = cc3d.linear_attention_plan(cc3d.make_linear_attention_desc(1, 1, h, d, d, dtype=dtype))
    for p in range(t):
        x = zero[:, p:p + 1]
        cc3d.linear_attention_forward(one, x, x, x, o[:, p:p + 1], log_decay=dev(decay), h_in=state, h_out=state)
    torch.cuda.synchronize()
    near(h_out, want, old_depth(t, decay) * ho.EPS32 * want, "one call")
    # (a factor's rounding each token, the exponential's few units, and the product's)
    near(state, want, 6 * t * ho.EPS32 * want, "token by token")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("g", [0.0, -0.01, -0.5, -2.0, -20.0])
@pytest.mark.parametrize("t,ragged", [(1, None), (20, None), (70, None), (130, [130, 0, 64, 7]), (3000, [3000, 0, 1, 700])])
def test_infinite_states_stay_infinite(cuda_device, t, ragged, g, dtype):
    """An infinity among h_in (dh_out) fades to an infinity, through blocks and segments with tokens and without; whatever it
    does not reach keeps its bits."""
    n = len(ragged) if ragged else 2
    c = Linear(n, t, 2, 24, 40, dtype=dtype, ragged=ragged)
    decay = torch.full((2,), g, device=DEV)
    assert t < 3000 or min(c.plan.info["chunks"], c.plan.info["backward_chunks"]) > 3
    for name, call in (("h_in", c.forward), ("dh_out", lambda **kw: c.backward(("dk", "dv", "dh_in"), **kw))):
        clean = call(log_decay=decay)
        x = c.i[name].clone()
        x[:, 0, 3, 5], x[:, 0, 11, 5] = INF, -INF
        got = call(log_decay=decay, **{name: x})
        torch.cuda.synchronize()
        out = "h_out" if name == "h_in" else "dh_in"
        assert bool((got[out][:, 0, 3, 5] == INF).all()) and bool((got[out][:, 0, 11, 5] == -INF).all()), name
        got[out][:, 0, [3, 11], 5] = clean[out][:, 0, [3, 11], 5]
        for k in got:
            same(got[k][..., 1, :, :] if k == out else got[k][:, :, 1], clean[k][..., 1, :, :] if k == out else clean[k][:, :, 1], k)
        same(got[out], clean[out], out)
        if name == "h_in" and g > -2:
            # column 5 of what the state met
            rest = [e for e in range(40) if e != 5]
            same(got["o"][..., rest], clean["o"][..., rest])
            assert not bool(torch.isfinite(got["o"][0, :, 0, 5]).any())


def growing_case(n, t, h, dk, dv, dtype, g, ragged, seed, zeros=0):
    c = Linear(n, t, h, dk, dv, dtype=dtype, ragged=ragged, seed=seed)
    i = dict(c.i)
    i["log_decay"] = torch.linspace(g, 0.6 * g, h, device=DEV)
    if zeros:  # tokens that add nothing
        for x in ("k", "v"):
            i[x] = i[x].clone()
            i[x][:, :zeros] = 0
        i["h_in"] = None
    args = [d64(i[x].cpu()) for x in ("q", "k", "v", "log_decay")] + [float(c.plan.desc.scale)]
    return c, i, args


# n, t, valid tokens, g, tokens of zeros before: states grow to 1e3 to 1e35 and fit fp32
GROWTH = [(1, 5, None, 1.6, 0), (1, 1, None, 3.0, 0), (1, 1, None, 60.0, 0), (2, 2, None, 30.0, 0), (1, 12, None, 5.0, 0),
          (1, 20, None, 3.5, 0), (1, 40, None, 1.5, 0), (1, 33, None, 2.1, 0), (3, 64, [64, 5, 1], 1.1, 0), (4, 100, [1, 5, 0, 40], 1.5, 0),
          (4, 3000, [1, 20, 0, 40], 1.6, 0), (1, 20, None, 5.0, 8), (1, 64, None, 2.0, 40), (1, 130, None, 2.0, 100),
          (2, 3000, [1995, 2000], 2.5, 1980), (2, 3000, [3000, 3000], 2.5, 2970)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", [(16, 16), (50, 100), (128, 128)])
@pytest.mark.parametrize("n,t,ragged,g,zeros", GROWTH)
def test_strong_growth(cuda_device, n, t, ragged, g, zeros, dk, dv, dtype):
    """Decays far above one, where the growth over a block of 64 tokens is no fp32 number and the states are."""
    c, i, args = growing_case(n, t, 2, dk, dv, dtype, g, ragged, 110, zeros)
    got = c.forward(**{k: i[k] for k in ("k", "v", "log_decay", "h_in")})
    torch.cuda.synchronize()
    args += [None if i["h_in"] is None else d64(i["h_in"].cpu()), ragged, 2]
    want, last = ho.linear(*args)
    mag, mag_last = ho.linear(*args, mag=True)
    assert float(mag_last.abs().max()) < 3e37
    depth, bf = ho.linear_depth(t, dk, dv), dtype == BF
    near(got["o"], want, ho.linear_bound(mag, want, dtype, depth, 2.0 ** -8 if bf else 0.0), "o")
    near(got["h_out"], last, ho.linear_bound(mag_last, last, F32, depth, 0.0), "h_out")


# (the products of states and their gradients grow as often as both do together)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", [(16, 16), (50, 100), (128, 128)])
@pytest.mark.parametrize("n,t,ragged,g", [(1, 1, None, 3.0), (1, 1, None, 60.0), (1, 5, None, 1.6), (1, 20, None, 3.2), (1, 33, None, 1.9),
                                          (1, 40, None, 1.5), (4, 100, [1, 5, 0, 40], 1.5), (4, 3000, [1, 20, 0, 40], 1.6)])
def test_strong_growth_backward(cuda_device, n, t, ragged, g, dk, dv, dtype):
    c, i, args = growing_case(n, t, 2, dk, dv, dtype, g, ragged, 111)
    args += [d64(i[x].cpu()) for x in ("do", "h_in", "dh_out")] + [ragged, 2]
    want, mag = ho.linear_grad(*args), ho.linear_grad(*args, mag=True)
    assert max(float(x.max()) for x in mag.values()) < 3e37
    depth, bf = 2 * ho.linear_depth(t, dk, dv) + 2, dtype == BF
    for ask in (("dq", "dk", "dv", "dlog_decay", "dh_in"), ("dq", "dk", "dv", "dh_in")):
        got = c.backward(ask, log_decay=i["log_decay"])
        torch.cuda.synchronize()
        for x in ask:
            f32 = x in ("dh_in", "dlog_decay")
            near(got[x], want[x], ho.linear_bound(mag[x], want[x], F32 if f32 else dtype, depth + n * t * (x == "dlog_decay"),
                                                  2.0 ** -8 if bf and not f32 else 0.0), x)



@pytest.mark.parametrize("dtype", [BF, F32])
def test_streamed_states_keep_32_bits(cuda_device, dtype):
    """The state of chunks of 3, 64, 40, 1 and 17 tokens: nothing of what is added to it is rounded to the tensors' type."""
    sizes = [3, 64, 40, 1, 17]
    t = sum(sizes)
    c = Linear(2, t, 3, 40, 24, dtype=dtype, seed=140)
    i = c.i
    args = [d64(i[x].cpu()) for x in ("q", "k", "v", "log_decay")] + [float(c.plan.desc.scale), d64(i["h_in"].cpu()), None, 3]
    last, mag = ho.linear(*args)[1], ho.linear(*args, mag=True)[1]
    state, at = i["h_in"].clone(), 0
    for m in sizes:
        plan = cc3d.linear_attention_plan(cc3d.make_linear_attention_desc(2, m, 3, 40, 24, dtype=dtype))
        q, k, v = (i[x][:, at:at + m] for x in ("q", "k", "v"))
        cc3d.linear_attention_forward(plan, q, k, v, nan(2, m, 3, 24, dtype=dtype), log_decay=i["log_decay"], h_in=state,
                                      h_out=state, workspace=space(plan))
        at += m
    torch.cuda.synchronize()
    near(state, last, ho.linear_bound(mag, last, F32, ho.linear_depth(t, 40, 24) + 8 * len(sizes), 0.0), "state")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("t", [1, 20, 70, 3000])
def test_a_decay_that_is_no_number_stays_with_its_head(cuda_device, t, dtype):
    c = Linear(2, t, 3, 24, 40, dtype=dtype)
    decay = c.i["log_decay"].clone()
    decay[1] = float("nan")
    for call in (c.forward, c.backward):
        clean, got = call(), call(log_decay=decay)
        torch.cuda.synchronize()
        for k, v in got.items():
            heads = {"h_out": 1, "dh_in": 1, "dlog_decay": 0}.get(k, 2)
            pick = lambda x, h: x.select(heads, h)
            for h in (0, 2):
                same(pick(v, h), pick(clean[k], h), k)
            if k in ("o", "h_out", "dh_in", "dlog_decay"):
                assert bool(torch.isnan(pick(v, 1)).all()), k
