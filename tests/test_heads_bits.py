"""The states of bf16 linear attention and the decay's gradient keep 32 bits:
results of single terms, where nothing averages and a bound can be close.

A term is f times a product of bf16 values, f of up to 64 tokens at |g| = 0.02:
exponents of up to 1.9, three of whose roundings move f by 0.7 of that each (4
units of 2^-24), two exponentials (4), three products of factors, f v (1) and
the sum of its three parts (2): 16 units.  Two parts would be off by up to 2^-18
of the term, 64 units; the first test shows that some of these terms are.
"""
import pytest
import torch

import causal_conv3d_video_amd as cc3d
import heads_oracle as ho

F64, BF = torch.float64, torch.bfloat16
UNITS = 16
T, H, D, G = 40, 16, 16, -0.02
SPOTS = [0, 3, 17, 31, 32, 39]


def values(gen, *shape):
    return (1 + torch.rand(*shape, generator=gen)).to(BF)


def added(spot):
    """q, k, v, do [1, T, H, D] with one token that is not zero."""
    gen = torch.Generator().manual_seed(130 + spot)
    x = [torch.zeros(1, T, H, D, dtype=BF) for _ in range(4)]
    for v in x:
        v[:, spot] = values(gen, 1, H, D)
    return x


def one_state(seed):
    """A state [1, H, D, D] with one element that is not zero."""
    gen = torch.Generator().manual_seed(seed)
    s = torch.zeros(1, H, D, D)
    s[0, :, 5, 9] = 1 + torch.rand(H, generator=gen)
    return s


def parts(v, n):
    """v as n bf16 parts hold it."""
    out, rest = torch.zeros_like(v), v.clone()
    for _ in range(n):
        p = rest.to(BF).to(v.dtype)
        out, rest = out + p, rest - p
    return out


@pytest.mark.parametrize("spot", SPOTS)
def test_two_parts_are_outside_the_bound(spot):
    _, k, v, _ = added(spot)
    f = torch.exp(torch.tensor(G * (T - 1 - spot), dtype=F64))
    fv = (f * v[0, spot].to(F64)).float().to(F64)
    assert spot == T - 1 or float(((parts(fv, 2) - fv) / fv).abs().max()) > 2 * UNITS * ho.EPS32
    assert float(((parts(fv, 3) - fv) / fv).abs().max()) == 0
    s = one_state(131)[0, :, 5, 9].to(F64)
    assert float(((parts(s, 2) - s) / s).abs().max()) > 2 * UNITS * ho.EPS32


def close(got, want, what):
    off = ((got.cpu().to(F64) - want) / torch.where(want == 0, 1.0, want)).abs()
    assert float(off.max()) <= UNITS * ho.EPS32, (what, float(off.max()) / ho.EPS32)


def run(**kw):
    dev = {k: v.to("cuda:0") for k, v in kw.items()}
    decay = torch.full((H,), G, device="cuda:0")
    plan = cc3d.linear_attention_plan(cc3d.make_linear_attention_desc(1, T, H, D, D, scale=0.25))
    space = torch.empty(max(16, plan.info["workspace_bytes"], plan.info["backward_workspace_bytes"]), dtype=torch.uint8, device="cuda:0")
    o, h_out, dh_in = torch.empty_like(dev["v"]), torch.empty(1, H, D, D, device="cuda:0"), torch.empty(1, H, D, D, device="cuda:0")
    dlog = torch.empty(H, device="cuda:0")
    q, k, v, do = (dev[x] for x in ("q", "k", "v", "do"))
    cc3d.linear_attention_forward(plan, q, k, v, o, log_decay=decay, h_in=dev.get("h_in"), h_out=h_out, workspace=space)
    cc3d.linear_attention_backward(plan, q, k, v, do, log_decay=decay, h_in=dev.get("h_in"), dh_out=dev.get("dh_out"), dh_in=dh_in,
                                   dlog_decay=dlog, workspace=space)
    torch.cuda.synchronize()
    return h_out, dh_in, dlog


@pytest.mark.gpu
@pytest.mark.parametrize("spot", SPOTS)
def test_states_of_bf16_calls_keep_their_bits(cuda_device, spot):
    q, k, v, do = added(spot)
    h_out, dh_in, _ = run(q=q, k=k, v=v, do=do)
    f = torch.exp(torch.tensor(G, dtype=F64))
    term = lambda a, b: a[:, spot].to(F64)[..., None] * b[:, spot].to(F64)[:, :, None]
    close(h_out, f ** (T - 1 - spot) * term(k, v), "h_out")
    close(dh_in, 0.25 * f ** (spot + 1) * term(q, do), "dh_in")


@pytest.mark.gpu
@pytest.mark.parametrize("spot", SPOTS)
def test_decay_gradients_of_bf16_calls_keep_their_bits(cuda_device, spot):
    """One element of a state that came in, met by one token's q and do; and one that goes on to the end."""
    q, k, v, do = added(spot)
    zero, s, f = torch.zeros_like(q), one_state(131), torch.exp(torch.tensor(G, dtype=F64))
    e = s[0, :, 5, 9].to(F64)
    _, _, dlog = run(q=q, k=zero, v=zero, do=do, h_in=s)
    close(dlog, (spot + 1) * f ** (spot + 1) * 0.25 * q[0, spot, :, 5].to(F64) * e * do[0, spot, :, 9].to(F64), "q S do")
    _, _, dlog = run(q=zero, k=k, v=v, do=zero, dh_out=s)
    late = T - 1 - spot
    close(dlog, late * f ** late * k[0, spot, :, 5].to(F64) * e * v[0, spot, :, 9].to(F64), "k G v")
    _, _, dlog = run(q=zero, k=zero, v=zero, do=zero, h_in=s, dh_out=s)
    close(dlog, T * f ** T * e * e, "<S, G>")
