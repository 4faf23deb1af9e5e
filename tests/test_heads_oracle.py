"""The plain 64-bit forms of the operators on heads and groups against torch's
differentiation of plain formulas, on the CPU."""
import pytest
import torch

import heads_oracle as ho

F64 = torch.float64


def _same(a, b, what):
    # two orders of the same sums of at most some thousand terms in 64 bits
    assert a.shape == b.shape
    assert not a.numel() or float((a - b).abs().max()) <= 1e-11 * max(1.0, float(b.abs().max())), what


@pytest.mark.parametrize("shared", [(4, 4, 4), (2, 2, 4), (4, 1, 1), (1, 2, 4)])
@pytest.mark.parametrize("ln", [None, [9, 0, 1, 14]])
def test_linear(shared, ln):
    g = torch.Generator().manual_seed(1)
    n, t, h, dk, dv = 4, 9, 4, 3, 5

    def rn(*shape):
        return torch.randn(*shape, generator=g, dtype=F64)

    q, k, v = rn(n, t, shared[0], dk), rn(n, t, shared[1], dk), rn(n, t, shared[2], dv)
    dec, h_in, do, dh = -rn(h).abs(), rn(n, h, dk, dv), rn(n, t, h, dv), rn(n, h, dk, dv)
    leaves = [x.clone().requires_grad_() for x in (q, k, v, dec, h_in)]
    lq, lk, lv, lg, lh = leaves
    # the sums over all earlier tokens, a matrix of decays a sequence
    total = 0
    o, last = ho.linear(q, k, v, dec, 0.7, h_in, ln, h)
    for i, m in enumerate(ho.lens(ln, n, t)):
        at = torch.arange(m, dtype=F64)
        apart = at[:, None] - at[None]
        fade = torch.exp(lg[:, None, None] * apart.clamp(min=0)) * (apart >= 0)
        qq, kk, vv = (x[i, :m].repeat_interleave(h // x.shape[2], 1).transpose(0, 1) for x in (lq, lk, lv))
        lead = torch.exp(lg[:, None] * (at + 1))[..., None]
        oo = 0.7 * ((qq @ kk.transpose(1, 2) * fade) @ vv + (qq * lead) @ lh[i])
        tail = torch.exp(lg[:, None] * (m - 1 - at))[..., None]
        ss = torch.exp(lg * m)[:, None, None] * lh[i] + (kk * tail).transpose(1, 2) @ vv
        _same(o[i, :m], oo.transpose(0, 1).detach(), "o")
        assert not o[i, m:].any()
        _same(last[i], ss.detach(), "state")
        total = total + (oo * do[i, :m].transpose(0, 1)).sum() + (ss * dh[i]).sum()
    total.backward()
    got = ho.linear_grad(q, k, v, dec, 0.7, do, h_in, dh, ln, h)
    for name, leaf in zip(("dq", "dk", "dv", "dlog_decay", "dh_in"), leaves):
        _same(got[name], leaf.grad, name)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary(layout):
    g = torch.Generator().manual_seed(2)
    x = torch.randn(2, 5, 3, 12, generator=g, dtype=F64)
    pos = torch.tensor([[0, 1, 2, 3, 4], [70, 3, 9, -5, 1000]])
    f = ho.frequencies(8)
    y = ho.rotary(x, pos, f, 2, layout)
    _same(ho.rotary(y, pos, f, 2, layout, back=True), x, "the turn undone")
    assert torch.equal(y[0, 0], x[0, 0]) and torch.equal(y[..., :2], x[..., :2]) and torch.equal(y[..., 10:], x[..., 10:])
    # products of two turned vectors go by the difference of their positions
    a, b = (ho.rotary(x[:1, :1].expand(1, 5, 3, 12), torch.arange(s, s + 5)[None], f, 2, layout) for s in (3, 40))
    _same((a[0, 1] * a[0, 4]).sum(-1), (b[0, 1] * b[0, 4]).sum(-1), "relative")


def test_frequencies():
    import math
    f = ho.frequencies(8)
    assert f[0] == 1 and abs(float(f[2]) - 0.01) < 1e-12
    base = ho.frequencies(8, scaling="base", factor=4.0)
    assert base[0] == 1 and abs(float(base[3] * 4 / f[3]) - 1) < 1e-12   # the slowest pair, stretched by the factor
    _same(ho.frequencies(8, scaling="linear", factor=4.0), f / 4, "linear")
    parts = ho.frequencies(8, scaling="parts", factor=4.0, original=1000, fast=32.0, slow=1.0)
    turns = 1000 * f / (2 * math.pi)
    assert turns[0] > 32 and parts[0] == f[0] and turns[3] < 1 and abs(float(parts[3] * 4 / f[3]) - 1) < 1e-12
    assert f[2] / 4 < parts[2] < f[2]


@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("ln", [None, [6, 0, 1]])
def test_group(act, ln):
    g = torch.Generator().manual_seed(3)
    n, p, c, groups = 3, 6, 12, 3
    x, w, b, dy = (torch.randn(*s, generator=g, dtype=F64) for s in ((n, p, c), (c,), (c,), (n, p, c)))
    lx, lw, lb = (v.clone().requires_grad_() for v in (x, w, b))
    total = 0
    out = ho.group(x, groups, w, b, act, 1e-3, ln)
    for i, m in enumerate(ho.lens(ln, n, p)):
        if not m:
            continue
        # torch's group norm takes channels first
        y = torch.nn.functional.group_norm(lx[i, :m].T[None], groups, lw, lb, 1e-3)[0].T
        y = torch.nn.functional.silu(y) if act else y
        _same(out["y"][i, :m], y.detach(), "y")
        total = total + (y * dy[i, :m]).sum()
    total.backward()
    got = ho.group(x, groups, w, b, act, 1e-3, ln, dy)
    for name, leaf in (("dx", lx), ("dw", lw), ("db", lb)):
        _same(got[name], leaf.grad, name)
