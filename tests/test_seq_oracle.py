"""The plain 64-bit forms of the sequence operators against themselves on the
CPU: every by-formula gradient against central differences of the forward
form along random directions, and chunked calls against one call."""
import itertools

import pytest
import torch

import seq_oracle as so

F64 = torch.float64


def _rn(g, *shape, scale=1.0, mean=0.0):
    return torch.randn(*shape, generator=g, dtype=F64) * scale + mean


def _slope(f, inputs, names, g, grads):
    """(f(x + e v) - f(x - e v)) / 2e against <gradient, v> for a random direction in each input.

    f is evaluated in float64 at e = 1e-5: truncation e^2 f''' / 6 ~ 1e-10 and
    rounding 1e-16 / e ~ 1e-11 of f, both far below the 1e-6 asked for."""
    for name in names:
        v = torch.randn(inputs[name].shape, generator=g, dtype=F64)
        e = 1e-5
        hi = f({**inputs, name: inputs[name] + e * v})
        lo = f({**inputs, name: inputs[name] - e * v})
        want = float((grads[name] * v).sum())
        got = float(hi - lo) / (2 * e)
        assert abs(got - want) <= 1e-6 * max(1.0, abs(want), float((grads[name] * v).abs().sum())), (name, got, want)


@pytest.mark.parametrize("k,act,ragged", [(1, True, False), (3, False, True), (4, True, True)])
def test_conv1d_gradients_match_differences(k, act, ragged):
    g = torch.Generator().manual_seed(7 + k)
    n, t, c = 3, 6, 5
    ln = [0, 2, 6] if ragged else None
    i = dict(x=_rn(g, n, t, c), w=_rn(g, k, c), b=_rn(g, c), cache=_rn(g, n, k - 1, c))
    dy, dtail = _rn(g, n, t, c), _rn(g, n, k - 1, c)

    def f(v):
        y, tail, _ = so.conv1d(v["x"], v["w"], v["b"], act, v["cache"], ln)
        return (y * dy).sum() + (tail * dtail).sum()

    dx, dw, db, dc = so.conv1d_grad(i["x"], i["w"], i["b"], act, dy, i["cache"], dtail, ln)
    _slope(f, i, ["x", "w", "b", "cache"], g, dict(x=dx, w=dw, b=db, cache=dc))


@pytest.mark.parametrize("groups,use_softplus,ragged", [(1, True, False), (2, True, True), (2, False, True)])
def test_scan_gradients_match_differences(groups, use_softplus, ragged):
    g = torch.Generator().manual_seed(11 + groups)
    n, t, c, s = 3, 5, 4, 3
    ln = [5, 0, 3] if ragged else None
    i = dict(u=_rn(g, n, t, c), dt=_rn(g, n, t, c, scale=0.3, mean=0.0 if use_softplus else 0.5),
             a=-torch.rand(c, s, generator=g, dtype=F64) - 0.1, b=_rn(g, n, t, groups, s), c=_rn(g, n, t, groups, s),
             d=_rn(g, c), z=_rn(g, n, t, c), bias=_rn(g, c, scale=0.2), h_in=_rn(g, n, c, s))
    dy, dh = _rn(g, n, t, c), _rn(g, n, c, s)

    def f(v):
        y, h, _ = so.scan(v["u"], v["dt"], v["a"], v["b"], v["c"], v["d"], v["z"], v["bias"], v["h_in"], ln, use_softplus)
        return (y * dy).sum() + (h * dh).sum()

    o = so.scan_grad(i["u"], i["dt"], i["a"], i["b"], i["c"], dy, i["d"], i["z"], i["bias"], i["h_in"], dh, ln,
                     use_softplus)
    _slope(f, i, list(i), g, dict(u=o["du"], dt=o["ddt"], a=o["da"], b=o["db"], c=o["dc"], d=o["dd"], z=o["dz"],
                                  bias=o["ddt_bias"], h_in=o["dh_in"]))


@pytest.mark.parametrize("post,pre,act,gate_rows", [("rms", "rms", True, 1), ("layer", "layer", True, 3),
                                                    (None, "rms", False, 2), ("layer", None, False, 1)])
def test_join_gradients_match_differences(post, pre, act, gate_rows):
    g = torch.Generator().manual_seed(23)
    r, c = 7, 6
    gates = (r + gate_rows - 1) // gate_rows
    i = dict(y=_rn(g, r, c), res=_rn(g, r, c), gate=_rn(g, gates, c), scale=_rn(g, c))
    for side, kind in (("post", post), ("pre", pre)):
        if kind:
            i[side + "_w"], i[side + "_b"] = _rn(g, c), _rn(g, c)
    dxo, dh = _rn(g, r, c), (_rn(g, r, c) if pre else None)
    opts = dict(post=post, pre=pre, act=act, eps=1e-3, gate_act=True, gate_rows=gate_rows)

    def f(v):
        x, h, _ = so.join(**v, **opts)
        return (x * dxo).sum() + (0 if h is None else (h * dh).sum())

    o, _ = so.join_grad(dx_out=dxo, dh=dh, **i, **opts)
    named = dict(y="dy", res="dresidual", gate="dgate", scale="dscale", post_w="dpost_w", post_b="dpost_b",
                 pre_w="dpre_w", pre_b="dpre_b")
    _slope(f, i, list(i), g, {k: o[named[k]] for k in i})


@pytest.mark.parametrize("cut", [1, 3])
def test_chunked_forms_equal_one_call(cut):
    g = torch.Generator().manual_seed(5)
    n, t, c, k, s = 2, 7, 4, 3, 3
    x, w, b, cache = _rn(g, n, t, c), _rn(g, k, c), _rn(g, c), _rn(g, n, k - 1, c)
    whole, tail, _ = so.conv1d(x, w, b, True, cache)
    first, mid, _ = so.conv1d(x[:, :cut], w, b, True, cache)
    rest, end, _ = so.conv1d(x[:, cut:], w, b, True, mid)
    assert torch.equal(torch.cat([first, rest], 1), whole) and torch.equal(end, tail)
    dt, a = _rn(g, n, t, c), -torch.rand(c, s, generator=g, dtype=F64)
    bb, cc = _rn(g, n, t, 2, s), _rn(g, n, t, 2, s)
    y, h, _ = so.scan(x, dt, a, bb, cc)
    y1, h1, _ = so.scan(x[:, :cut], dt[:, :cut], a, bb[:, :cut], cc[:, :cut])
    y2, h2, _ = so.scan(x[:, cut:], dt[:, cut:], a, bb[:, cut:], cc[:, cut:], h_in=h1)
    assert torch.equal(torch.cat([y1, y2], 1), y) and torch.equal(h2, h)


def test_the_comparison_finds_a_wrong_value():
    g = torch.Generator().manual_seed(9)
    ref = _rn(g, 4, 5)
    for dtype, off in itertools.product((torch.float32, torch.bfloat16), (0, 1)):
        got = ref.to(dtype)
        if off:
            got[2, 3] += 0.05 * got[2, 3].abs() + 0.05
            with pytest.raises(AssertionError):
                so.assert_close(got, ref, ref.abs(), 16, "planted")
        else:
            so.assert_close(got, ref, ref.abs(), 16, "as it is")
    got = ref.to(torch.float32)
    got[0, 0] = float("nan")
    with pytest.raises(AssertionError):
        so.assert_close(got, ref, ref.abs(), 16, "NaN")
