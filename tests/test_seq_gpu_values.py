"""Values at the edges of the sequence operators' arithmetic on the GPU."""
import pytest
import torch

import causal_conv3d_video_amd as cc3d
import seq_oracle as so
import test_seq_gpu as base

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
DEV = base.DEV
INF = float("inf")


def _scan_bounds(i, lengths, softplus):
    """(reference, magnitudes) of y and h_out, and of the gradients."""
    o = [base.d64(i[k]) for k in ("u", "dt", "a", "b", "c", "d", "z", "dt_bias", "h_in")] + [lengths, softplus]
    g = [base.d64(i[k]) for k in ("u", "dt", "a", "b", "c", "dy", "d", "z", "dt_bias", "h_in", "dh_out")] + [lengths,
                                                                                                            softplus]
    return (so.scan(*o)[:2], so.scan(*o, mag=True)[:2]), (so.scan_grad(*g), so.scan_grad(*g, mag=True))


def _scan(i, n, t, c, s, g, dtype, softplus, lengths=None, names=()):
    """y, h_out and the named gradients of one call each way."""
    plan = cc3d.selective_scan_plan(cc3d.make_scan_desc(n, t, c, s, groups=g, softplus=softplus, dtype=dtype))
    j = {k: base.dev(v) for k, v in i.items()}
    lt = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV)
    opt = dict(d=j["d"], z=j["z"], dt_bias=j["dt_bias"], h_in=j["h_in"], lengths=lt)
    ins = [j[k] for k in ("u", "dt", "a", "b", "c")]
    y, h = base.nan(n, t, c, dtype=dtype), base.nan(n, c, s)
    cc3d.selective_scan_forward(plan, *ins, y, h_out=h, workspace=base.space(plan), **opt)
    like = dict(du="u", ddt="dt", da="a", db="b", dc="c", dd="d", dz="z", ddt_bias="dt_bias")
    got = {k: base.nan(*(j[like[k]].shape if k in like else (n, c, s)),
                       dtype=dtype if k in ("du", "ddt", "db", "dc", "dz") else F32) for k in names}
    if names:
        cc3d.selective_scan_backward(plan, *ins, j["dy"], dh_out=j["dh_out"], workspace=base.space(plan, True), **opt, **got)
    return y, h, got


# ---------------------------------------------------------------- softplus

def test_softplus_is_good_to_a_few_roundings_over_its_range(cuda_device):
    """With u = B = C = 1 and no state, y is delta itself, and so is du with
    dy = 1: through the single-token kernel, the kernel of many tokens and the
    backward one.  In units of 2**-24 of the value: the exponential's argument
    is rounded twice, 1.25 |v| of a negative v and at most 1.25 of a positive
    one; the exponential 2; 1 + e, whose loss is added back through a
    reciprocal and a product, 4; the logarithm 2, its factor 2, their sum 1;
    below 12 with the positive argument's share, 14 with the loss of its own
    next order."""
    v = torch.cat([torch.linspace(-30, 21, 60000, dtype=F32)]
                  + [x + torch.linspace(-1e-3, 1e-3, 512, dtype=F32) for x in (-20., -16., -8., -4., -2., 0., 20.)])
    c = v.numel()
    want = so.softplus(v.double())
    bound = (14 + 1.25 * torch.clamp(-v.double(), min=0)) * so.EPS32 * want
    one = torch.ones(c, 1, device=DEV)
    seen = {}
    for t in (1, 3):
        plan = cc3d.selective_scan_plan(cc3d.make_scan_desc(1, t, c, 1, dtype=F32))
        dt = v.to(DEV).expand(1, t, c).contiguous()
        u, bc = torch.ones(1, t, c, device=DEV), torch.ones(1, t, 1, device=DEV)
        # (a state that is forgotten at once: every token's y is its own delta)
        y, du = base.nan(1, t, c), base.nan(1, t, c)
        cc3d.selective_scan_forward(plan, u, dt, -1e30 * one, bc, bc, y, workspace=base.space(plan))
        cc3d.selective_scan_backward(plan, u, dt, -1e30 * one, bc, bc, u, du=du, workspace=base.space(plan, True))
        seen.update({("y", t): y, ("du", t): du})
    for what, got in seen.items():
        for q in range(got.shape[1]):
            over = (got[0, q].cpu().double() - want).abs() - bound
            k = int(over.argmax())
            assert float(over[k]) <= 0, (what, q, float(v[k]), float(over[k] / (so.EPS32 * want[k])))


# ------------------------------------------------------- growing recurrences

@pytest.mark.parametrize("t,s,ragged", [(700, 16, False), (700, 4, True), (330, 40, True)])
def test_growing_recurrences_stay_finite_where_the_formula_does(cuda_device, t, s, ragged):
    """Every token's decay is e**3, so a chunk of 32 tokens multiplies by more
    than fp32 holds; inputs are zero but in the last 20 tokens and gradients
    but in the first 20, so nothing in the formula comes near that."""
    n, c, g = 3, 70, 2
    i = base.scan_inputs(n, t, c, s, g, F32, False, "dz", 500 + t + s)
    i["dt"] = torch.full((n, t, c), -1.0)
    i["a"] = torch.full((c, s), -3.0)
    ln = [t, t - 6, 150] if ragged else None
    for q in range(n):
        end = t if ln is None else ln[q]
        i["u"][q, :end - 20] = 0
        i["dy"][q, 20:] = 0
    names = ("du", "ddt", "da", "db", "dc", "dd", "dz", "dh_in")
    y, h, got = _scan(i, n, t, c, s, g, F32, False, ln, names)
    ((ry, rh), (my, mh)), (ref, mag) = _scan_bounds(i, ln, False)
    depth = 4 * t + 2 * s + 640  # as in test_seq_gpu: exponents here are 3, their roundings far below 64
    so.assert_close(y, ry, my, depth, "y")
    so.assert_close(h, rh, mh, depth, "h_out")
    for k, v in got.items():
        so.assert_close(v, ref[k], mag[k], 2 * depth + n * t + c, k)


def test_a_chunk_may_grow_by_more_than_fp32_holds(cuda_device):
    """States of 1e-30 times e**144 over the first chunk, and gradients the same over the last."""
    n, t, c, s = 2, 200, 64, 16
    i = base.scan_inputs(n, t, c, s, 1, F32, False, "h", 510)
    i["a"] = torch.full((c, s), -6.0)
    for first, k in ((0, "h_in"), (t - 24, "dh_out")):
        i["dt"] = torch.zeros(n, t, c)
        i["dt"][:, first:first + 24] = -1.0
        j = dict(i, u=torch.zeros(n, t, c), dy=torch.zeros(n, t, c), h_in=None, dh_out=None)
        j[k] = i[k] * 1e-30
        y, h, got = _scan(j, n, t, c, s, 1, F32, False, None, ("dh_in",))
        ((ry, rh), (my, mh)), (ref, mag) = _scan_bounds(j, None, False)
        # an exponent of 144, formed of at most three rounded products
        depth = 4 * t + 2 * s + 640 + 4 * 144
        so.assert_close(y, ry, my, depth, "y")
        so.assert_close(h, rh, mh, depth, "h_out")
        so.assert_close(got["dh_in"], ref["dh_in"], mag["dh_in"], depth, "dh_in")


# ------------------------------- zeros after the valid tokens, whatever precedes

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("s", [4, 8, 16, 64])
def test_scan_results_after_an_infinite_token_are_zero(cuda_device, s, dtype):
    n, t, c, g = 3, 75, 40, 2
    i = base.scan_inputs(n, t, c, s, g, dtype, True, "dzbh", 530 + s)
    ln = [5, 70, 13]
    for q, end in enumerate(ln):
        i["u"][q, end - 1, 3] = INF
    names = ("du", "ddt", "db", "dc", "dz")
    y, _, got = _scan(i, n, t, c, s, g, dtype, True, ln, names)
    for k, v in dict(got, y=y).items():
        for q, end in enumerate(ln):
            assert bool((v[q, end:] == 0).all()), (k, q)


@pytest.mark.parametrize("dtype,c,k", [(BF, 24, 4), (F32, 24, 4), (BF, 5, 3), (F32, 9, 8), (BF, 16, 2)])
def test_conv1d_gradients_after_an_infinite_token_are_zero(cuda_device, dtype, c, k):
    g = torch.Generator().manual_seed(540 + c)
    n, t = 4, 40
    x, w, dy = base.rn(g, n, t, c, dtype=dtype), base.rn(g, k, c, dtype=dtype), base.rn(g, n, t, c, dtype=dtype)
    ln = [5, 33, 8, 39]
    for q, end in enumerate(ln):
        x[q, end - 1, 2] = INF
    plan = cc3d.causal_conv1d_plan(cc3d.make_conv1d_desc(n, t, c, k, act="silu", dtype=dtype))
    dx = base.nan(n, t, c, dtype=dtype)
    cc3d.causal_conv1d_backward(plan, base.dev(x), base.dev(w), None, base.dev(dy), dx=dx, workspace=base.space(plan, True),
                                lengths=torch.tensor(ln, dtype=torch.int32, device=DEV))
    for q, end in enumerate(ln):
        assert bool((dx[q, end:] == 0).all()), q
        assert bool(torch.isfinite(dx[q, :max(0, end - k)].float()).all()), q


# ------------------------------------------------ states forgotten at once

@pytest.mark.parametrize("t,s", [(1, 16), (5, 16), (6, 4), (131, 16), (200, 40)])
def test_states_forgotten_at_once(cuda_device, t, s):
    """A = -inf: exp(delta A) is zero for every step, and a sequence's state
    does not change after its last token."""
    n, c = 4, 36
    i = base.scan_inputs(n, t, c, s, 2, F32, True, "dzbh", 520 + t)
    i["a"][:, 0] = -INF
    i["a"][5, s // 2] = -INF
    ln = [t, 0, 1, max(1, t - 2)]
    names = ("du", "da", "db", "dc", "dd", "dz", "dh_in")  # ddt's formula is inf * 0 there
    y, h, got = _scan(i, n, t, c, s, 2, F32, True, ln, names)
    ((ry, rh), (my, mh)), (ref, mag) = _scan_bounds(i, ln, True)
    depth = 4 * t + 2 * s + 640
    so.assert_close(y, ry, my, depth, "y")
    so.assert_close(h, rh, mh, depth, "h_out")
    for k, v in got.items():
        so.assert_close(v, ref[k], mag[k], 2 * depth + n * t + c, k)


# ------------------------------------------------------- masks by the step

@pytest.mark.parametrize("t,s", [(1, 16), (7, 4), (150, 16), (150, 64)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_steps_masked_by_infinity_or_the_lowest_value_leave_the_state(cuda_device, t, s, dtype):
    """softplus(-inf) = 0: such a token changes no state and has no gradient of its step; so with the type's lowest value."""
    n, c = 3, 40
    i = base.scan_inputs(n, t, c, s, 2, dtype, True, "dzbh", 560 + t)
    names = ("du", "ddt", "da", "db", "dc", "dd", "dz", "ddt_bias", "dh_in")
    for low in (-INF, float(torch.finfo(dtype).min)):
        i["dt"][:, t // 3:] = low
        i["dt"][1] = low
        y, h, got = _scan(i, n, t, c, s, 2, dtype, True, None, names)
        ref_in = dict(i, dt=i["dt"].clamp(min=-1e30))  # the same steps of zero, without the oracle's inf - inf
        ((ry, rh), (my, mh)), (ref, mag) = _scan_bounds(ref_in, None, True)
        depth = 4 * t + 2 * s + 640
        so.assert_close(y, ry, my, depth, "y")
        so.assert_close(h, rh, mh, depth, "h_out")
        assert torch.equal(h[1].cpu(), i["h_in"][1])
        for k, v in got.items():
            so.assert_close(v, ref[k], mag[k], 2 * depth + n * t + c, k)


def test_not_a_number_in_a_reaches_its_channel_only(cuda_device):
    n, t, c, s = 2, 150, 40, 16
    i = base.scan_inputs(n, t, c, s, 2, F32, True, "dzbh", 570)
    names = ("du", "ddt", "dz", "dh_in")
    clean = _scan(i, n, t, c, s, 2, F32, True, None, names)
    i["a"][7, 3] = base.NAN
    got = _scan(i, n, t, c, s, 2, F32, True, None, names)
    keep = torch.arange(c) != 7
    for k in names:
        axis = 1 if k == "dh_in" else 2
        assert torch.equal(got[2][k].cpu().index_select(axis, keep.nonzero()[:, 0]),
                           clean[2][k].cpu().index_select(axis, keep.nonzero()[:, 0])), k
    assert torch.equal(got[0].cpu()[..., keep], clean[0].cpu()[..., keep])
    assert bool(torch.isnan(got[0][..., 7]).all()) and bool(torch.isnan(got[1][:, 7, 3]).all())
    assert bool(torch.isnan(got[2]["dh_in"][:, 7, 3]).all())


# -------------------------------------------- rows that a workgroup does not have

@pytest.mark.parametrize("r,c,gate_rows", [(33, 24, 33), (17, 8, 17), (40003, 24, 1), (700, 515, 7)])
def test_an_infinite_gate_reaches_its_own_channel_of_the_sums_only(cuda_device, r, c, gate_rows):
    """An infinite gate makes its rows' norm zero and, at its channel, no number:
    dpre_w of the other channels and dpre_b are sums of numbers, whatever a
    workgroup does with the lines of lanes that have no row in its last step."""
    g = torch.Generator().manual_seed(580 + c)
    y, res, dh = base.rn(g, r, c), base.rn(g, r, c), base.rn(g, r, c)
    gate = base.rn(g, -(-r // gate_rows), c)
    gate[-1, 3] = INF
    plan = cc3d.norm_join_plan(cc3d.make_join_desc(r, c, post="rms", pre="rms", gate_rows=gate_rows, dtype=F32))
    dw, db = base.nan(c), base.nan(c)
    one = torch.ones(c, device=DEV)
    cc3d.norm_join_backward(plan, base.dev(y), base.dev(res), dh=base.dev(dh), gate=base.dev(gate), pre_w=one, pre_b=one * 0,
                            dpre_w=dw, dpre_b=db, workspace=base.space(plan, True))
    keep = torch.arange(c) != 3
    assert bool(torch.isfinite(dw.cpu()[keep]).all()) and bool(torch.isfinite(db.cpu()).all())
