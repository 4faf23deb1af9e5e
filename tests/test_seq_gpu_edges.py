"""More sizes of the sequence operators at the edges of the kernels' layouts,
through the checks and bounds of test_seq_gpu: rows shorter than a vector or
one element past a lane, wave or workgroup, groups of one channel, states that
fill no lane, chunk lengths and their neighbours, time-major views, random
draws, and sequences of unequal length next to NaN."""
import random

import pytest
import torch

import causal_conv3d_video_amd as cc3d
import seq_oracle as so
import test_seq_gpu as base

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
DEV = base.DEV


@pytest.mark.parametrize("c", [1, 3, 7, 9, 15, 17, 65, 509])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_conv1d_row_lengths(cuda_device, c, dtype):
    base.test_conv1d_forward_and_backward(None, 3, 21, c, 4, "silu", dtype, True, 3, True, True)


@pytest.mark.parametrize("k", range(1, 9))
def test_conv1d_taps_longer_than_the_sequence(cuda_device, k):
    for t in (1, 2, 5, 8, 9, 17):
        base.test_conv1d_forward_and_backward(None, 4, t, 11, k, "silu", F32, True, 0, True, True)


@pytest.mark.parametrize("c", [1, 3, 7, 9, 63, 65, 127, 129, 255, 257, 511, 513, 1023, 1025, 2049, 4095, 4097, 8190])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_join_row_lengths(cuda_device, c, dtype):
    r = 37 if c < 1000 else 11
    base.test_join_forward_and_backward(None, r, c, "layer", "rms", "silu", 5, "silu", True, True, True, dtype, 1)
    base.test_join_forward_and_backward(None, r, c, "rms", "layer", None, 1, None, True, True, True, dtype, 0)


@pytest.mark.parametrize("r,gate_rows", [(1, 1), (2, 2), (1000, 999), (1000, 500), (5000, 4), (5001, 5000), (70, 1000)])
def test_join_gates_shared_by_many_or_few(cuda_device, r, gate_rows):
    base.test_join_forward_and_backward(None, r, 24, "rms", "rms", None, gate_rows, "silu", True, True, False, F32, 0)


@pytest.mark.parametrize("c,g,s", [(6, 6, 16), (6, 6, 3), (3, 1, 16), (9, 3, 20), (2, 2, 64), (5, 1, 33), (129, 1, 16),
                                   (33, 1, 8), (130, 2, 4), (260, 4, 1), (257, 1, 5), (66, 2, 48)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_scan_channels_groups_and_states(cuda_device, c, g, s, dtype):
    base.test_scan_forward_and_backward(None, 2, 13, c, s, g, dtype, True, 1, True, "dzbh")


@pytest.mark.parametrize("t", [1, 2, 3, 4, 5, 7, 8, 9, 31, 32, 33, 63, 64, 65, 66, 127, 128, 129, 193])
def test_scan_lengths_about_the_chunks(cuda_device, t):
    base.test_scan_forward_and_backward(None, 3, t, 20, 16, 1, F32, True, 0, True, "dzbh")
    base.test_scan_forward_and_backward(None, 4, t, 18, 4, 2, BF, True, 0, True, "dh")


def test_scan_many_chunks(cuda_device):
    """More chunks than one workgroup of the join takes at once."""
    base.test_scan_forward_and_backward(None, 1, 9000, 3, 2, 1, F32, False, 0, True, "dzbh")


def test_random_draws(cuda_device):
    r = random.Random(20261206)
    for _ in range(40):
        dtype = r.choice([BF, F32])
        base.test_conv1d_forward_and_backward(None, r.randint(1, 5), r.randint(1, 70), r.randint(1, 200), r.randint(1, 8),
                                              r.choice(["silu", None]), dtype, r.random() < 0.5, r.randint(0, 9),
                                              r.random() < 0.5, r.random() < 0.5)
        g = r.choice([1, 1, 2, 3])
        base.test_scan_forward_and_backward(None, r.randint(1, 4), r.randint(1, 90), g * r.randint(1, 50), r.randint(1, 64), g,
                                            dtype, r.random() < 0.5, r.randint(0, 9), r.random() < 0.7,
                                            "".join(q for q in "dzbh" if r.random() < 0.6))
        kinds = r.choice([("rms", "rms"), ("layer", "rms"), (None, "layer"), ("rms", None)])
        base.test_join_forward_and_backward(None, r.randint(1, 90), r.randint(1, 700), kinds[0], kinds[1],
                                            r.choice(["silu", None]) if kinds[1] else None, r.choice([0, 1, 3, 40]),
                                            r.choice(["silu", None]), r.random() < 0.5, r.random() < 0.5,
                                            r.random() < 0.5, dtype, r.randint(0, 9))


def test_time_major_views(cuda_device):
    """Tensors laid out [T][N][C], passed as their [N, T, C] views, outputs too."""
    g = torch.Generator().manual_seed(71)
    n, t, c, s, k = 5, 40, 24, 16, 4

    def major(x):
        return x.transpose(0, 1).contiguous().to(DEV).transpose(0, 1)

    x, w = base.rn(g, n, t, c, dtype=BF), base.rn(g, k, c, dtype=BF)
    plan = cc3d.causal_conv1d_plan(cc3d.make_conv1d_desc(n, t, c, k, act="silu"))
    y = base.nan(t, n, c, dtype=BF).transpose(0, 1)
    cc3d.causal_conv1d_forward(plan, major(x), w.to(DEV), None, y)
    dense = base.nan(n, t, c, dtype=BF)
    cc3d.causal_conv1d_forward(plan, x.to(DEV), w.to(DEV), None, dense)
    assert torch.equal(y, dense)
    i = base.scan_inputs(n, t, c, s, 2, BF, True, "dzbh", 72)
    sp = cc3d.selective_scan_plan(cc3d.make_scan_desc(n, t, c, s, groups=2))
    for call in (base.dev, major):
        j = {q: (call(v) if q in ("u", "dt", "b", "c", "z", "dy") else base.dev(v)) for q, v in i.items()}
        o = {q: base.nan(t, n, c, dtype=BF).transpose(0, 1) for q in ("y", "du", "ddt", "dz")}
        o["db"] = base.nan(t, n, 2, s, dtype=BF).transpose(0, 1)
        cc3d.selective_scan_forward(sp, j["u"], j["dt"], j["a"], j["b"], j["c"], o["y"], d=j["d"], z=j["z"],
                                    dt_bias=j["dt_bias"], h_in=j["h_in"], workspace=base.space(sp))
        cc3d.selective_scan_backward(sp, j["u"], j["dt"], j["a"], j["b"], j["c"], j["dy"], d=j["d"], z=j["z"],
                                     dt_bias=j["dt_bias"], h_in=j["h_in"], dh_out=j["dh_out"], du=o["du"], ddt=o["ddt"],
                                     db=o["db"], dz=o["dz"], workspace=base.space(sp, True))
        if call is base.dev:
            first = o
    for q, v in o.items():
        assert torch.equal(v, first[q]) and bool(torch.isfinite(v.float()).all()), q


def test_join_gate_gradient_of_a_gate_row_beside_one_with_nan(cuda_device):
    """A NaN in one gate row's rows leaves the next gate row's gradient as it is."""
    g = torch.Generator().manual_seed(73)
    gate_rows, gates, c = 5, 700, 16
    r = gate_rows * gates
    y, res, gate = base.rn(g, r, c), base.rn(g, r, c), base.rn(g, gates, c)
    dx = base.rn(g, r, c)
    plan = cc3d.norm_join_plan(cc3d.make_join_desc(r, c, post="rms", pre=None, gate_rows=gate_rows, dtype=F32))

    def grad(yy):
        out = base.nan(gates, c)
        cc3d.norm_join_backward(plan, base.dev(yy), base.dev(res), dx_out=base.dev(dx), gate=base.dev(gate), dgate=out,
                                workspace=base.space(plan, True))
        return out.cpu()

    clean = grad(y)
    for bad in (0, 3, 699):
        z = y.clone()
        z[bad * gate_rows + 4] = float("nan")
        got = grad(z)
        keep = torch.ones(gates, dtype=torch.bool)
        keep[bad] = False
        assert torch.equal(got[keep], clean[keep]) and bool(torch.isnan(got[bad]).all())


def test_far_tokens_are_refused(cuda_device):
    """Views whose tokens are 2**25 elements apart: the scan says so (unsupported), nothing is launched."""
    n, c, s = 1, 4, 2
    big = torch.zeros((1 << 25) + 8, dtype=BF, device=DEV)
    far = big.as_strided((n, 2, c), (0, 1 << 25, 1))
    near = torch.zeros(n, 2, c, dtype=BF, device=DEV)
    bc = torch.zeros(n, 2, s, dtype=BF, device=DEV)
    a = -torch.ones(c, s, device=DEV)
    plan = cc3d.selective_scan_plan(cc3d.make_scan_desc(n, 2, c, s))
    out = torch.full_like(near, 7.0)
    with pytest.raises(cc3d.CC3DError) as e:
        cc3d.selective_scan_forward(plan, far, near, a, bc, bc, out)
    assert e.value.status == cc3d.CC3D_ERR_UNSUPPORTED
    torch.cuda.synchronize()
    assert bool((out == 7.0).all())
    cc3d.selective_scan_forward(plan, near, near, a, bc, bc, out)
    assert bool((out == 0).all())


def test_device_side_lengths_out_of_range_are_clamped(cuda_device):
    g = torch.Generator().manual_seed(74)
    n, t, c, k = 4, 6, 16, 3
    x, w = base.dev(base.rn(g, n, t, c)), base.dev(base.rn(g, k, c))
    plan = cc3d.causal_conv1d_plan(cc3d.make_conv1d_desc(n, t, c, k, dtype=F32))
    outs = []
    for ln in ([-7, 2**31 - 1, 3, -2**31], [0, t, 3, 0]):
        y, co = base.nan(n, t, c), base.nan(n, k - 1, c)
        cc3d.causal_conv1d_forward(plan, x, w, None, y, cache_out=co,
                                   lengths=torch.tensor(ln, dtype=torch.int32, device=DEV))
        outs.append((y, co))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert bool((outs[0][0][0] == 0).all()) and bool((outs[0][1][0] == 0).all())
    assert so.EPS32 > 0
