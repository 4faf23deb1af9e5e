"""Sequence operators on the GPU at sizes where a grid goes on in turns and
where counts pass 32 bits.  A sequence's results do not depend on how many
sequences a call has, so a large call is compared bit for bit with calls of
one sequence, which test_seq_gpu compares with the 64-bit forms."""
import pytest
import torch

import causal_conv3d_video_amd as cc3d
import test_seq_gpu as base

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
DEV = base.DEV


def _same_inputs(n, t, c, s, g, seed):
    """One sequence's inputs, and views of them as n sequences."""
    i = base.scan_inputs(1, t, c, s, g, BF, True, "dzb", seed)
    one = {k: base.dev(v) for k, v in i.items()}
    many = {k: (v.expand(n, *v.shape[1:]) if v is not None and v.dim() > 2 else v) for k, v in one.items()}
    return one, many


def _backward(j, n, t, c, s, g, lengths=None, **got):
    plan = cc3d.selective_scan_plan(cc3d.make_scan_desc(n, t, c, s, groups=g))
    space = torch.empty(plan.info["backward_workspace_bytes"], dtype=torch.uint8, device=DEV)
    cc3d.selective_scan_backward(plan, j["u"], j["dt"], j["a"], j["b"], j["c"], j["dy"], d=j["d"], z=j["z"],
                                 dt_bias=j["dt_bias"], lengths=lengths, workspace=space, **got)


@pytest.mark.parametrize("n,t,c,s,g", [
    (40, 1000, 128, 64, 4),    # 20 million sums of dB and dC: a grid's turn takes 17 million
    (64, 65, 1024, 64, 1),     # 131072 workgroups of the chunks' join: a grid has 65536
    (1024, 8192, 128, 64, 4),  # 2**32 sums of dB and dC: as many threads as no launch has
])
def test_grids_go_on_in_turns(cuda_device, n, t, c, s, g):
    one, many = _same_inputs(n, t, c, s, g, 600 + n)
    want = dict(du=base.nan(1, t, c, dtype=BF), db=base.nan(1, t, g, s, dtype=BF), dc=base.nan(1, t, g, s, dtype=BF),
                dh_in=base.nan(1, c, s))
    _backward(one, 1, t, c, s, g, **want)
    got = {k: base.nan(n, *v.shape[1:], dtype=v.dtype) for k, v in want.items()}
    _backward(many, n, t, c, s, g, **got)
    for k, v in want.items():
        assert bool(torch.isfinite(v.float()).all()), k
        for q in range(0, n, 64):
            part = got[k][q:q + 64]
            assert torch.equal(part, v.expand_as(part)), (k, q)


def test_a_row_of_b_and_c_past_32_bits(cuda_device):
    """One token of 2**25 + 64 groups of 64 states: the last groups' B and C lie past 2**31 elements."""
    c, s, part = (1 << 25) + 64, 64, 128
    g = torch.Generator(device=DEV).manual_seed(610)

    def rn(*shape, dtype=BF, scale=1.0):
        return torch.randn(*shape, generator=g, device=DEV, dtype=dtype).mul_(scale)

    u, dt, b, cc = rn(1, 1, c), rn(1, 1, c), rn(1, 1, c, s), rn(1, 1, c, s)
    a = rn(c, s, dtype=F32).abs_().neg_()
    h_in = rn(1, c, s, dtype=F32)

    def call(lo, hi):
        n = hi - lo
        plan = cc3d.selective_scan_plan(cc3d.make_scan_desc(1, 1, n, s, groups=n))
        y = base.nan(1, 1, n, dtype=BF)
        cc3d.selective_scan_forward(plan, u[:, :, lo:hi], dt[:, :, lo:hi], a[lo:hi], b[:, :, lo:hi], cc[:, :, lo:hi], y,
                                    h_in=h_in[:, lo:hi].contiguous())
        return y

    whole = call(0, c)
    for lo in (0, (1 << 25) - part // 2, c - part):
        y = call(lo, lo + part)
        assert bool(torch.isfinite(y.float()).all()) and torch.equal(whole[:, :, lo:lo + part], y), lo


def test_conv1d_of_all_channels_32_bits_count(cuda_device):
    """C = 2**31 - 1, one tap and no activation: y = w x and dx = w dy, rounded once."""
    c = (1 << 31) - 1
    g = torch.Generator(device=DEV).manual_seed(620)
    x, w = (torch.randn(c, generator=g, device=DEV, dtype=BF) for _ in range(2))
    plan = cc3d.causal_conv1d_plan(cc3d.make_conv1d_desc(1, 1, c, 1))
    y = torch.full_like(x, float("nan"))
    cc3d.causal_conv1d_forward(plan, x.view(1, 1, c), w.view(1, c), None, y.view(1, 1, c))
    assert torch.equal(y, x * w)
    y.fill_(float("nan"))
    space = torch.empty(plan.info["backward_workspace_bytes"], dtype=torch.uint8, device=DEV)
    cc3d.causal_conv1d_backward(plan, x.view(1, 1, c), w.view(1, c), None, x.view(1, 1, c), dx=y.view(1, 1, c), workspace=space)
    assert torch.equal(y, x * w)
