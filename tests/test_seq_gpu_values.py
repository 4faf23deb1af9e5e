"""Values at the edges of the sequence operators' arithmetic on the GPU."""
import pytest
import torch

import causal_conv3d_video_amd as cc3d
import seq_oracle as so
import test_seq_gpu as base

pytestmark = pytest.mark.gpu
F32 = torch.float32
DEV = base.DEV


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
