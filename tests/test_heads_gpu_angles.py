"""Rotary positions on the GPU: the angles of fp32 heads to their last bits."""
import pytest
import torch

import causal_conv3d_video_amd as cc3d
import heads_oracle as ho
from test_heads_gpu import DEV, F32
from test_seq_gpu import nan

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rot,d", [(64, 64), (50, 100)])
@pytest.mark.parametrize("back", [False, True])
def test_angles_of_fp32_heads(cuda_device, rot, d, back):
    """Pairs (1, 0) become the cosine and the sine themselves.  Two roundings of up to 2^-24 / sqrt(12) in the mean square,
    the function's own and that of what is added back to it, are 2.5e-8 together; a half turn in 32 bits would leave 2.9e-8
    more (pi 2^-24 / sqrt(12) where it is above 1/2, times a sine)."""
    gen = torch.Generator().manual_seed(120)
    n, t = 4, 2000
    pos = torch.randint(0, 1 << 20, (n, t), generator=gen, dtype=torch.int32)
    x = torch.zeros(n, t, 1, d, device=DEV)
    x[..., :rot // 2] = 1.0
    y = nan(n, t, 1, d)
    plan = cc3d.rotary_plan(cc3d.make_rotary_desc(n, t, 1, 0, d, rot=rot, dtype=F32))
    (cc3d.rotary_backward if back else cc3d.rotary_forward)(plan, x, None, y, None, positions=pos.to(DEV))
    torch.cuda.synchronize()
    want = ho.rotary(x.cpu().double(), pos, ho.frequencies(rot), 0, "half", back=back)
    off = (y.cpu().double() - want)[..., :rot]
    assert float(off.square().mean().sqrt()) <= 2.6e-8
    assert float(off.abs().max()) <= 2 * ho.EPS32
