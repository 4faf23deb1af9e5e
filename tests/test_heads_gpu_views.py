"""Views of the same memory whose strides differ only where there is nothing to step to."""
import pytest
import torch

import causal_conv3d_video_amd as cc3d
from test_heads_gpu import BF, DEV
from test_heads_gpu_edges import same
from test_seq_gpu import dev, nan, rn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,t", [(5, 1), (1, 5), (1, 1)])
def test_rotary_in_place_with_other_strides_of_single_steps(cuda_device, n, t):
    """A token of a step as [N, 1, ...] of one tensor and of another's view of it."""
    gen = torch.Generator().manual_seed(150)
    q = dev(rn(gen, n, t, 4, 32, dtype=BF))
    strides = list(q.stride())
    for dim, size in ((0, n), (1, t)):
        if size == 1:
            strides[dim] += 4096
    out = torch.as_strided(q, q.shape, strides)
    want = nan(n, t, 4, 32, dtype=BF)
    plan = cc3d.rotary_plan(cc3d.make_rotary_desc(n, t, 4, 0, 32))
    at = torch.full((n,), 77, dtype=torch.int32, device=DEV)
    cc3d.rotary_forward(plan, q, None, want, None, offsets=at)
    cc3d.rotary_forward(plan, q, None, out, None, offsets=at)
    torch.cuda.synchronize()
    same(q, want)
