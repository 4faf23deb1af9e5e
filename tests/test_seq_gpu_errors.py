"""Errors of other runtime calls beside the sequence operators' launches."""
import ctypes

import pytest
import torch

import test_seq_gpu as base

pytestmark = pytest.mark.gpu


def test_an_error_of_another_call_is_not_taken_for_one_of_the_launch(cuda_device):
    """The runtime keeps a thread's last error until it is asked for it: here that of a device that is not there."""
    hip = ctypes.CDLL("libamdhip64.so.7")
    launch, o, _ = base._everything(57)
    launch()
    torch.cuda.synchronize()
    first = {k: v.clone() for k, v in o.items()}
    for v in o.values():
        v.fill_(base.NAN)
    torch.cuda.synchronize()
    assert hip.hipGetLastError() == 0
    bad = hip.hipSetDevice(1 << 20)
    assert bad != 0
    try:
        launch()
        assert hip.hipGetLastError() == bad  # still there for whom it concerns
    finally:
        hip.hipGetLastError()
    torch.cuda.synchronize()
    for k, v in o.items():
        assert torch.equal(v, first[k]), k
