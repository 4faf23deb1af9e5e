"""Sizes at the limits of the sequence operators' launches, on the CPU: what a
launch cannot hold is refused before any launch, by the plan or, where only the
backward pass or the gradients asked for are too large, by the call."""
import os

from test_sanitizers import ROOT, SAN, _build_and_run


def test_launch_limits_under_sanitizers(tmp_path):
    exe = str(tmp_path / "seq_limits_driver")
    csrc = os.path.join(ROOT, "causal_conv3d_video_amd", "csrc")
    out = _build_and_run(tmp_path, ["g++", "-std=c++17"] + SAN + [
        "-I", os.path.join(ROOT, "include"), "-I", csrc, os.path.join(csrc, "cc3d_seq_plan.cpp"),
        os.path.join(ROOT, "tests", "sanitize", "seq_limits_driver.cpp"), "-o", exe], exe)
    assert " 0 failed checks" in out
