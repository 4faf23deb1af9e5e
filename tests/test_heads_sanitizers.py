"""Host sanitizer build (AddressSanitizer and UndefinedBehaviorSanitizer) of
the plans and argument checks of the operators on heads and groups, driven over
a grid of shapes with the launches stubbed out."""
import os

from test_sanitizers import ROOT, SAN, _build_and_run


def test_heads_plans_under_sanitizers(tmp_path):
    exe = str(tmp_path / "heads_driver")
    csrc = os.path.join(ROOT, "causal_conv3d_video_amd", "csrc")
    out = _build_and_run(tmp_path, ["g++", "-std=c++17"] + SAN + [
        "-I", os.path.join(ROOT, "include"), "-I", csrc, os.path.join(csrc, "cc3d_heads_plan.cpp"),
        os.path.join(ROOT, "tests", "sanitize", "heads_driver.cpp"), "-o", exe], exe)
    assert " 0 failed checks" in out
