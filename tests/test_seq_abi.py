"""Host-side tests of the sequence operators' C ABI (include/cc3d_seq.h): the
library exports what the header declares, plans give their sizes, and the
documented refusals come back before any launch.  No GPU is used: every call
here is one that the checks refuse (pointers are made-up addresses that are
never read)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _build_if_missing():
    lib = os.path.join(ROOT, "causal_conv3d_video_amd", "libcc3d.so")
    if not os.path.exists(lib):
        import importlib.util
        spec = importlib.util.spec_from_file_location("cc3d_build", os.path.join(ROOT, "causal_conv3d_video_amd", "build.py"))
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
        mod.build()
    return lib


LIB = _build_if_missing()

import causal_conv3d_video_amd as cc3d  # noqa: E402
from causal_conv3d_video_amd import seq  # noqa: E402

BAD, UNSUP = cc3d.CC3D_ERR_INVALID_ARG, cc3d.CC3D_ERR_UNSUPPORTED


def test_library_exports_every_declared_symbol():
    text = open(os.path.join(ROOT, "include", "cc3d_seq.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    declared = sorted(set(re.findall(r"\b((?:causal_conv1d|selective_scan|norm_join)_\w+)\s*\(", text)))
    assert set(declared) == set(cc3d.SEQ_EXPORTED_SYMBOLS)
    nm = subprocess.run(["nm", "-D", "--defined-only", LIB], capture_output=True, text=True, check=True).stdout
    assert set(declared) <= set(re.findall(r"\s[TW]\s+(\S+)", nm))


def _refused(make, status, *a, **kw):
    before = cc3d.causal_conv3d_counters()
    with pytest.raises(cc3d.CC3DError) as e:
        make(*a, **kw)
    assert e.value.status == status
    after = cc3d.causal_conv3d_counters()
    name = "invalid" if status == BAD else "unsupported"
    assert after[name] == before[name] + 1


def test_plan_refusals():
    def conv(n=1, t=1, c=1, k=1, **kw):
        return cc3d.causal_conv1d_plan(cc3d.make_conv1d_desc(n, t, c, k, **kw))

    def scan(n=1, t=1, d=4, s=1, g=1, **kw):
        return cc3d.selective_scan_plan(cc3d.make_scan_desc(n, t, d, s, groups=g, **kw))

    def join(r=1, c=1, **kw):
        return cc3d.norm_join_plan(cc3d.make_join_desc(r, c, **kw))

    for kw in (dict(n=0), dict(t=0), dict(c=0), dict(k=0), dict(n=-1)):
        _refused(conv, BAD, **kw)
    _refused(conv, UNSUP, k=9)
    _refused(conv, UNSUP, t=(1 << 30) + 1)
    for kw in (dict(n=0), dict(t=0), dict(d=0), dict(s=0), dict(g=0), dict(g=3)):
        _refused(scan, BAD, **kw)
    _refused(scan, UNSUP, s=65)
    _refused(scan, UNSUP, n=1 << 30, d=1 << 20)
    for kw in (dict(r=0), dict(c=0), dict(gate_rows=0), dict(eps=0.0), dict(eps=float("nan")), dict(eps=float("inf")),
               dict(pre=None, act="silu")):
        _refused(join, BAD, **kw)
    _refused(join, UNSUP, c=8193)
    for make in (cc3d.make_conv1d_desc, cc3d.make_scan_desc):
        with pytest.raises(TypeError):
            make(1, 1, 1, 1, dtype=torch.float16)
    with pytest.raises(ValueError):
        cc3d.make_conv1d_desc(1, 1, 1, 1, act="gelu")
    with pytest.raises(ValueError):
        cc3d.make_join_desc(1, 1, post="batch")
    lib = cc3d._lib
    assert lib.causal_conv1d_plan(None, ctypes.byref(ctypes.c_void_p())) == BAD
    assert lib.selective_scan_plan_info(None, ctypes.byref(seq.SeqInfo())) == BAD
    lib.norm_join_plan_destroy(None)


def test_plan_sizes():
    p = cc3d.selective_scan_plan(cc3d.make_scan_desc(1, 1, 64, 16))
    assert p.info["chunks"] == 1 and p.info["workspace_bytes"] == 0
    p = cc3d.selective_scan_plan(cc3d.make_scan_desc(1, 4096, 64, 16))
    assert p.info["chunks"] > 1 and p.info["workspace_bytes"] >= p.info["chunks"] * 64 * 17 * 4
    assert p.info["backward_workspace_bytes"] > 0
    assert cc3d.causal_conv1d_plan(cc3d.make_conv1d_desc(2, 100, 64, 4)).info["workspace_bytes"] == 0
    p.close()
    p.close()


# ---- argument checks of a call.  Every buffer gets an address range of its own, 1 GiB apart.

def _rows(slot, batch, row, off=0):
    return seq.Rows((slot + 1) << 30 | off, batch, row)


def _conv1d(dtype=torch.bfloat16, n=2, t=10, c=16, k=4):
    plan = cc3d.causal_conv1d_plan(cc3d.make_conv1d_desc(n, t, c, k, act="silu", dtype=dtype))
    a = seq.Conv1dArgs()
    for i, name in enumerate(("x", "y", "dy", "dx")):
        setattr(a, name, _rows(i, t * c, c))
    for i, name in enumerate(("w", "b", "cache_in", "cache_out", "dcache_out", "dcache_in", "dw", "db", "lengths")):
        setattr(a, name, (10 + i) << 30)
    a.workspace, a.workspace_bytes = 30 << 30, plan.info["backward_workspace_bytes"]
    return plan, a


def _status(fn, plan, a):
    """The status of a call that must not launch: a call that the checks pass is never made here."""
    st = getattr(cc3d._lib, fn)(plan.handle, ctypes.byref(a), None)
    assert st == BAD, (fn, st)


CONV_FAULTS = {
    "no input": lambda a: setattr(a.x, "p", None),
    "no weights": lambda a: setattr(a, "w", None),
    "misaligned input": lambda a: setattr(a.x, "p", a.x.p + 1),
    "misaligned weights": lambda a: setattr(a, "w", a.w + 1),
    "misaligned lengths": lambda a: setattr(a, "lengths", a.lengths + 2),
    "negative stride": lambda a: setattr(a.x, "row", -16),
    "a stride that leaves the address space": lambda a: setattr(a.x, "batch", 1 << 62),
}


@pytest.mark.parametrize("name", list(CONV_FAULTS))
@pytest.mark.parametrize("fn", ["causal_conv1d_forward", "causal_conv1d_backward"])
def test_conv1d_argument_refusals(fn, name):
    plan, a = _conv1d()
    CONV_FAULTS[name](a)
    _status(fn, plan, a)


def test_conv1d_output_refusals():
    f, b = "causal_conv1d_forward", "causal_conv1d_backward"
    for fn, fault in (
            (f, lambda a: setattr(a.y, "p", None)), (b, lambda a: setattr(a.dy, "p", None)),
            (f, lambda a: setattr(a.y, "row", 15)),            # rows of 16 that overlap
            (f, lambda a: setattr(a.y, "batch", 159)),         # sequences that overlap
            (f, lambda a: setattr(a.y, "p", a.x.p)),           # in place
            (f, lambda a: setattr(a.y, "p", a.x.p + 2 * 16 * 19)),  # its first row on the input's last
            (f, lambda a: setattr(a, "cache_out", a.cache_in)),
            (f, lambda a: setattr(a, "cache_out", a.w - 2)),
            (b, lambda a: setattr(a.dx, "p", a.dy.p)),
            (b, lambda a: setattr(a, "dw", a.db - 4)),
            (b, lambda a: setattr(a, "dw", a.dw + 2)),
            (b, lambda a: setattr(a, "workspace", None)),
            (b, lambda a: setattr(a, "workspace", a.workspace + 8)),
            (b, lambda a: setattr(a, "workspace_bytes", a.workspace_bytes - 1)),
            (b, lambda a: setattr(a, "workspace", a.dx.p))):
        plan, a = _conv1d()
        fault(a)
        _status(fn, plan, a)
    assert cc3d._lib.causal_conv1d_forward(None, ctypes.byref(_conv1d()[1]), None) == BAD
    assert cc3d._lib.causal_conv1d_forward(_conv1d()[0].handle, None, None) == BAD


def _scan():
    n, t, d, s, g = 2, 10, 8, 4, 2
    plan = cc3d.selective_scan_plan(cc3d.make_scan_desc(n, t, d, s, groups=g, dtype=torch.float32))
    a = seq.ScanArgs()
    for i, name in enumerate(("u", "dt", "b", "c", "z", "y", "dy", "du", "ddt", "dz", "db", "dc")):
        w = g * s if name in ("b", "c", "db", "dc") else d
        setattr(a, name, _rows(i, t * w, w))
    for i, name in enumerate(("a", "d", "dt_bias", "h_in", "h_out", "dh_out", "dh_in", "da", "dd", "ddt_bias", "lengths")):
        setattr(a, name, (20 + i) << 30)
    a.workspace, a.workspace_bytes = 40 << 30, plan.info["backward_workspace_bytes"]
    return plan, a


def test_scan_argument_refusals():
    f, b = "selective_scan_forward", "selective_scan_backward"
    for fn, fault in (
            [(w, lambda a, q=q: setattr(getattr(a, q), "p", None)) for w in (f, b) for q in ("u", "dt", "b", "c")] + [
                (f, lambda a: setattr(a.y, "p", None)), (b, lambda a: setattr(a.dy, "p", None)),
                (f, lambda a: setattr(a, "a", None)), (f, lambda a: setattr(a, "a", a.a + 2)),
                (f, lambda a: setattr(a, "h_out", a.h_in + 4)),   # shifted: only the very same buffer may be both
                (f, lambda a: setattr(a.y, "p", a.u.p)),
                (f, lambda a: setattr(a.z, "p", a.z.p + 2)),
                (b, lambda a: setattr(a.z, "p", None)),           # dz without z
                (b, lambda a: setattr(a, "d", None)),             # dd without d
                (b, lambda a: setattr(a, "dt_bias", None)),
                (b, lambda a: setattr(a, "dh_in", a.h_in)),
                (b, lambda a: setattr(a.db, "p", a.b.p)),
                (b, lambda a: setattr(a, "workspace_bytes", 16))]):
        plan, a = _scan()
        fault(a)
        _status(fn, plan, a)


def _join(**kw):
    r, c = 12, 16
    opts = dict(post="rms", pre="layer", act="silu", gate_rows=4, dtype=torch.float32)
    opts.update(kw)
    plan = cc3d.norm_join_plan(cc3d.make_join_desc(r, c, **opts))
    a = seq.JoinArgs()
    for i, name in enumerate(("y", "residual", "gate", "x_out", "h_out", "dx_out", "dh", "dy", "dresidual", "dgate")):
        setattr(a, name, _rows(i, 0, c))
    for i, name in enumerate(("scale", "post_w", "post_b", "pre_w", "pre_b", "dscale", "dpost_w", "dpost_b", "dpre_w",
                              "dpre_b")):
        setattr(a, name, (20 + i) << 30)
    a.workspace, a.workspace_bytes = 40 << 30, plan.info["backward_workspace_bytes"]
    return plan, a


def test_join_argument_refusals():
    f, b = "norm_join_forward", "norm_join_backward"

    def without(*names):
        def fault(a):
            for q in names:
                v = getattr(a, q)
                if isinstance(v, seq.Rows):
                    v.p = None
                else:
                    setattr(a, q, None)
        return fault

    for fn, fault, kw in (
            (f, without("y"), {}), (f, without("y", "residual", "gate", "scale", "post_w", "post_b"), {}),
            (f, without("h_out"), {}), (b, without("dx_out", "dh"), {}), (b, without("residual"), {}),
            (b, without("gate"), {}), (b, without("scale"), {}), (b, without("pre_b"), {}),
            (f, lambda a: None, dict(post=None)),               # weights of a norm that is not there
            (f, lambda a: None, dict(pre=None, act=None)),
            (b, without("pre_w", "pre_b", "dpre_w", "dpre_b"), dict(pre=None, act=None)),  # dh without the norm
            (f, lambda a: setattr(a.x_out, "p", a.residual.p), {}), (f, lambda a: setattr(a.h_out, "row", 8), {}),
            (f, lambda a: setattr(a.h_out, "p", a.x_out.p), {}), (b, lambda a: setattr(a.dgate, "p", a.gate.p), {}),
            (b, lambda a: setattr(a, "dscale", a.dpost_w), {}),
            (b, lambda a: setattr(a, "workspace", None), {})):
        plan, a = _join(**kw)
        fault(a)
        _status(fn, plan, a)


def test_python_refuses_tensors_of_the_wrong_kind():
    plan = cc3d.causal_conv1d_plan(cc3d.make_conv1d_desc(1, 4, 8, 2))
    x = torch.zeros(1, 4, 8, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        cc3d.causal_conv1d_forward(plan, x, x, None, x)          # not on a GPU
    with pytest.raises(TypeError):
        cc3d.selective_scan_forward(plan, x, x, x, x, x, x)      # another operator's plan
    with pytest.raises(TypeError):
        cc3d.norm_join_forward(plan, x, x)
