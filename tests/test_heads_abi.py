"""Host-side tests of the C ABI of the operators on heads and groups
(include/cc3d_heads.h): exports, plan sizes and the documented refusals, which
come back before any launch.  No GPU is used: every call here is one that the
checks refuse (pointers are made-up addresses that are never read)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from test_seq_abi import BAD, LIB, ROOT, UNSUP, _refused

import causal_conv3d_video_amd as cc3d
from causal_conv3d_video_amd import heads, seq


def test_library_exports_every_declared_symbol():
    text = open(os.path.join(ROOT, "include", "cc3d_heads.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    declared = sorted(set(re.findall(r"\b((?:linear_attention|rotary|group_norm)_\w+)\s*\(", text)))
    assert set(declared) == set(cc3d.HEADS_EXPORTED_SYMBOLS)
    nm = subprocess.run(["nm", "-D", "--defined-only", LIB], capture_output=True, text=True, check=True).stdout
    assert set(declared) <= set(re.findall(r"\s[TW]\s+(\S+)", nm))


def linear(n=1, t=1, h=4, dk=8, dv=8, **kw):
    return cc3d.linear_attention_plan(cc3d.make_linear_attention_desc(n, t, h, dk, dv, **kw))


def rotary(n=1, t=1, hq=2, hk=1, d=8, **kw):
    return cc3d.rotary_plan(cc3d.make_rotary_desc(n, t, hq, hk, d, **kw))


def group(n=1, p=1, c=8, g=2, **kw):
    return cc3d.group_norm_plan(cc3d.make_group_norm_desc(n, p, c, g, **kw))


def test_plan_refusals():
    inf, nan = float("inf"), float("nan")
    for kw in (dict(n=0), dict(t=0), dict(h=0), dict(dk=0), dict(dv=0), dict(n=-1), dict(q_heads=3), dict(k_heads=0),
               dict(v_heads=8), dict(scale=inf), dict(scale=nan)):
        _refused(linear, BAD, **kw)
    for kw in (dict(dk=257), dict(dv=257), dict(t=(1 << 30) + 1), dict(n=1 << 30, h=1 << 20), dict(n=1 << 28, t=64)):
        _refused(linear, UNSUP, **kw)
    for kw in (dict(n=0), dict(t=0), dict(hq=0), dict(hk=-1), dict(d=0, rot=2), dict(rot=0), dict(rot=3), dict(rot=10),
               dict(first=-1, rot=4), dict(first=2, rot=8), dict(theta=0.0), dict(theta=inf), dict(amplitude=nan),
               dict(scaling="linear", factor=0.0), dict(scaling="linear", factor=nan), dict(scaling="base", factor=2.0, rot=2),
               dict(scaling="parts", factor=2.0, original=0), dict(scaling="parts", factor=2.0, original=10, fast=1.0, slow=1.0),
               dict(scaling="parts", factor=2.0, original=10, slow=-1.0)):
        _refused(rotary, BAD, **kw)
    for kw in (dict(d=1026, rot=8), dict(d=1000, rot=258), dict(t=(1 << 30) + 1), dict(hq=1 << 30), dict(n=1 << 30, t=1 << 10)):
        _refused(rotary, UNSUP, **kw)
    for kw in (dict(n=0), dict(p=0), dict(c=0), dict(g=0), dict(g=3), dict(eps=0.0), dict(eps=nan), dict(eps=inf)):
        _refused(group, BAD, **kw)
    for kw in (dict(c=8200), dict(p=(1 << 30) + 1), dict(n=1 << 30, p=1 << 16)):
        _refused(group, UNSUP, **kw)
    for make in (lambda **kw: cc3d.make_linear_attention_desc(1, 1, 1, 1, 1, **kw),
                 lambda **kw: cc3d.make_rotary_desc(1, 1, 1, 1, 2, **kw), lambda **kw: cc3d.make_group_norm_desc(1, 1, 1, 1, **kw)):
        with pytest.raises(TypeError):
            make(dtype=torch.float16)
    with pytest.raises(ValueError):
        cc3d.make_rotary_desc(1, 1, 1, 1, 2, layout="other")
    with pytest.raises(ValueError):
        cc3d.make_rotary_desc(1, 1, 1, 1, 2, scaling="other")
    with pytest.raises(ValueError):
        cc3d.make_group_norm_desc(1, 1, 1, 1, act="gelu")
    for op in ("linear_attention", "rotary", "group_norm"):
        assert getattr(cc3d._lib, op + "_plan")(None, ctypes.byref(ctypes.c_void_p())) == BAD
        assert getattr(cc3d._lib, op + "_plan_info")(None, ctypes.byref(seq.SeqInfo())) == BAD
        getattr(cc3d._lib, op + "_plan_destroy")(None)


def test_codes_that_python_does_not_make():
    h = ctypes.c_void_p()
    for field, value in (("layout", 2), ("layout", -1), ("scaling", 4), ("scaling", -1), ("dtype", 9)):
        d = cc3d.make_rotary_desc(1, 1, 1, 1, 8)
        setattr(d, field, value)
        assert cc3d._lib.rotary_plan(ctypes.byref(d), ctypes.byref(h)) == BAD and not h.value
    d = cc3d.make_group_norm_desc(1, 1, 8, 1)
    d.act = 2
    assert cc3d._lib.group_norm_plan(ctypes.byref(d), ctypes.byref(h)) == BAD
    d = cc3d.make_linear_attention_desc(1, 1, 1, 8, 8)
    d.dtype = -1
    assert cc3d._lib.linear_attention_plan(ctypes.byref(d), ctypes.byref(h)) == BAD


def test_plan_sizes():
    assert linear(t=32, h=2).info["workspace_bytes"] == 0            # short calls take token after token
    p = linear(t=8192, h=2, dk=64, dv=64)
    assert p.info["chunks"] > 1 and p.info["workspace_bytes"] == 2 * p.info["chunks"] * 64 * 64 * 4
    assert linear(n=4096, t=64, h=2).info["workspace_bytes"] == 0    # enough heads to fill the card
    # a state for each block of 64 tokens, padded, and shared heads' sums
    assert p.info["backward_workspace_bytes"] >= 2 * 128 * 64 * 64 * 4
    shared = linear(t=8192, h=2, dk=64, dv=64, k_heads=1)
    assert shared.info["backward_workspace_bytes"] >= p.info["backward_workspace_bytes"] + 2 * 8192 * 64 * 4
    assert rotary(t=100).info == {"workspace_bytes": 0, "backward_workspace_bytes": 0, "chunks": 1, "backward_chunks": 1}
    assert group(n=1000).info["workspace_bytes"] == 0 and group(n=1000).info["backward_workspace_bytes"] > 0
    assert group(n=2, p=5000).info["workspace_bytes"] > 0
    p.close()
    p.close()


# ---- argument checks of a call.  Every buffer gets an address range of its own, 1 GiB apart.

def _rows(slot, batch, row):
    return seq.Rows((slot + 1) << 30, batch, row)


def _status(fn, plan, a, want=BAD):
    st = getattr(cc3d._lib, fn)(plan.handle, ctypes.byref(a), None)
    assert st == want, (fn, st)


def _linear(t=100):
    n, h, dk, dv = 2, 4, 8, 16
    plan = linear(n, t, h, dk, dv, k_heads=2)
    a = heads.LinearArgs()
    for i, (name, w) in enumerate((("q", h * dk), ("k", 2 * dk), ("v", h * dv), ("o", h * dv), ("grad_o", h * dv),
                                   ("dq", h * dk), ("dk", 2 * dk), ("dv", h * dv))):
        setattr(a, name, _rows(i, t * w, w))
    for i, name in enumerate(("log_decay", "h_in", "h_out", "dh_out", "dh_in", "dlog_decay", "lengths")):
        setattr(a, name, (20 + i) << 30)
    a.workspace, a.workspace_bytes = 40 << 30, plan.info["backward_workspace_bytes"]
    return plan, a


def test_linear_argument_refusals():
    f, b = "linear_attention_forward", "linear_attention_backward"
    for fn, fault in (
            [(w, lambda a, q=q: setattr(getattr(a, q), "p", None)) for w in (f, b) for q in ("q", "k", "v")] + [
                (f, lambda a: setattr(a.o, "p", None)), (b, lambda a: setattr(a.grad_o, "p", None)),
                (f, lambda a: setattr(a.q, "p", a.q.p + 1)), (f, lambda a: setattr(a, "log_decay", a.log_decay + 2)),
                (f, lambda a: setattr(a, "h_out", a.h_in + 4)), (f, lambda a: setattr(a, "h_out", a.h_in + 2)),
                (f, lambda a: setattr(a.o, "p", a.v.p)), (f, lambda a: setattr(a.o, "row", 63)),
                (f, lambda a: setattr(a.q, "row", -8)), (f, lambda a: setattr(a.q, "batch", 1 << 60)),
                (f, lambda a: setattr(a, "lengths", a.lengths + 1)),
                (b, lambda a: setattr(a, "log_decay", None)),      # dlog_decay without it
                (b, lambda a: setattr(a.dk, "p", a.k.p)), (b, lambda a: setattr(a.dq, "p", a.dv.p)),
                (b, lambda a: setattr(a, "dh_in", a.dh_out)), (b, lambda a: setattr(a, "dh_in", a.h_in)),
                (b, lambda a: setattr(a, "workspace", None)), (b, lambda a: setattr(a, "workspace", a.workspace + 8)),
                (b, lambda a: setattr(a, "workspace_bytes", a.workspace_bytes - 1)),
                (b, lambda a: setattr(a, "workspace", a.dv.p))]):
        plan, a = _linear()
        fault(a)
        _status(fn, plan, a)
    for fn, names in ((f, ("q", "k", "v", "o")), (b, ("q", "k", "v", "grad_o", "dq", "dk", "dv"))):
        for name in names:
            plan, a = _linear()
            v = getattr(a, name)
            v.p, v.row, v.batch = 1 << 50, 1 << 24, 100 << 24
            _status(fn, plan, a, UNSUP)
        assert getattr(cc3d._lib, fn)(None, ctypes.byref(a), None) == BAD
        assert getattr(cc3d._lib, fn)(plan.handle, None, None) == BAD


def _rotary():
    n, t, hq, hk, d = 2, 10, 4, 2, 8
    plan = rotary(n, t, hq, hk, d)
    a = heads.RotaryArgs()
    for i, (name, w) in enumerate((("q", hq * d), ("k", hk * d), ("q_out", hq * d), ("k_out", hk * d))):
        setattr(a, name, _rows(i, t * w, w))
    a.offsets, a.lengths = 20 << 30, 21 << 30
    return plan, a


@pytest.mark.parametrize("fn", ["rotary_forward", "rotary_backward"])
def test_rotary_argument_refusals(fn):
    for fault in (
            [lambda a, q=q: setattr(getattr(a, q), "p", None) for q in ("q", "k", "q_out", "k_out")] + [
                lambda a: setattr(a, "positions", 30 << 30),           # and offsets
                lambda a: setattr(a, "offsets", a.offsets + 2), lambda a: setattr(a.q_out, "p", a.q.p + 2),
                lambda a: setattr(a.k_out, "p", a.q.p), lambda a: setattr(a.q_out, "p", a.k_out.p),
                lambda a: (setattr(a.q_out, "p", a.q.p), setattr(a.q_out, "row", 40), setattr(a.q_out, "batch", 400)),
                lambda a: setattr(a.q_out, "row", 31), lambda a: setattr(a.k, "row", -1)]):
        plan, a = _rotary()
        fault(a)
        _status(fn, plan, a)
    plan = rotary(2, 10, 4, 0, 8)
    _status(fn, plan, _rotary()[1])                                    # k in a plan without k heads


@pytest.mark.parametrize("fn", ["rotary_forward", "rotary_backward"])
def test_rotary_refuses_one_buffer_for_q_and_k_that_is_written(fn):
    n, t, h, d = 2, 10, 4, 8
    for q, k, q_out, k_out in ((0, 0, 0, 0), (0, 0, 0, 1), (0, 0, 1, 0), (0, 1, 0, 0), (0, 1, 1, 1), (0, 1, 2, 2), (0, 1, 1, 0)):
        plan, a = rotary(n, t, h, h, d), heads.RotaryArgs()
        for name, slot in (("q", q), ("k", k), ("q_out", q_out), ("k_out", k_out)):
            setattr(a, name, _rows(slot, t * h * d, h * d))
        _status(fn, plan, a)


def _group(**kw):
    n, p, c, g = 2, 3000, 16, 4
    plan = group(n, p, c, g, **kw)
    a = heads.GroupArgs()
    for i, name in enumerate(("x", "y", "dy", "dx")):
        setattr(a, name, _rows(i, p * c, c))
    for i, name in enumerate(("w", "b", "stats", "dw", "db", "lengths")):
        setattr(a, name, (20 + i) << 30)
    a.workspace, a.workspace_bytes = 40 << 30, max(plan.info["workspace_bytes"], plan.info["backward_workspace_bytes"])
    return plan, a


def test_group_argument_refusals():
    f, b = "group_norm_forward", "group_norm_backward"
    for fn, fault in (
            (f, lambda a: setattr(a.x, "p", None)), (f, lambda a: setattr(a.y, "p", None)), (b, lambda a: setattr(a.dy, "p", None)),
            (f, lambda a: setattr(a.y, "p", a.x.p)), (f, lambda a: setattr(a, "stats", a.stats + 4)),
            (f, lambda a: setattr(a, "stats", a.workspace)), (f, lambda a: setattr(a, "w", a.w + 1)),
            (f, lambda a: setattr(a.x, "row", -1)), (f, lambda a: setattr(a, "workspace_bytes", 16)),
            (f, lambda a: setattr(a, "workspace", None)),
            (b, lambda a: setattr(a, "w", None)), (b, lambda a: setattr(a, "b", None)), (b, lambda a: setattr(a, "dw", a.db)),
            (b, lambda a: setattr(a.dx, "p", a.dy.p)), (b, lambda a: setattr(a, "workspace", a.dx.p)),
            (b, lambda a: setattr(a, "lengths", a.lengths + 2))):
        plan, a = _group()
        fault(a)
        _status(fn, plan, a)


def test_python_refuses_tensors_of_the_wrong_kind():
    x = torch.zeros(1, 1, 4, 8, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        cc3d.linear_attention_forward(linear(), x, x, x, x)      # not on a GPU
    with pytest.raises(TypeError):
        cc3d.rotary_forward(linear(), x, x, x, x)                # another operator's plan
    with pytest.raises(TypeError):
        cc3d.group_norm_forward(group(), x, x)
