"""Operators on heads and groups of channels: Python binding of
include/cc3d_heads.h.

  linear_attention  a matrix state for each head, with a decay
  rotary            rotary positions of its q and k
  group_norm        norm of groups of channels, with an activation

Plans, streams, workspaces, ``lengths`` and errors are those of the sequence
operators (seq.py).  Tensors of heads are [N, T, H, D] (or [N, T, H*D]) with
the heads of a token next to each other; sequences and tokens may have any
strides, so a part of a wider projection is passed in place.  States are
[N, H, Dk, Dv] fp32, maps [N, P, C].
"""
import ctypes
import math
import struct

import torch

from . import CC3D_BF16, _lib
from .seq import (_ACTS, _F32, _I32, _NONE, Rows, SeqInfo, SeqPlan, _args, _call, _code, _dense, _device_of,
                  _dtype_code, _plan_of, _seq, _SHAPES, _space)

HEADS_EXPORTED_SYMBOLS = tuple(
    "%s_%s" % (op, what) for op in ("linear_attention", "rotary", "group_norm")
    for what in ("plan", "plan_info", "plan_destroy", "forward", "backward"))

_i32, _f64, _vp = ctypes.c_int32, ctypes.c_double, ctypes.c_void_p
_LAYOUTS = {"half": 0, "interleaved": 1}
_SCALINGS = {None: 0, "linear": 1, "base": 2, "parts": 3}


class LinearDesc(ctypes.Structure):
    _fields_ = [(name, _i32) for name in ("n", "t", "heads", "q_heads", "k_heads", "v_heads", "dk", "dv")] + [
        ("scale", ctypes.c_float), ("dtype", _i32)]


class RotaryDesc(ctypes.Structure):
    _fields_ = [(name, _i32) for name in ("n", "t", "q_heads", "k_heads", "d", "rot", "first", "layout", "scaling",
                                          "dtype")] + [
        (name, _f64) for name in ("theta", "factor", "original", "fast", "slow", "amplitude")]


class GroupDesc(ctypes.Structure):
    _fields_ = [(name, _i32) for name in ("n", "p", "c", "groups", "act")] + [("eps", ctypes.c_float), ("dtype", _i32)]


LinearArgs = _args("LinearArgs", ("q", "k", "v", "o", "grad_o", "dq", "dk", "dv"),
                   ("log_decay", "h_in", "h_out", "dh_out", "dh_in", "dlog_decay", "lengths"))
GroupArgs = _args("GroupArgs", ("x", "y", "dy", "dx"), ("w", "b", "stats", "dw", "db", "lengths"))


class RotaryArgs(ctypes.Structure):
    _fields_ = [(r, Rows) for r in ("q", "k", "q_out", "k_out")] + [(p, _vp) for p in ("positions", "offsets", "lengths")]


RotaryArgs.pack = struct.Struct("=15Q").pack

for _op, _desc in (("linear_attention", LinearDesc), ("rotary", RotaryDesc), ("group_norm", GroupDesc)):
    _f = getattr(_lib, _op + "_plan")
    _f.argtypes, _f.restype = [ctypes.POINTER(_desc), ctypes.POINTER(_vp)], ctypes.c_int
    _f = getattr(_lib, _op + "_plan_info")
    _f.argtypes, _f.restype = [_vp, ctypes.POINTER(SeqInfo)], ctypes.c_int
    _f = getattr(_lib, _op + "_plan_destroy")
    _f.argtypes, _f.restype = [_vp], None
    for _way in ("_forward", "_backward"):
        _f = getattr(_lib, _op + _way)
        _f.argtypes, _f.restype = [_vp, _vp, _vp], ctypes.c_int  # the packed block, or a pointer to one


def _linear_shapes(d):
    flat = {name: (d.n, d.t, h * w) for name, h, w in (("q", d.q_heads, d.dk), ("k", d.k_heads, d.dk),
                                                       ("v", d.v_heads, d.dv), ("o", d.heads, d.dv))}
    split = {name + "4": (d.n, d.t, h, w) for name, h, w in (("q", d.q_heads, d.dk), ("k", d.k_heads, d.dk),
                                                             ("v", d.v_heads, d.dv), ("o", d.heads, d.dv))}
    return {**flat, **split, "state": (d.n, d.heads, d.dk, d.dv), "heads": (d.heads,), "n": (d.n,)}


_SHAPES.update({
    "linear_attention": _linear_shapes,
    "rotary": lambda d: {"q": (d.n, d.t, d.q_heads * d.d), "q4": (d.n, d.t, d.q_heads, d.d),
                         "k": (d.n, d.t, d.k_heads * d.d), "k4": (d.n, d.t, d.k_heads, d.d), "positions": (d.n, d.t),
                         "n": (d.n,)},
    "group_norm": lambda d: {"x": (d.n, d.p, d.c), "c": (d.c,), "stats": (d.n, d.groups, 2), "n": (d.n,)},
})


def _plan(op, desc):
    return SeqPlan(op, desc, torch.bfloat16 if desc.dtype == CC3D_BF16 else torch.float32)


# --------------------------------------------------------------------------
# linear_attention
# --------------------------------------------------------------------------

def make_linear_attention_desc(n, t, heads, dk, dv, q_heads=None, k_heads=None, v_heads=None, scale=None,
                               dtype=torch.bfloat16):
    """n sequences of t tokens; `heads` states of dk by dv (1..256); q_heads,
    k_heads, v_heads: heads of q, k, v, divisors of `heads` (default: as many).
    scale: of the result (default: dk ** -0.5)."""
    scale = float(dk) ** -0.5 if scale is None and dk > 0 else 0.0 if scale is None else scale
    return LinearDesc(n, t, heads, heads if q_heads is None else q_heads, heads if k_heads is None else k_heads,
                      heads if v_heads is None else v_heads, dk, dv, scale, _dtype_code(dtype))


def linear_attention_plan(desc):
    return _plan("linear_attention", desc)


def linear_attention_forward(plan, q, k, v, o, log_decay=None, h_in=None, h_out=None, lengths=None, workspace=None,
                             stream=None):
    """o[t] = scale q[t] S[t] with S[t] = exp(log_decay) S[t-1] + k[t]^T v[t]
    from h_in (None: zeros); h_out receives the last state (it may be the h_in
    tensor).  log_decay: [heads] fp32, or None for no decay.  A decode step is
    a plan with t = 1."""
    sh, ty = _plan_of(plan, "linear_attention")
    dev = _device_of(q, "q")
    state = sh["state"]
    args = LinearArgs.pack(
        *_seq(q, "q", sh["q"], ty, dev, sh["q4"]), *_seq(k, "k", sh["k"], ty, dev, sh["k4"]),
        *_seq(v, "v", sh["v"], ty, dev, sh["v4"]), *_seq(o, "o", sh["o"], ty, dev, sh["o4"]),
        0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, _dense(log_decay, "log_decay", sh["heads"], _F32, dev),
        _dense(h_in, "h_in", state, _F32, dev), _dense(h_out, "h_out", state, _F32, dev), 0, 0, 0,
        _dense(lengths, "lengths", sh["n"], _I32, dev), *_space(workspace, plan.info["workspace_bytes"], dev))
    _call(_lib.linear_attention_forward, "linear_attention_forward", plan, args, dev, stream)


def linear_attention_backward(plan, q, k, v, do, log_decay=None, h_in=None, dh_out=None, dq=None, dk=None, dv=None,
                              dlog_decay=None, dh_in=None, lengths=None, workspace=None, stream=None):
    """Gradients of linear_attention_forward from do and dh_out (None: zeros),
    each into the tensor given for it (or none): dq, dk, dv of the plan's dtype,
    summed over the heads that share one; dlog_decay, dh_in fp32."""
    sh, ty = _plan_of(plan, "linear_attention")
    dev = _device_of(q, "q")
    state = sh["state"]
    args = LinearArgs.pack(
        *_seq(q, "q", sh["q"], ty, dev, sh["q4"]), *_seq(k, "k", sh["k"], ty, dev, sh["k4"]),
        *_seq(v, "v", sh["v"], ty, dev, sh["v4"]), 0, 0, 0, *_seq(do, "do", sh["o"], ty, dev, sh["o4"]),
        *_seq(dq, "dq", sh["q"], ty, dev, sh["q4"]), *_seq(dk, "dk", sh["k"], ty, dev, sh["k4"]),
        *_seq(dv, "dv", sh["v"], ty, dev, sh["v4"]), _dense(log_decay, "log_decay", sh["heads"], _F32, dev),
        _dense(h_in, "h_in", state, _F32, dev), 0, _dense(dh_out, "dh_out", state, _F32, dev),
        _dense(dh_in, "dh_in", state, _F32, dev), _dense(dlog_decay, "dlog_decay", sh["heads"], _F32, dev),
        _dense(lengths, "lengths", sh["n"], _I32, dev), *_space(workspace, plan.info["backward_workspace_bytes"], dev))
    _call(_lib.linear_attention_backward, "linear_attention_backward", plan, args, dev, stream)


# --------------------------------------------------------------------------
# rotary
# --------------------------------------------------------------------------

def make_rotary_desc(n, t, q_heads, k_heads, d, rot=None, first=0, layout="half", theta=10000.0, scaling=None, factor=1.0,
                     original=0, fast=32.0, slow=1.0, amplitude=None, dtype=torch.bfloat16):
    """Channels [first, first + rot) (rot None: up to d) of heads of width d are
    turned; k_heads may be 0.  layout: "half" or "interleaved".  scaling: None,
    "linear", "base" or "parts" (see cc3d_heads.h), by `factor`; "parts" also
    takes `original` (trained tokens), `fast` and `slow` (turns), and its default
    amplitude is 0.1 ln(factor) + 1, else 1."""
    code = _code(_SCALINGS, scaling, "scaling")
    if amplitude is None:
        amplitude = 0.1 * math.log(factor) + 1.0 if scaling == "parts" and factor > 0 else 1.0
    return RotaryDesc(n, t, q_heads, k_heads, d, d - first if rot is None else rot, first,
                      _code(_LAYOUTS, layout, "layout"), code, _dtype_code(dtype), theta, factor, original, fast, slow,
                      amplitude)


def rotary_plan(desc):
    return _plan("rotary", desc)


def _rotary(name, plan, q, k, q_out, k_out, positions, offsets, lengths, stream):
    sh, ty = _plan_of(plan, "rotary")
    dev = _device_of(q, "q")
    args = RotaryArgs.pack(
        *_seq(q, "q", sh["q"], ty, dev, sh["q4"]),
        *(_seq(k, "k", sh["k"], ty, dev, sh["k4"]) if k is not None else _NONE),
        *_seq(q_out, "q_out", sh["q"], ty, dev, sh["q4"]),
        *(_seq(k_out, "k_out", sh["k"], ty, dev, sh["k4"]) if k_out is not None else _NONE),
        _dense(positions, "positions", sh["positions"], _I32, dev), _dense(offsets, "offsets", sh["n"], _I32, dev),
        _dense(lengths, "lengths", sh["n"], _I32, dev))
    _call(getattr(_lib, name), name, plan, args, dev, stream)


def rotary_forward(plan, q, k, q_out, k_out, positions=None, offsets=None, lengths=None, stream=None):
    """q_out and k_out: q and k with every head's pairs turned by their token's
    position: positions[n, t] (int32 [N, T]), else offsets[n] + t (int32 [N];
    None: zeros).  An output may be its input.  k and k_out are None in a plan
    without k heads."""
    _rotary("rotary_forward", plan, q, k, q_out, k_out, positions, offsets, lengths, stream)


def rotary_backward(plan, dq_out, dk_out, dq, dk, positions=None, offsets=None, lengths=None, stream=None):
    """Gradients of q and k from those of q_out and k_out: the turn undone."""
    _rotary("rotary_backward", plan, dq_out, dk_out, dq, dk, positions, offsets, lengths, stream)


# --------------------------------------------------------------------------
# group_norm
# --------------------------------------------------------------------------

def make_group_norm_desc(n, p, c, groups, act=None, eps=1e-6, dtype=torch.bfloat16):
    """n samples (frames, or tokens with p = 1) of p positions of c channels
    (1..8192) in `groups` groups; act: None or "silu"."""
    return GroupDesc(n, p, c, groups, _code(_ACTS, act, "act"), eps, _dtype_code(dtype))


def group_norm_plan(desc):
    return _plan("group_norm", desc)


def group_norm_forward(plan, x, y, w=None, b=None, stats=None, lengths=None, workspace=None, stream=None):
    """y = act((x - mean) * rstd * w + b), mean and rstd of each group of a
    sample's valid positions; stats, fp32 [N, groups, 2], receives them."""
    sh, ty = _plan_of(plan, "group_norm")
    dev = _device_of(x, "x")
    args = GroupArgs.pack(
        *_seq(x, "x", sh["x"], ty, dev), *_seq(y, "y", sh["x"], ty, dev), 0, 0, 0, 0, 0, 0,
        _dense(w, "w", sh["c"], ty, dev), _dense(b, "b", sh["c"], ty, dev), _dense(stats, "stats", sh["stats"], _F32, dev),
        0, 0, _dense(lengths, "lengths", sh["n"], _I32, dev), *_space(workspace, plan.info["workspace_bytes"], dev))
    _call(_lib.group_norm_forward, "group_norm_forward", plan, args, dev, stream)


def group_norm_backward(plan, x, dy, w=None, b=None, stats=None, dx=None, dw=None, db=None, lengths=None, workspace=None,
                        stream=None):
    """Gradients of group_norm_forward: dx of the plan's dtype, dw and db fp32;
    each may be None.  stats: what the forward call wrote (None: computed
    again)."""
    sh, ty = _plan_of(plan, "group_norm")
    dev = _device_of(x, "x")
    args = GroupArgs.pack(
        *_seq(x, "x", sh["x"], ty, dev), 0, 0, 0, *_seq(dy, "dy", sh["x"], ty, dev), *_seq(dx, "dx", sh["x"], ty, dev),
        _dense(w, "w", sh["c"], ty, dev), _dense(b, "b", sh["c"], ty, dev), _dense(stats, "stats", sh["stats"], _F32, dev),
        _dense(dw, "dw", sh["c"], _F32, dev), _dense(db, "db", sh["c"], _F32, dev),
        _dense(lengths, "lengths", sh["n"], _I32, dev), *_space(workspace, plan.info["backward_workspace_bytes"], dev))
    _call(_lib.group_norm_backward, "group_norm_backward", plan, args, dev, stream)
