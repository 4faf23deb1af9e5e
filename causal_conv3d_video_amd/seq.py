"""Streaming state-space operators: Python binding of include/cc3d_seq.h.

  causal_conv1d   short cached causal convolution of each channel
  selective_scan  selective state space recurrence
  norm_join       norm, gate, residual scale and sum, then norm and activation

Each has a plan (host metadata only), a forward and a backward call, with the
arguments' shapes channels last: activations [N, T, C], B and C of the scan
[N, T, G, S] (or [N, T, G*S]), states [N, C, S] fp32, convolution taps [K, C].
The last dimension of a tensor is contiguous; the others of an activation may
have any strides, so a part of a wider projection is passed in place.
``lengths`` is an int32 CUDA tensor [N] of valid tokens, or None.  Outputs are
caller-owned tensors, and so is the workspace: a CUDA tensor of at least
plan.info["workspace_bytes"] (backward: "backward_workspace_bytes") bytes,
None when that is 0.  Calls are asynchronous on ``stream`` (default: the
current torch stream); a refused one raises CC3DError, a tensor of the wrong
kind TypeError or ValueError.
"""
import ctypes
import struct

import torch

from . import CC3D_BF16, CC3D_F32, CC3D_OK, CC3DError, _lib

SEQ_EXPORTED_SYMBOLS = tuple(
    "%s_%s" % (op, what) for op in ("causal_conv1d", "selective_scan", "norm_join")
    for what in ("plan", "plan_info", "plan_destroy", "forward", "backward"))

_i32, _i64, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
_ACTS = {None: 0, "silu": 1}
_NORMS = {None: 0, "rms": 1, "layer": 2}
_DTYPES = {torch.float32: CC3D_F32, torch.bfloat16: CC3D_BF16}


def _code(table, key, what):
    try:
        return table[key]
    except (KeyError, TypeError):
        raise ValueError("%s must be one of %s, got %r" % (what, sorted(table, key=str), key)) from None


def _dtype_code(dtype):
    if dtype not in _DTYPES:
        raise TypeError("dtype must be torch.bfloat16 or torch.float32")
    return _DTYPES[dtype]


class Rows(ctypes.Structure):
    _fields_ = [("p", _vp), ("batch", _i64), ("row", _i64)]


class SeqInfo(ctypes.Structure):
    _fields_ = [("workspace_bytes", _i64), ("backward_workspace_bytes", _i64), ("chunks", _i32),
                ("backward_chunks", _i32)]


class Conv1dDesc(ctypes.Structure):
    _fields_ = [(name, _i32) for name in ("n", "t", "c", "k", "act", "dtype")]


class ScanDesc(ctypes.Structure):
    _fields_ = [(name, _i32) for name in ("n", "t", "d", "states", "groups", "softplus", "dtype")]


class JoinDesc(ctypes.Structure):
    _fields_ = [("rows", _i64), ("gate_rows", _i64)] + [(n, _i32) for n in ("c", "post", "pre", "act", "gate_act")] + [
        ("eps", ctypes.c_float), ("dtype", _i32)]


def _args(name, rows, pointers):
    """An argument block: views first, then pointers and the workspace.  Every
    field is 64 bits wide, so a call packs one as plain numbers (``pack``)."""
    fields = [(r, Rows) for r in rows] + [(p, _vp) for p in pointers] + [("workspace", _vp), ("workspace_bytes", _i64)]
    block = type(name, (ctypes.Structure,), {"_fields_": fields})
    block.pack = struct.Struct("=%dQ" % (3 * len(rows) + len(pointers) + 2)).pack
    return block


Conv1dArgs = _args("Conv1dArgs", ("x", "y", "dy", "dx"),
                   ("w", "b", "cache_in", "cache_out", "dcache_out", "dcache_in", "dw", "db", "lengths"))
ScanArgs = _args("ScanArgs", ("u", "dt", "b", "c", "z", "y", "dy", "du", "ddt", "dz", "db", "dc"),
                 ("a", "d", "dt_bias", "h_in", "h_out", "dh_out", "dh_in", "da", "dd", "ddt_bias", "lengths"))
JoinArgs = _args("JoinArgs", ("y", "residual", "gate", "x_out", "h_out", "dx_out", "dh", "dy", "dresidual", "dgate"),
                 ("scale", "post_w", "post_b", "pre_w", "pre_b", "dscale", "dpost_w", "dpost_b", "dpre_w", "dpre_b"))

for _op, _desc, _blk in (("causal_conv1d", Conv1dDesc, Conv1dArgs), ("selective_scan", ScanDesc, ScanArgs),
                         ("norm_join", JoinDesc, JoinArgs)):
    _f = getattr(_lib, _op + "_plan")
    _f.argtypes, _f.restype = [ctypes.POINTER(_desc), ctypes.POINTER(_vp)], ctypes.c_int
    _f = getattr(_lib, _op + "_plan_info")
    _f.argtypes, _f.restype = [_vp, ctypes.POINTER(SeqInfo)], ctypes.c_int
    _f = getattr(_lib, _op + "_plan_destroy")
    _f.argtypes, _f.restype = [_vp], None
    for _way in ("_forward", "_backward"):
        _f = getattr(_lib, _op + _way)
        _f.argtypes, _f.restype = [_vp, _vp, _vp], ctypes.c_int  # the packed block, or a pointer to one


class SeqPlan:
    """Owns a plan handle of one operator (host metadata only)."""

    def __init__(self, op, desc, dtype):
        self.op, self.desc, self.dtype = op, desc, dtype
        self.handle = None
        h = _vp()
        st = getattr(_lib, op + "_plan")(ctypes.byref(desc), ctypes.byref(h))
        if st != CC3D_OK:
            raise CC3DError(st, op + "_plan")
        self.handle = h.value
        info = SeqInfo()
        getattr(_lib, op + "_plan_info")(self.handle, ctypes.byref(info))
        self.info = {name: getattr(info, name) for name, _ in SeqInfo._fields_}
        self.shapes = _SHAPES[op](desc)

    def close(self):
        if self.handle:
            getattr(_lib, self.op + "_plan_destroy")(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# Shapes of a plan's tensors, worked out once.
_SHAPES = {
    "causal_conv1d": lambda d: {"seq": (d.n, d.t, d.c), "cache": (d.n, d.k - 1, d.c), "w": (d.k, d.c), "c": (d.c,),
                                "n": (d.n,)},
    "selective_scan": lambda d: {"seq": (d.n, d.t, d.d), "bc": (d.n, d.t, d.groups * d.states),
                                 "split": (d.n, d.t, d.groups, d.states), "state": (d.n, d.d, d.states),
                                 "a": (d.d, d.states), "c": (d.d,), "n": (d.n,)},
    "norm_join": lambda d: {"rows": (d.rows, d.c), "gates": (-(-d.rows // d.gate_rows), d.c), "c": (d.c,)},
}

_F32, _I32 = torch.float32, torch.int32
_Tensor = torch.Tensor


def _plan_of(plan, op):
    if not isinstance(plan, SeqPlan) or plan.op != op:
        raise TypeError("expected a plan of %s_plan" % op)
    return plan.shapes, plan.dtype


def _check(t, name, dtype, device):
    """The reason a tensor is refused, or nothing when kind, type and device are right."""
    if not isinstance(t, _Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA (HIP) tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.get_device() != device:
        raise ValueError("%s is on %s, the other tensors on cuda:%d" % (name, t.device, device))


def _device_of(t, name):
    if not isinstance(t, _Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA (HIP) tensor" % name)
    return t.get_device()


def _dense(t, name, shape, dtype, device):
    """The address of a dense tensor of exactly this shape; 0 for None."""
    if t is None:
        return 0
    if not (isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == device):
        _check(t, name, dtype, device)
    if t.shape != shape or not t.is_contiguous():
        raise ValueError("%s: expected a dense %s tensor, got shape %s strides %s"
                         % (name, shape, tuple(t.shape), tuple(t.stride())))
    return t.data_ptr()


_NONE = (0, 0, 0)


def _seq(t, name, shape, dtype, device, split=None):
    """(address, batch stride, row stride) of a view of [N, T, C]; split: [N, T, G, S] is taken too."""
    if t is None:
        return _NONE
    if not (isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == device):
        _check(t, name, dtype, device)
    st = t.stride()
    if t.shape == shape:
        ok = st[2] == 1 or shape[2] == 1
    else:
        ok = split is not None and t.shape == split and (st[3] == 1 or split[3] == 1) and \
            (st[2] == split[3] or split[2] == 1)
    if not ok:
        raise ValueError("%s: expected %s with a contiguous last dimension, got shape %s strides %s"
                         % (name, shape if split is None else split, tuple(t.shape), st))
    return t.data_ptr(), st[0], st[1]


def _rows(t, name, shape, dtype, device):
    """(address, 0, row stride) of a view of [rows, C] of a tensor [..., C] whose leading dimensions step evenly."""
    if t is None:
        return _NONE
    if not (isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == device):
        _check(t, name, dtype, device)
    rows, c = shape
    if t.is_contiguous() and t.shape[-1:] == (c,) and t.numel() == rows * c:
        return t.data_ptr(), 0, c
    dims, st = t.shape, t.stride()
    ok = t.dim() >= 1 and dims[-1] == c and t.numel() == rows * c and (st[-1] == 1 or c == 1)
    row, n = c, 1
    if ok:
        for i in range(t.dim() - 2, -1, -1):
            if dims[i] == 1:
                continue
            if n == 1:
                row = st[i]
            elif st[i] != row * n:
                ok = False
                break
            n *= dims[i]
    if not ok:
        raise ValueError("%s: expected %d evenly spaced rows of %d contiguous elements, got shape %s strides %s"
                         % (name, rows, c, tuple(dims), st))
    return t.data_ptr(), 0, row


def _space(t, nbytes, device):
    """(address, bytes) of the workspace."""
    if t is None:
        if nbytes > 0:
            raise ValueError("this call needs a workspace of %d bytes" % nbytes)
        return 0, 0
    if not isinstance(t, _Tensor) or not t.is_cuda or not t.is_contiguous():
        raise TypeError("workspace must be a contiguous CUDA (HIP) tensor")
    have = t.numel() * t.element_size()
    if have < nbytes:
        raise ValueError("workspace holds %d bytes, the plan needs %d" % (have, nbytes))
    if t.get_device() != device:
        raise ValueError("workspace is on %s, the other tensors on cuda:%d" % (t.device, device))
    return t.data_ptr(), have


def _current_stream(device):
    return torch.cuda.current_stream(device).cuda_stream


# The same number without the Stream object around it (1.1 us of a call), where this torch has it.
_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)


def _call(fn, what, plan, args, device, stream):
    if stream is None:
        handle = _stream_of(device)
    else:
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if device != torch.cuda.current_device():
        with torch.cuda.device(device):
            st = fn(plan.handle, args, handle)
    else:
        st = fn(plan.handle, args, handle)
    if st != CC3D_OK:
        raise CC3DError(st, what)


# --------------------------------------------------------------------------
# causal_conv1d
# --------------------------------------------------------------------------

def make_conv1d_desc(n, t, c, k, act=None, dtype=torch.bfloat16):
    """n sequences of t tokens of c channels, k taps (1..8); act: None or "silu"."""
    return Conv1dDesc(n, t, c, k, _code(_ACTS, act, "act"), _dtype_code(dtype))


def causal_conv1d_plan(desc):
    return SeqPlan("causal_conv1d", desc, torch.bfloat16 if desc.dtype == CC3D_BF16 else torch.float32)


def causal_conv1d_forward(plan, x, w, b, y, cache_in=None, cache_out=None, lengths=None, stream=None):
    """y = act(b + sum_k w[k] * [cache_in; x][t + k]); cache_out receives the
    last k - 1 tokens of [cache_in; x].  b may be None."""
    sh, ty = _plan_of(plan, "causal_conv1d")
    dev = _device_of(x, "x")
    seq, cache = sh["seq"], sh["cache"]
    args = Conv1dArgs.pack(
        *_seq(x, "x", seq, ty, dev), *_seq(y, "y", seq, ty, dev), 0, 0, 0, 0, 0, 0, _dense(w, "w", sh["w"], ty, dev),
        _dense(b, "b", sh["c"], ty, dev), _dense(cache_in, "cache_in", cache, ty, dev),
        _dense(cache_out, "cache_out", cache, ty, dev), 0, 0, 0, 0, _dense(lengths, "lengths", sh["n"], _I32, dev), 0, 0)
    _call(_lib.causal_conv1d_forward, "causal_conv1d_forward", plan, args, dev, stream)


def causal_conv1d_backward(plan, x, w, b, dy, dx=None, dw=None, db=None, cache_in=None, dcache_out=None,
                           dcache_in=None, lengths=None, workspace=None, stream=None):
    """Gradients of causal_conv1d_forward into dx, dcache_in (the plan's
    dtype) and dw, db (fp32); each may be None."""
    sh, ty = _plan_of(plan, "causal_conv1d")
    dev = _device_of(x, "x")
    seq, cache = sh["seq"], sh["cache"]
    args = Conv1dArgs.pack(
        *_seq(x, "x", seq, ty, dev), 0, 0, 0, *_seq(dy, "dy", seq, ty, dev), *_seq(dx, "dx", seq, ty, dev),
        _dense(w, "w", sh["w"], ty, dev), _dense(b, "b", sh["c"], ty, dev), _dense(cache_in, "cache_in", cache, ty, dev),
        0, _dense(dcache_out, "dcache_out", cache, ty, dev), _dense(dcache_in, "dcache_in", cache, ty, dev),
        _dense(dw, "dw", sh["w"], _F32, dev), _dense(db, "db", sh["c"], _F32, dev),
        _dense(lengths, "lengths", sh["n"], _I32, dev), *_space(workspace, plan.info["backward_workspace_bytes"], dev))
    _call(_lib.causal_conv1d_backward, "causal_conv1d_backward", plan, args, dev, stream)


# --------------------------------------------------------------------------
# selective_scan
# --------------------------------------------------------------------------

def make_scan_desc(n, t, d, states, groups=1, softplus=True, dtype=torch.bfloat16):
    """n sequences of t tokens of d channels with `states` states each (1..64),
    B and C shared by the d / groups channels of a group."""
    return ScanDesc(n, t, d, states, groups, int(bool(softplus)), _dtype_code(dtype))


def selective_scan_plan(desc):
    return SeqPlan("selective_scan", desc, torch.bfloat16 if desc.dtype == CC3D_BF16 else torch.float32)


def selective_scan_forward(plan, u, dt, a, b, c, y, d=None, z=None, dt_bias=None, h_in=None, h_out=None, lengths=None,
                           workspace=None, stream=None):
    """y = (sum_s C h + d u) silu(z) with h = exp(delta a) h + delta u B,
    delta = softplus(dt + dt_bias), from h_in; h_out receives the last state
    (it may be the h_in tensor).  A decode step is a plan with t = 1."""
    sh, ty = _plan_of(plan, "selective_scan")
    dev = _device_of(u, "u")
    seq, bc, split, state, ch = sh["seq"], sh["bc"], sh["split"], sh["state"], sh["c"]
    args = ScanArgs.pack(
        *_seq(u, "u", seq, ty, dev), *_seq(dt, "dt", seq, ty, dev), *_seq(b, "b", bc, ty, dev, split),
        *_seq(c, "c", bc, ty, dev, split), *_seq(z, "z", seq, ty, dev), *_seq(y, "y", seq, ty, dev),
        0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0,
        _dense(a, "a", sh["a"], _F32, dev), _dense(d, "d", ch, _F32, dev), _dense(dt_bias, "dt_bias", ch, _F32, dev),
        _dense(h_in, "h_in", state, _F32, dev), _dense(h_out, "h_out", state, _F32, dev), 0, 0, 0, 0, 0,
        _dense(lengths, "lengths", sh["n"], _I32, dev), *_space(workspace, plan.info["workspace_bytes"], dev))
    _call(_lib.selective_scan_forward, "selective_scan_forward", plan, args, dev, stream)


def selective_scan_backward(plan, u, dt, a, b, c, dy, d=None, z=None, dt_bias=None, h_in=None, dh_out=None, du=None,
                            ddt=None, da=None, db=None, dc=None, dd=None, dz=None, ddt_bias=None, dh_in=None,
                            lengths=None, workspace=None, stream=None):
    """Gradients of selective_scan_forward, each into the tensor given for it
    (or none): du, ddt, db, dc, dz of the plan's dtype, da, dd, ddt_bias,
    dh_in fp32.  dh_out: gradient of h_out."""
    sh, ty = _plan_of(plan, "selective_scan")
    dev = _device_of(u, "u")
    seq, bc, split, state, ch = sh["seq"], sh["bc"], sh["split"], sh["state"], sh["c"]
    args = ScanArgs.pack(
        *_seq(u, "u", seq, ty, dev), *_seq(dt, "dt", seq, ty, dev), *_seq(b, "b", bc, ty, dev, split),
        *_seq(c, "c", bc, ty, dev, split), *_seq(z, "z", seq, ty, dev), 0, 0, 0, *_seq(dy, "dy", seq, ty, dev),
        *_seq(du, "du", seq, ty, dev), *_seq(ddt, "ddt", seq, ty, dev), *_seq(dz, "dz", seq, ty, dev),
        *_seq(db, "db", bc, ty, dev, split), *_seq(dc, "dc", bc, ty, dev, split),
        _dense(a, "a", sh["a"], _F32, dev), _dense(d, "d", ch, _F32, dev), _dense(dt_bias, "dt_bias", ch, _F32, dev),
        _dense(h_in, "h_in", state, _F32, dev), 0, _dense(dh_out, "dh_out", state, _F32, dev),
        _dense(dh_in, "dh_in", state, _F32, dev), _dense(da, "da", sh["a"], _F32, dev), _dense(dd, "dd", ch, _F32, dev),
        _dense(ddt_bias, "ddt_bias", ch, _F32, dev), _dense(lengths, "lengths", sh["n"], _I32, dev),
        *_space(workspace, plan.info["backward_workspace_bytes"], dev))
    _call(_lib.selective_scan_backward, "selective_scan_backward", plan, args, dev, stream)


# --------------------------------------------------------------------------
# norm_join
# --------------------------------------------------------------------------

def make_join_desc(rows, c, post="rms", pre="rms", act=None, gate_act=None, gate_rows=1, eps=1e-6,
                   dtype=torch.bfloat16):
    """rows of c channels (1..8192); post and pre: None, "rms" or "layer", the
    norm of y and that of the sum; act after the second norm and gate_act of
    the gate: None or "silu"; gate_rows rows share a gate row."""
    return JoinDesc(rows, gate_rows, c, _code(_NORMS, post, "post"), _code(_NORMS, pre, "pre"), _code(_ACTS, act, "act"),
                    _code(_ACTS, gate_act, "gate_act"), eps, _dtype_code(dtype))


def norm_join_plan(desc):
    return SeqPlan("norm_join", desc, torch.bfloat16 if desc.dtype == CC3D_BF16 else torch.float32)


def norm_join_forward(plan, y, residual, x_out=None, h_out=None, gate=None, scale=None, post_w=None, post_b=None,
                      pre_w=None, pre_b=None, stream=None):
    """x_out = residual + scale * gate_act(gate) * (norm(y) * post_w + post_b);
    h_out = act(norm(x_out) * pre_w + pre_b).  y None: x_out is residual (a
    block's first norm); residual None: zeros."""
    sh, ty = _plan_of(plan, "norm_join")
    dev = _device_of(y, "y") if y is not None else _device_of(residual, "residual")
    rows, c = sh["rows"], sh["c"]
    args = JoinArgs.pack(
        *_rows(y, "y", rows, ty, dev), *_rows(residual, "residual", rows, ty, dev),
        *_rows(gate, "gate", sh["gates"], ty, dev), *_rows(x_out, "x_out", rows, ty, dev),
        *_rows(h_out, "h_out", rows, ty, dev), 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0,
        _dense(scale, "scale", c, ty, dev), _dense(post_w, "post_w", c, ty, dev), _dense(post_b, "post_b", c, ty, dev),
        _dense(pre_w, "pre_w", c, ty, dev), _dense(pre_b, "pre_b", c, ty, dev), 0, 0, 0, 0, 0, 0, 0)
    _call(_lib.norm_join_forward, "norm_join_forward", plan, args, dev, stream)


def norm_join_backward(plan, y, residual, dx_out=None, dh=None, gate=None, scale=None, post_w=None, post_b=None,
                       pre_w=None, pre_b=None, dy=None, dresidual=None, dgate=None, dscale=None, dpost_w=None,
                       dpost_b=None, dpre_w=None, dpre_b=None, workspace=None, stream=None):
    """Gradients of norm_join_forward from dx_out and dh (either may be None):
    dy, dresidual, dgate of the plan's dtype, the others fp32; each may be
    None."""
    sh, ty = _plan_of(plan, "norm_join")
    dev = _device_of(y, "y") if y is not None else _device_of(residual, "residual")
    rows, gates, c = sh["rows"], sh["gates"], sh["c"]
    args = JoinArgs.pack(
        *_rows(y, "y", rows, ty, dev), *_rows(residual, "residual", rows, ty, dev), *_rows(gate, "gate", gates, ty, dev),
        0, 0, 0, 0, 0, 0, *_rows(dx_out, "dx_out", rows, ty, dev), *_rows(dh, "dh", rows, ty, dev),
        *_rows(dy, "dy", rows, ty, dev), *_rows(dresidual, "dresidual", rows, ty, dev),
        *_rows(dgate, "dgate", gates, ty, dev),
        _dense(scale, "scale", c, ty, dev), _dense(post_w, "post_w", c, ty, dev), _dense(post_b, "post_b", c, ty, dev),
        _dense(pre_w, "pre_w", c, ty, dev), _dense(pre_b, "pre_b", c, ty, dev), _dense(dscale, "dscale", c, _F32, dev),
        _dense(dpost_w, "dpost_w", c, _F32, dev), _dense(dpost_b, "dpost_b", c, _F32, dev),
        _dense(dpre_w, "dpre_w", c, _F32, dev), _dense(dpre_b, "dpre_b", c, _F32, dev),
        *_space(workspace, plan.info["backward_workspace_bytes"], dev))
    _call(_lib.norm_join_backward, "norm_join_backward", plan, args, dev, stream)
