"""Plain 64-bit forms of the operators on heads and groups (linear_attention,
rotary, group_norm), forward and by-formula gradients, on the CPU, and the
error bounds that the GPU tests use.

With ``mag=True`` a linear form is evaluated on absolute values, which bounds
the sum of the absolute values of the terms of each result.
"""
import torch

F64 = torch.float64
EPS32 = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # of a value, at most


def lens(lengths, n, t):
    if lengths is None:
        return [t] * n
    return [min(max(int(v), 0), t) for v in lengths]


# ------------------------------------------------------ linear attention

def _heads(x, h):
    return x.repeat_interleave(h // x.shape[2], 2)


def linear(q, k, v, g, scale, h_in=None, lengths=None, heads=None, mag=False):
    """(o, h_out), token by token.  q, k, v [N, T, H', D]; g [H]."""
    n, t, _, dk = q.shape
    dv = v.shape[3]
    if mag:
        q, k, v, scale = q.abs(), k.abs(), v.abs(), abs(scale)
        h_in = None if h_in is None else h_in.abs()
    q, k, v = _heads(q, heads), _heads(k, heads), _heads(v, heads)
    f = torch.exp(g)[:, None, None]
    o, last = torch.zeros(n, t, heads, dv, dtype=F64), torch.zeros(n, heads, dk, dv, dtype=F64)
    for i, ln in enumerate(lens(lengths, n, t)):
        s = torch.zeros(heads, dk, dv, dtype=F64) if h_in is None else h_in[i]
        for p in range(ln):
            s = f * s + k[i, p][..., None] * v[i, p][:, None]
            o[i, p] = scale * (q[i, p][..., None] * s).sum(1)
        last[i] = s
    return o, last


def linear_grad(q, k, v, g, scale, do, h_in=None, dh_out=None, lengths=None, heads=None, mag=False):
    """dict of dq, dk, dv, dlog_decay, dh_in: the states walked back."""
    n, t, _, dk = q.shape
    dv = v.shape[3]
    counts = [x.shape[2] for x in (q, k, v)]
    if mag:
        q, k, v, do, scale = q.abs(), k.abs(), v.abs(), do.abs(), abs(scale)
        h_in = None if h_in is None else h_in.abs()
        dh_out = None if dh_out is None else dh_out.abs()
    q, k, v = _heads(q, heads), _heads(k, heads), _heads(v, heads)
    f = torch.exp(g)[:, None, None]
    dq, dkk, dvv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, dh = torch.zeros(heads, dtype=F64), torch.zeros(n, heads, dk, dv, dtype=F64)
    for i, ln in enumerate(lens(lengths, n, t)):
        s = [torch.zeros(heads, dk, dv, dtype=F64) if h_in is None else h_in[i]]
        for p in range(ln):
            s.append(f * s[-1] + k[i, p][..., None] * v[i, p][:, None])
        gs = torch.zeros(heads, dk, dv, dtype=F64) if dh_out is None else dh_out[i]
        for p in range(ln - 1, -1, -1):
            gs = gs + scale * q[i, p][..., None] * do[i, p][:, None]
            dq[i, p] = scale * (s[p + 1] * do[i, p][:, None]).sum(2)
            dkk[i, p] = (gs * v[i, p][:, None]).sum(2)
            dvv[i, p] = (gs * k[i, p][..., None]).sum(1)
            dg += (gs * f * s[p]).sum((1, 2))
            gs = gs * f
        dh[i] = gs

    def fold(x, c):
        return x.reshape(n, t, c, heads // c, x.shape[3]).sum(3)

    return {"dq": fold(dq, counts[0]), "dk": fold(dkk, counts[1]), "dv": fold(dvv, counts[2]), "dlog_decay": dg,
            "dh_in": dh}


def linear_depth(t, dk, dv):
    """Roundings of 2^-24 on the way to a term's place in a result: a factor
    exp(g d) of d tokens carries the rounding of its exponent, |g d| log2(e) <=
    150 where fp32 holds it, twice, and so across blocks: 300; sums over the
    width of a head, over 64 tokens and over the blocks and segments."""
    return 300 + 2 * (dk + dv) + 128 + t


def linear_bound(mag, value, dtype, depth, inner):
    """|error| of a result: `inner` of the terms for what is rounded between
    two products, depth roundings of 32 bits, and the result's own."""
    return (inner + depth * EPS32) * mag + HALF_STEP[dtype] * (value.abs() + (inner + depth * EPS32) * mag)


# ---------------------------------------------------------------- rotary

def frequencies(rot, theta=10000.0, scaling=None, factor=1.0, original=0, fast=32.0, slow=1.0):
    import math
    if scaling == "base":
        theta *= factor ** (rot / (rot - 2))
    f = [theta ** (-2.0 * j / rot) for j in range(rot // 2)]
    if scaling == "linear":
        f = [v / factor for v in f]
    if scaling == "parts":
        keep = [min(1.0, max(0.0, (original * v / (2 * math.pi) - slow) / (fast - slow))) for v in f]
        f = [v * k + v / factor * (1 - k) for v, k in zip(f, keep)]
    return torch.tensor(f, dtype=F64)


def rotary(x, pos, f, first, layout, amplitude=1.0, back=False, lengths=None, mag=False):
    """x [N, T, H, D], pos [N, T]: (result, sum of the terms' absolute values)."""
    n, t, _, _ = x.shape
    rot = 2 * f.shape[0]
    ang = pos.to(F64)[..., None] * f
    c, s = (amplitude * torch.cos(ang))[:, :, None], (amplitude * torch.sin(ang))[:, :, None]
    if back:
        s = -s
    y = x.clone()
    at = torch.arange(rot // 2)
    ia, ib = (first + at, first + rot // 2 + at) if layout == "half" else (first + 2 * at, first + 2 * at + 1)
    a, b = x[..., ia], x[..., ib]
    if mag:
        y = x.abs()
        y[..., ia] = y[..., ib] = abs(amplitude) * (a.abs() + b.abs())
    else:
        y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    for i, ln in enumerate(lens(lengths, n, t)):
        y[i, ln:] = 0
    return y


# ------------------------------------------------------------ group norm

def silu_slope(v):
    s = torch.sigmoid(v)
    return s * (1 + v * (1 - s))


def group(x, groups, w, b, act, eps, lengths=None, dy=None):
    """dict of y and stats, with their bounds per rounding (y_unit,
    stats_unit), or with dy of dx, dw, db and theirs.

    A unit is what one relative rounding of 2^-24 in the elements, the mean or
    the sums moves a result by: an element off its mean by d is known to about
    max|x| of the group, rstd to max|x| rstd, so xn to (1 + max|x| rstd)
    (1 + |xn|)."""
    n, p, c = x.shape
    cg = c // groups
    y, dx = torch.zeros_like(x), torch.zeros_like(x)
    uy, ux = torch.zeros_like(x), torch.zeros_like(x)
    stats, us = torch.zeros(n, groups, 2, dtype=F64), torch.zeros(n, groups, 2, dtype=F64)
    one = torch.ones(c, dtype=F64)
    w, b = (one if w is None else w), (0 * one if b is None else b)
    dw, db, uw, ub = (torch.zeros(c, dtype=F64) for _ in range(4))
    for i, ln in enumerate(lens(lengths, n, p)):
        for g in range(groups if ln else 0):
            at = slice(g * cg, (g + 1) * cg)
            v = x[i, :ln, at]
            mean = v.mean()
            rs = 1 / torch.sqrt(((v - mean) ** 2).mean() + eps)
            stats[i, g, 0], stats[i, g, 1] = mean, rs
            big = v.abs().max()
            us[i, g, 0], us[i, g, 1] = big, rs * (1 + big * rs)
            xn = (v - mean) * rs
            un = (1 + big * rs) * (1 + xn.abs())
            u = xn * w[at] + b[at]
            uu = un * w[at].abs() + b[at].abs() + u.abs()
            sl = silu_slope(u) if act else torch.ones_like(u)
            y[i, :ln, at] = u * torch.sigmoid(u) if act else u
            # (the activation's slope is at most 1.1; its exponential's argument is |u|, its own roundings a few)
            uy[i, :ln, at] = 1.1 * uu + (8 + u.abs()) * u.abs() if act else uu
            if dy is None:
                continue
            d = dy[i, :ln, at] * sl
            # (the slope's slope is at most 0.5)
            ud = dy[i, :ln, at].abs() * ((0.5 * uu + 8 + u.abs()) if act else 1) + d.abs()
            dw[at] += (d * xn).sum(0)
            db[at] += d.sum(0)
            uw[at] += (ud * xn.abs() + d.abs() * un).sum(0)
            ub[at] += ud.sum(0)
            gw, ugw = d * w[at], ud * w[at].abs()
            dx[i, :ln, at] = rs * (gw - gw.mean() - xn * (gw * xn).mean())
            m2, um2 = (gw * xn).mean().abs(), (ugw * xn.abs() + gw.abs() * un).mean()
            terms = gw.abs() + gw.abs().mean() + xn.abs() * (gw * xn).abs().mean()
            ux[i, :ln, at] = rs * (ugw + ugw.mean() + un * m2 + xn.abs() * um2 + terms * (1 + big * rs))
    if dy is None:
        return {"y": y, "stats": stats, "y_unit": uy, "stats_unit": us}
    return {"dx": dx, "dw": dw, "db": db, "dx_unit": ux, "dw_unit": uw, "db_unit": ub}
