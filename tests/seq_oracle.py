"""Plain 64-bit forms of the sequence operators (causal_conv1d,
selective_scan, norm_join), forward and by-formula gradients, token by token
on the CPU, and the error bounds that the GPU tests use.

Each function takes float64 tensors.  With ``mag=True`` it evaluates the same
formula on absolute values (every difference a sum, every activation's slope
its bound), which bounds the sum of the absolute values of the terms of each
result.  An fp32 evaluation in any order of a chain of `depth` operations
differs from the exact value by at most about depth * 2**-24 times that sum.
"""
import torch

EPS32 = 2.0 ** -24   # half a unit in the last place of 1 in fp32
F64 = torch.float64


def silu(v):
    return v * torch.sigmoid(v)


def silu_slope(v):
    s = torch.sigmoid(v)
    return s * (1 + v * (1 - s))


SLOPE_MAX = 1.1  # |silu'| <= 1.0998


def softplus(v):
    return torch.where(v > 30, v, torch.log1p(torch.exp(torch.clamp(v, max=30.0))))


def lens(lengths, n, t):
    if lengths is None:
        return [t] * n
    return [min(max(int(v), 0), t) for v in lengths]


# ---------------------------------------------------------------- conv1d

def conv1d(x, w, b, act, cache=None, lengths=None, mag=False):
    """(y, cache_out, p): p is the argument of the activation (zero outside)."""
    n, t, c = x.shape
    k = w.shape[0]
    if mag:
        x, w = x.abs(), w.abs()
        b = None if b is None else b.abs()
        cache = None if cache is None else cache.abs()
    y, p = torch.zeros(n, t, c, dtype=F64), torch.zeros(n, t, c, dtype=F64)
    tail = torch.zeros(n, k - 1, c, dtype=F64)
    for i, ln in enumerate(lens(lengths, n, t)):
        head = torch.zeros(k - 1, c, dtype=F64) if cache is None else cache[i]
        z = torch.cat([head, x[i, :ln]])
        for q in range(ln):
            v = torch.zeros(c, dtype=F64) if b is None else b.clone()
            for j in range(k):
                v = v + w[j] * z[q + j]
            p[i, q] = v
            y[i, q] = silu(v) if act and not mag else v
        tail[i] = z[ln:ln + k - 1]
    return y, tail, p


def conv1d_grad(x, w, b, act, dy, cache=None, dtail=None, lengths=None, mag=False):
    """Gradients dx, dw, db, dcache."""
    n, t, c = x.shape
    k = w.shape[0]
    p = conv1d(x, w, b, act, cache, lengths)[2]
    if mag:
        x, w, dy = x.abs(), w.abs(), dy.abs()
        cache = None if cache is None else cache.abs()
        dtail = None if dtail is None else dtail.abs()
    dx = torch.zeros(n, t, c, dtype=F64)
    dw, db = torch.zeros(k, c, dtype=F64), torch.zeros(c, dtype=F64)
    dcache = torch.zeros(n, k - 1, c, dtype=F64)
    for i, ln in enumerate(lens(lengths, n, t)):
        head = torch.zeros(k - 1, c, dtype=F64) if cache is None else cache[i]
        z = torch.cat([head, x[i, :ln]])
        dz = torch.zeros_like(z)
        if dtail is not None:
            dz[ln:ln + k - 1] += dtail[i]
        for q in range(ln):
            g = dy[i, q] * ((SLOPE_MAX if mag else silu_slope(p[i, q])) if act else 1.0)
            db += g
            for j in range(k):
                dz[q + j] += w[j] * g
                dw[j] += g * z[q + j]
        dcache[i] = dz[:k - 1]
        dx[i, :ln] = dz[k - 1:]
    return dx, dw, db, dcache


# ------------------------------------------------------------------ scan

def scan(u, dt, a, b, c, d=None, z=None, bias=None, h_in=None, lengths=None, use_softplus=True, mag=False):
    """(y, h_out, kept): b and c are [N, T, G, S]; kept[i][t] is the state before token t of sequence i."""
    n, t, ch = u.shape
    s, g = a.shape[1], b.shape[2]
    grp = torch.arange(ch) // (ch // g)
    y = torch.zeros(n, t, ch, dtype=F64)
    h_out = torch.zeros(n, ch, s, dtype=F64)
    kept = []
    ab = (lambda v: v.abs()) if mag else (lambda v: v)
    for i, ln in enumerate(lens(lengths, n, t)):
        h = torch.zeros(ch, s, dtype=F64) if h_in is None else ab(h_in[i])
        states = [h]
        for q in range(ln):
            raw = dt[i, q] if bias is None else dt[i, q] + bias
            delta = softplus(raw) if use_softplus else raw
            h = torch.exp(delta[:, None] * a) * h + (ab(delta) * ab(u[i, q]))[:, None] * ab(b[i, q])[grp]
            states.append(h)
            v = (h * ab(c[i, q])[grp]).sum(-1)
            if d is not None:
                v = v + ab(d) * ab(u[i, q])
            if z is not None:
                v = v * ab(silu(z[i, q]))
            y[i, q] = v
        h_out[i] = h
        kept.append(states)
    return y, h_out, kept


def scan_grad(u, dt, a, b, c, dy, d=None, z=None, bias=None, h_in=None, dh_out=None, lengths=None,
              use_softplus=True, mag=False):
    """Gradients as a dict."""
    n, t, ch = u.shape
    s, g = a.shape[1], b.shape[2]
    grp = torch.arange(ch) // (ch // g)
    kept = scan(u, dt, a, b, c, d, z, bias, h_in, lengths, use_softplus, mag)[2]
    ab = (lambda v: v.abs()) if mag else (lambda v: v)
    out = {k: torch.zeros(v.shape, dtype=F64) for k, v in
           (("du", u), ("ddt", dt), ("da", a), ("db", b), ("dc", c), ("dz", u))}
    out["dd"] = torch.zeros(ch, dtype=F64)
    out["ddt_bias"] = torch.zeros(ch, dtype=F64)
    out["dh_in"] = torch.zeros(n, ch, s, dtype=F64)
    for i, ln in enumerate(lens(lengths, n, t)):
        gh = torch.zeros(ch, s, dtype=F64) if dh_out is None else ab(dh_out[i])
        for q in range(ln - 1, -1, -1):
            raw = dt[i, q] if bias is None else dt[i, q] + bias
            delta = softplus(raw) if use_softplus else raw
            decay = torch.exp(delta[:, None] * a)
            uu, dd = ab(u[i, q]), ab(delta)
            bb, cc = ab(b[i, q])[grp], ab(c[i, q])[grp]
            h1, h0 = kept[i][q + 1], kept[i][q]
            gy = ab(dy[i, q])
            if z is not None:
                y0 = (h1 * cc).sum(-1) + (0 if d is None else ab(d) * uu)
                out["dz"][i, q] = gy * y0 * (SLOPE_MAX if mag else silu_slope(z[i, q]))
                gy = gy * ab(silu(z[i, q]))
            gh = gh + gy[:, None] * cc
            gb = (gh * bb).sum(-1)
            through = gh * decay * h0
            out["du"][i, q] = dd * gb + (0 if d is None else ab(d) * gy)
            r = (through * ab(a)).sum(-1) + uu * gb
            r = r * (torch.sigmoid(raw) if use_softplus else 1.0)
            out["ddt"][i, q] = r
            out["ddt_bias"] += r
            out["dd"] += gy * uu
            out["da"] += through * dd[:, None]
            out["db"][i, q] = (gh * (dd * uu)[:, None]).reshape(g, ch // g, s).sum(1)
            out["dc"][i, q] = (h1 * gy[:, None]).reshape(g, ch // g, s).sum(1)
            gh = gh * decay
        out["dh_in"][i] = gh
    return out


# ------------------------------------------------------------------ join

def _norm(v, kind, eps, w, b, mag_v=None):
    """(normalised, reciprocal root, output); mag_v: the magnitude form of v, whose row maximum over the root is the
    condition number of the row's norm."""
    xc = v - v.mean(-1, keepdim=True) if kind == "layer" else v
    rs = 1 / torch.sqrt((xc ** 2).mean(-1, keepdim=True) + eps)
    xn = xc * rs
    o = xn if w is None else xn * w
    if b is not None:
        o = o + b
    return xn, rs, o


def join(y, res, *, post, pre, act, eps, gate=None, gate_act=False, gate_rows=1, scale=None, post_w=None, post_b=None,
         pre_w=None, pre_b=None):
    """(x, h, bounds): bounds are the magnitudes of x and h."""
    rows = (y if y is not None else res).shape[0]
    x = torch.zeros_like(y) if res is None else res
    xm = x.abs()
    if y is not None:
        n1, n1m = y, y.abs()
        if post:
            xn, rs, n1 = _norm(y, post, eps, post_w, post_b)
            cond = (y.abs().amax(-1, keepdim=True) * rs).clamp(min=1)
            n1m = cond * (xn.abs() + 1) * (1 if post_w is None else post_w.abs()) + (0 if post_b is None else post_b.abs())
        f = torch.ones_like(y)
        if gate is not None:
            gt = gate[torch.arange(rows) // gate_rows]
            f = f * (silu(gt) if gate_act else gt)
        if scale is not None:
            f = f * scale
        x, xm = x + f * n1, xm + f.abs() * n1m
    if not pre:
        return x, None, (xm, None)
    xn, rs, h = _norm(x, pre, eps, pre_w, pre_b)
    cond = (xm.amax(-1, keepdim=True) * rs).clamp(min=1)
    hm = cond * (xn.abs() + 1) * (1 if pre_w is None else pre_w.abs()) + (0 if pre_b is None else pre_b.abs())
    return x, (silu(h) if act else h), (xm, hm)


def join_grad(y, res, dx_out, dh, *, post, pre, act, eps, gate=None, gate_act=False, gate_rows=1, scale=None,
              post_w=None, post_b=None, pre_w=None, pre_b=None):
    """(gradients, bounds) as dicts, by the formulas; the bounds carry the norms' condition numbers along."""
    rows, c = (y if y is not None else res).shape
    one = torch.ones(rows, c, dtype=F64)
    at = torch.arange(rows) // gate_rows
    x = torch.zeros(rows, c, dtype=F64) if res is None else res
    xm = x.abs()
    if y is not None:
        xn1, rs1, n1 = (y, None, y) if not post else _norm(y, post, eps, post_w, post_b)
        cond1 = 1.0 if not post else (y.abs().amax(-1, keepdim=True) * rs1).clamp(min=1)
        xn1m = y.abs() if not post else cond1 * (xn1.abs() + 1)
        n1m = xn1m if post_w is None else xn1m * post_w.abs()
        n1m = n1m if post_b is None else n1m + post_b.abs()
        ga, slope = one, one
        if gate is not None:
            gt = gate[at]
            ga, slope = (silu(gt), silu_slope(gt)) if gate_act else (gt, one)
        sc = one if scale is None else one * scale
        x, xm = x + sc * ga * n1, xm + (sc * ga).abs() * n1m
    o, m = {}, {}
    dx = torch.zeros(rows, c, dtype=F64) if dx_out is None else dx_out
    dxm = dx.abs()
    if dh is not None:
        xn2, rs2, hp = _norm(x, pre, eps, pre_w, pre_b)
        cond2 = (xm.amax(-1, keepdim=True) * rs2).clamp(min=1)
        xn2m = cond2 * (xn2.abs() + 1)
        g, gm = dh, dh.abs()
        if act:
            hm = xn2m * (1 if pre_w is None else pre_w.abs()) + (0 if pre_b is None else pre_b.abs())
            g, gm = dh * silu_slope(hp), dh.abs() * (SLOPE_MAX + hm)
        o["dpre_w"], m["dpre_w"] = (g * xn2).sum(0), (gm * xn2m).sum(0)
        o["dpre_b"], m["dpre_b"] = g.sum(0), gm.sum(0)
        w = one if pre_w is None else one * pre_w
        d, dm = g * w, gm * w.abs()
        e = d - xn2 * (d * xn2).mean(-1, keepdim=True)
        em = cond2 * (dm + xn2m * (dm * xn2m).mean(-1, keepdim=True))
        if pre == "layer":
            e, em = e - d.mean(-1, keepdim=True), em + cond2 * dm.mean(-1, keepdim=True)
        dx, dxm = dx + rs2 * e, dxm + rs2 * em
    if res is not None:
        o["dresidual"], m["dresidual"] = dx, dxm
    if y is not None:
        o["dscale"], m["dscale"] = (dx * n1 * ga).sum(0), (dxm * n1m * ga.abs()).sum(0)
        if gate is not None:
            each, eachm = dx * n1 * sc * slope, dxm * n1m * sc.abs() * SLOPE_MAX
            o["dgate"] = torch.zeros_like(gate).index_add_(0, at, each)
            m["dgate"] = torch.zeros_like(gate).index_add_(0, at, eachm)
        dn, dnm = dx * sc * ga, dxm * (sc * ga).abs()
        o["dpost_w"], m["dpost_w"] = (dn * xn1).sum(0), (dnm * xn1m).sum(0)
        o["dpost_b"], m["dpost_b"] = dn.sum(0), dnm.sum(0)
        if post:
            w = one if post_w is None else one * post_w
            d, dm = dn * w, dnm * w.abs()
            e = d - xn1 * (d * xn1).mean(-1, keepdim=True)
            em = cond1 * (dm + xn1m * (dm * xn1m).mean(-1, keepdim=True))
            if post == "layer":
                e, em = e - d.mean(-1, keepdim=True), em + cond1 * dm.mean(-1, keepdim=True)
            dn, dnm = rs1 * e, rs1 * em
        o["dy"], m["dy"] = dn, dnm
    return o, m


# ------------------------------------------------------------- comparison

def assert_close(got, ref, mag, depth, what):
    """Every element within depth * 2**-24 of its magnitude, plus, for a
    bf16 result, the one rounding to 8 significant bits: half a step, at most
    2**-8 of the value."""
    assert tuple(got.shape) == tuple(ref.shape), (what, tuple(got.shape), tuple(ref.shape))
    g = got.detach().cpu().to(F64)
    assert bool(torch.isfinite(g).all()), (what, "values that are not finite", int((~torch.isfinite(g)).sum()))
    bound = depth * EPS32 * mag + 1e-35
    if got.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (ref.abs() + bound) + 2.0 ** -133
    over = (g - ref).abs() - bound
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 0, (what, "over the bound by", worst, "of", float(bound.flatten()[over.flatten().argmax()]),
                        "elements", int((over > 0).sum()), "of", over.numel())
