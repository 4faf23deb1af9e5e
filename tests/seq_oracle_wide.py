"""Plain 64-bit forms of causal_conv1d and selective_scan with their
gradients, whole tensors at a time on any device, for sizes that
seq_oracle's token-by-token loops are too slow for.  test_seq_oracle_wide
compares the two.  ``mag`` as in seq_oracle: the same formula on absolute
values."""
import torch

import seq_oracle as so

F64 = torch.float64


def valid(lengths, n, t, device):
    """[n][t][1]: 1 for a sequence's tokens, 0 after them."""
    ln = torch.tensor(so.lens(lengths, n, t), device=device)
    return (torch.arange(t, device=device)[None, :] < ln[:, None]).to(F64)[..., None], ln


def conv1d(x, w, b, act, cache=None, lengths=None, dy=None, dtail=None, mag=False):
    """y, cache_out; with dy also dx, dw, db, dcache (a dict)."""
    n, t, c = x.shape
    k = w.shape[0]
    on, ln = valid(lengths, n, t, x.device)

    def windows(x, cache):
        head = torch.zeros(n, k - 1, c, dtype=F64, device=x.device) if cache is None else cache
        return torch.cat([head, torch.where(on > 0, x, 0.0)], 1)

    def argument(z, w, b):
        p = sum(w[j] * z[:, j:j + t] for j in range(k))
        return p if b is None else p + b

    z = windows(x, cache)
    p = argument(z, w, b)
    slope = so.silu_slope(p) if act else torch.ones_like(p)
    out = {}
    if mag:
        z, w, b = z.abs(), w.abs(), None if b is None else b.abs()
        out["y"] = argument(z, w, b) * on
        slope = torch.full_like(p, so.SLOPE_MAX if act else 1.0)
    else:
        out["y"] = (so.silu(p) if act else p) * on
    tail_at = ln[:, None] + torch.arange(k - 1, device=x.device)[None, :]
    out["cache_out"] = torch.gather(z, 1, tail_at[..., None].expand(-1, -1, c))
    if dy is None:
        return out
    g = torch.where(on > 0, dy.abs() if mag else dy, 0.0) * slope
    dz = torch.zeros_like(z)
    for j in range(k):
        dz[:, j:j + t] += w[j] * g
    if dtail is not None:
        dz.scatter_add_(1, tail_at[..., None].expand(-1, -1, c), dtail.abs() if mag else dtail)
    out["db"] = g.sum((0, 1))
    out["dw"] = torch.stack([(g * z[:, j:j + t]).sum((0, 1)) for j in range(k)])
    out["dcache_in"], out["dx"] = dz[:, :k - 1], dz[:, k - 1:]
    return out


def scan(u, dt, a, b, c, d=None, z=None, bias=None, h_in=None, lengths=None, dy=None, dh_out=None, mag=False):
    """y, h_out; with dy also the gradients (a dict); b and c [n][t][G][S]; with softplus."""
    n, t, ch = u.shape
    s, groups = a.shape[1], b.shape[2]
    grp = torch.arange(ch, device=u.device) // (ch // groups)
    on, _ = valid(lengths, n, t, u.device)
    ab = (lambda v: v.abs()) if mag else (lambda v: v)
    raw = torch.where(on > 0, dt if bias is None else dt + bias, 0.0)
    delta = so.softplus(raw) * on
    clean = lambda v: torch.where(on > 0, v, 0.0)  # noqa: E731
    u, bb = ab(clean(u)), ab(torch.where(on[..., None] > 0, b, 0.0))
    cc = ab(torch.where(on[..., None] > 0, c, 0.0))
    sz = torch.ones_like(u) if z is None else ab(so.silu(clean(z)))
    h = torch.zeros(n, ch, s, dtype=F64, device=u.device) if h_in is None else ab(h_in)
    kept, y0 = [h], torch.zeros_like(u)
    for q in range(t):
        h = torch.exp(delta[:, q, :, None] * a) * h + (delta[:, q] * u[:, q])[..., None] * bb[:, q][:, grp]
        kept.append(h)
        y0[:, q] = (h * cc[:, q][:, grp]).sum(-1)
    if d is not None:
        y0 = y0 + ab(d) * u
    out = {"y": y0 * sz * on, "h_out": h}
    if dy is None:
        return out
    dy = ab(clean(dy))
    gy = dy * sz
    if z is not None:
        out["dz"] = dy * y0 * (so.SLOPE_MAX if mag else so.silu_slope(clean(z))) * on
    slope = torch.sigmoid(raw)
    g = torch.zeros(n, ch, s, dtype=F64, device=u.device) if dh_out is None else ab(dh_out)
    for name, like in (("du", u), ("ddt", u), ("db", bb), ("dc", bb), ("da", a)):
        out[name] = torch.zeros_like(like)
    for q in range(t - 1, -1, -1):
        decay = torch.exp(delta[:, q, :, None] * a)
        g = g + gy[:, q, :, None] * cc[:, q][:, grp]
        gb = (g * bb[:, q][:, grp]).sum(-1)
        through = g * decay * kept[q] * on[:, q, :, None]
        out["du"][:, q] = delta[:, q] * gb + (0 if d is None else ab(d) * gy[:, q])
        out["ddt"][:, q] = ((through * ab(a)).sum(-1) + u[:, q] * gb) * slope[:, q] * on[:, q]
        out["da"] += (through * delta[:, q, :, None]).sum(0)
        out["db"][:, q] = (g * (delta[:, q] * u[:, q])[..., None]).reshape(n, groups, ch // groups, s).sum(2)
        out["dc"][:, q] = (kept[q + 1] * gy[:, q, :, None]).reshape(n, groups, ch // groups, s).sum(2)
        g = g * decay
    out["ddt_bias"], out["dd"], out["dh_in"] = out["ddt"].sum((0, 1)), (gy * u).sum((0, 1)), g
    return out
