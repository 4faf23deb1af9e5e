"""The whole-tensor 64-bit forms against the token-by-token ones."""
import pytest
import torch

import seq_oracle as so
import seq_oracle_wide as wide

F64 = torch.float64


def _same(a, b, what):
    # two orders of the same sums of at most some hundred terms in 64 bits
    assert float((a - b).abs().max()) <= 1e-12 * max(1.0, float(b.abs().max())), what


@pytest.mark.parametrize("mag", [False, True])
@pytest.mark.parametrize("ln", [None, [7, 0, 1, 9]])
def test_conv1d(ln, mag):
    g = torch.Generator().manual_seed(1)
    n, t, c, k = 4, 7, 5, 4

    def rn(*shape):
        return torch.randn(*shape, generator=g, dtype=F64)

    x, w, b, cache, dy, dtail = rn(n, t, c), rn(k, c), rn(c), rn(n, k - 1, c), rn(n, t, c), rn(n, k - 1, c)
    got = wide.conv1d(x, w, b, True, cache, ln, dy, dtail, mag)
    y, tail, _ = so.conv1d(x, w, b, True, cache, ln, mag)
    want = dict(zip(("dx", "dw", "db", "dcache_in"), so.conv1d_grad(x, w, b, True, dy, cache, dtail, ln, mag)), y=y,
                cache_out=tail)
    assert set(got) == set(want)
    for name in want:
        _same(got[name], want[name], name)


@pytest.mark.parametrize("mag", [False, True])
@pytest.mark.parametrize("ln", [None, [6, 0, 1, 9]])
def test_scan(ln, mag):
    g = torch.Generator().manual_seed(2)
    n, t, c, s, groups = 4, 6, 6, 3, 2

    def rn(*shape):
        return torch.randn(*shape, generator=g, dtype=F64)

    u, dt, b, cc, d, z, bias = rn(n, t, c), rn(n, t, c), rn(n, t, groups, s), rn(n, t, groups, s), rn(c), rn(n, t, c), rn(c)
    a, h_in, dy, dh = -rn(c, s).abs(), rn(n, c, s), rn(n, t, c), rn(n, c, s)
    got = wide.scan(u, dt, a, b, cc, d, z, bias, h_in, ln, dy, dh, mag)
    y, h, _ = so.scan(u, dt, a, b, cc, d, z, bias, h_in, ln, True, mag)
    want = dict(so.scan_grad(u, dt, a, b, cc, dy, d, z, bias, h_in, dh, ln, True, mag), y=y, h_out=h)
    assert set(got) == set(want)
    for name in want:
        _same(got[name], want[name], name)
