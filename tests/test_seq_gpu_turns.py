"""Sequence operators on the GPU at sizes where a workgroup, a wave or a thread
takes more than one piece of the work: further rows of the join, further
chunks of the backward scan, further runs of the backward convolution, and long
runs.  Each test first works out from the plan that it does.  Bounds as in
test_seq_gpu; a sum over rows or tokens is as deep as the chain that adds it
(one worker's terms, its workgroup's lines, and every 16th worker's row)."""
import pytest
import torch

import causal_conv3d_video_amd as cc3d
import seq_oracle as so
import seq_oracle_wide as wide
import test_seq_gpu as base

pytestmark = pytest.mark.gpu
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
DEV = base.DEV


def close(got, ref, mag, depth, what):
    """seq_oracle.assert_close where the tensors are."""
    assert tuple(got.shape) == tuple(ref.shape), (what, tuple(got.shape), tuple(ref.shape))
    g = got.to(F64)
    assert bool(torch.isfinite(g).all()), what
    bound = depth * so.EPS32 * mag + 1e-35
    if got.dtype == BF:
        bound = bound + 2.0 ** -8 * (ref.abs() + bound) + 2.0 ** -133
    over = (g - ref).abs() - bound
    assert float(over.max()) <= 0, (what, float(over.max()), int((over > 0).sum()), over.numel())


# ----------------------------------------------------------------- conv1d

@pytest.mark.parametrize("n,t,c,k,dtype,ragged", [
    (7000, 5, 512, 4, BF, True),     # 3.4 runs a thread, each a whole sequence
    (20001, 9, 96, 3, F32, True),    # rows of twelve lanes' channels, 2.1 runs
    (200000, 3, 12, 5, BF, False),   # two lanes a row, one of them by halves
    (300000, 2, 5, 2, F32, True),    # fewer than eight channels
    (2, 17000, 2048, 4, BF, True),   # runs of 34 tokens each way, two a thread
    (1, 70000, 600, 8, F32, False),  # runs of 64, one wave a SIMD
])
def test_conv1d_takes_further_runs(cuda_device, n, t, c, k, dtype, ragged):
    plan = cc3d.causal_conv1d_plan(cc3d.make_conv1d_desc(n, t, c, k, act="silu", dtype=dtype))
    lanes = 1
    while lanes < 64 and lanes * 8 < c:
        lanes *= 2
    lines, rows = 256 // lanes, plan.info["backward_workspace_bytes"] // (4 * (k + 1) * c)
    seg = -(-t // plan.info["backward_chunks"])
    turns = n * plan.info["backward_chunks"] / (rows * lines)
    assert turns > 1.5 and (turns > 2 or seg > 32)

    g = torch.Generator(device=DEV).manual_seed(700 + c)

    def rn(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device=DEV, dtype=F32).mul_(scale).to(dtype)

    x, w, b, dy = rn(n, t, c), rn(k, c, scale=k ** -0.5), rn(c), rn(n, t, c)
    cache, dtail = rn(n, k - 1, c), rn(n, k - 1, c)
    ln = base.lengths_of(ragged, n, t)
    lt = None if ln is None else torch.tensor(ln, dtype=torch.int32, device=DEV)
    got = dict(y=torch.full_like(x, base.NAN), cache_out=torch.full_like(cache, base.NAN))
    cc3d.causal_conv1d_forward(plan, x, w, b, got["y"], cache_in=cache, cache_out=got["cache_out"], lengths=lt)
    got.update(dx=torch.full_like(x, base.NAN), dw=base.nan(k, c), db=base.nan(c), dcache_in=torch.full_like(cache, base.NAN))
    cc3d.causal_conv1d_backward(plan, x, w, b, dy, dx=got["dx"], dw=got["dw"], db=got["db"], cache_in=cache,
                                dcache_out=dtail, dcache_in=got["dcache_in"], lengths=lt, workspace=base.space(plan, True))
    a = [v.to(F64) for v in (x, w, b)] + [True, cache.to(F64), ln, dy.to(F64), dtail.to(F64)]
    ref, mag = wide.conv1d(*a), wide.conv1d(*a, mag=True)
    depth = 8 * (k + 2) + 64
    chain = (int(turns) + 1) * seg + lines + rows // 16 + 32
    for name, v in got.items():
        close(v, ref[name], mag[name], depth + (chain if name in ("dw", "db") else 0), name)


# ------------------------------------------------------------------- scan

@pytest.mark.parametrize("n,t,c,s,g,dtype,ragged", [
    (2, 600, 16384, 16, 2, BF, True),   # 20 chunks over 4 workers
    (3, 600, 8200, 12, 1, F32, True),   # a last tile of 8 channels
    (2, 900, 16384, 4, 1, BF, False),   # walks of four tokens
    (2, 900, 16384, 8, 4, F32, True),
    (2, 250, 16384, 64, 1, BF, True),   # four waves of states, one worker
    (3, 200, 8192, 24, 2, F32, False),  # two waves of states by two of channels
])
def test_scan_backward_takes_further_chunks(cuda_device, n, t, c, s, g, dtype, ragged):
    plan = cc3d.selective_scan_plan(cc3d.make_scan_desc(n, t, c, s, groups=g, dtype=dtype))
    sg = 1 if s <= 4 else 2 if s <= 8 else 4
    waves, each, wc = -(-s // (4 * sg)), 128 // sg, 1
    while wc * 2 * waves <= 4 and wc * each < c // g:
        wc *= 2
    tiles, items = g * -(-(c // g) // (each * wc)), n * plan.info["backward_chunks"]
    workers = min(items, -(-2048 // (tiles * waves * wc)))
    state = s * c
    assert plan.info["backward_workspace_bytes"] == 4 * (items * (2 * state + c) + workers * (state + 2 * waves * c)
                                                         + tiles * n * t * waves * 8 * sg)
    assert items >= 3 * workers

    i = {k: base.dev(v) for k, v in base.scan_inputs(n, t, c, s, g, dtype, True, "dzbh", 710 + c + s).items()}
    ln = base.lengths_of(ragged, n, t)
    lt = None if ln is None else torch.tensor(ln, dtype=torch.int32, device=DEV)
    opt = dict(d=i["d"], z=i["z"], dt_bias=i["dt_bias"], h_in=i["h_in"], lengths=lt)
    ins = [i[k] for k in ("u", "dt", "a", "b", "c")]
    got = dict(y=torch.full_like(i["u"], base.NAN), h_out=base.nan(n, c, s))
    cc3d.selective_scan_forward(plan, *ins, got["y"], h_out=got["h_out"], workspace=base.space(plan), **opt)
    like = dict(du="u", ddt="dt", da="a", db="b", dc="c", dd="d", dz="z", ddt_bias="dt_bias", dh_in="h_in")
    grads = {k: torch.full_like(i[v], base.NAN) for k, v in like.items()}
    cc3d.selective_scan_backward(plan, *ins, i["dy"], dh_out=i["dh_out"], workspace=base.space(plan, True), **opt, **grads)
    a = [i[k].to(F64) for k in ("u", "dt", "a", "b", "c", "d", "z", "dt_bias", "h_in")] + [ln, i["dy"].to(F64),
                                                                                          i["dh_out"].to(F64)]
    ref, mag = wide.scan(*a), wide.scan(*a, mag=True)
    depth = 4 * t + 2 * s + 640
    for name, v in dict(got, **grads).items():
        more = depth + n * t if name not in got else 0
        if name in ("db", "dc"):
            more += c // g
        close(v, ref[name], mag[name], depth + more, name)


# ------------------------------------------------------------------- join

@pytest.mark.parametrize("r,c,post,pre,act,gate_rows,gate_act,dtype", [
    (200003, 24, "rms", "rms", "silu", 1, "silu", F32),      # 3.1 steps forward, 12.2 backward, a gate row each
    (200003, 20, "layer", "rms", None, 7, "silu", BF),       # a gate row's place moves by no whole step
    (140001, 40, "rms", "layer", None, 0, None, BF),
    (40000, 24, "rms", "rms", "silu", 5000, "silu", F32),    # parts of gate rows, three steps each
    (40000, 48, "layer", "rms", None, 100, None, BF),        # whole gate rows, four steps each
    (51000, 24, "rms", None, None, 40, "silu", F32),         # three whole gate rows a workgroup
    (6403, 2048, "rms", "rms", None, 1, "silu", BF),         # rows of four waves, 3.1 steps forward
    (6403, 1100, "layer", "layer", "silu", 7, None, F32),
    (1700, 8192, "layer", "rms", "silu", 1, "silu", BF),     # rows of sixteen waves: none loaded ahead, 13 steps backward
    (1700, 4100, "rms", "layer", None, 0, None, F32),
])
def test_join_takes_further_rows(cuda_device, r, c, post, pre, act, gate_rows, gate_act, dtype):
    plan = cc3d.norm_join_plan(cc3d.make_join_desc(r, c, post=post, pre=pre, act=act, gate_act=gate_act,
                                                   gate_rows=max(1, gate_rows), eps=1e-5, dtype=dtype))
    lanes = 8
    while lanes * 8 < c:
        lanes *= 2
    threads = 256 if lanes <= 64 else lanes
    at_once = threads // lanes
    parted = plan.info["backward_workspace_bytes"] // (4 * c)
    gates = -(-r // gate_rows) if gate_rows else r
    kinds = 6 if gate_rows > 1 and gates < 1024 * 64 // threads else 5
    parts = parted // kinds
    assert parted == parts * kinds and r > 2 * parts * at_once
    if not gate_rows or c < 40 and gate_rows < 10 or c > 1000:
        assert r > 2 * at_once * (8192 * 64 // threads)  # forward

    i = base.join_case(r, c, post, pre, gate_rows, True, True, True, dtype, 720 + r + c)
    par = {k: base.dev(i[k]) for k in ("scale", "post_w", "post_b", "pre_w", "pre_b")}
    y, res, gate = base.dev(i["y"]), base.dev(i["res"]), base.dev(i["gate"])
    got = dict(x_out=torch.full_like(y, base.NAN))
    if pre:
        got["h_out"] = torch.full_like(y, base.NAN)
    cc3d.norm_join_forward(plan, y, res, gate=gate, **par, **got)
    opts = dict(post=post, pre=pre, act=act == "silu", eps=1e-5, gate_act=gate_act == "silu", gate_rows=max(1, gate_rows),
                **{k: base.d64(i[k]) for k in ("gate",) + tuple(par)})
    x, h, (xm, hm) = so.join(base.d64(i["y"]), base.d64(i["res"]), **opts)
    for name, want, m in (("x_out", x, xm), ("h_out", h, hm)):
        if name in got:
            close(got[name], base.dev(want), base.dev(m), 256, name)

    grads = {k: torch.full_like(v, base.NAN) for k, v in (("dy", y), ("dresidual", res), ("dgate", gate)) if v is not None}
    grads.update({"d" + k: base.nan(c) for k, v in par.items() if v is not None})
    cc3d.norm_join_backward(plan, y, res, dx_out=base.dev(i["dx_out"]), dh=base.dev(i["dh"]), gate=gate,
                            workspace=base.space(plan, True), **par, **grads)
    ref, mag = so.join_grad(base.d64(i["y"]), base.d64(i["res"]), base.d64(i["dx_out"]), base.d64(i["dh"]), **opts)
    # a worker's terms one after another, the workgroup's lines, every 16th (or 4th) row of partial sums
    chain = -(-r // (parts * at_once)) + 1 + at_once + parts // 16 + 16
    gate_chain = -(-max(1, gate_rows) // at_once) + at_once + parts // 4
    for k, v in grads.items():
        close(v, base.dev(ref[k]), base.dev(mag[k]), 1024 + (chain if v.dim() == 1 else gate_chain if k == "dgate" else 0), k)


# ------------------------------------------------------------------ graphs

def test_a_replayed_graph_of_the_backward_scan_with_much_lds(cuda_device):
    """64 states of 128 and more channels take 104 KiB a workgroup, more than a launch has unasked."""
    n, t, c, s = 2, 150, 160, 64
    i = {k: base.dev(v) for k, v in base.scan_inputs(n, t, c, s, 1, BF, True, "dzbh", 730).items()}
    plan = cc3d.selective_scan_plan(cc3d.make_scan_desc(n, t, c, s))
    got = {k: torch.full_like(i[v], base.NAN) for k, v in dict(du="u", da="a", db="b", dc="c", dh_in="h_in").items()}
    space = base.space(plan, True)

    def launch():
        cc3d.selective_scan_backward(plan, *[i[k] for k in ("u", "dt", "a", "b", "c")], i["dy"], d=i["d"], z=i["z"],
                                     dt_bias=i["dt_bias"], h_in=i["h_in"], dh_out=i["dh_out"], workspace=space, **got)

    launch()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        launch()
    for step in range(3):
        i["u"].mul_(0.9)
        for v in got.values():
            v.fill_(base.NAN)
        graph.replay()
        torch.cuda.synchronize()
        replayed = {k: v.clone() for k, v in got.items()}
        for v in got.values():
            v.fill_(base.NAN)
        launch()
        torch.cuda.synchronize()
        for k, v in got.items():
            assert bool(torch.isfinite(v.float()).all()) and torch.equal(v, replayed[k]), (step, k)
