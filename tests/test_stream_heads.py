"""The streaming example's mixer in heads: its block against a plain torch form
of the same block (outputs, carried state and every gradient), streamed chunks
against one call, and both mixers in front of the same decoder."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _turn(x, at):
    """Rotary positions, half layout: x [T, P, H, D], at: the frames' numbers."""
    d = x.shape[-1]
    half = d // 2
    f = 10000.0 ** (-2.0 * torch.arange(half, dtype=x.dtype) / (2 * half))
    ang = at.to(x.dtype)[:, None] * f
    c, s = torch.cos(ang)[:, None, None], torch.sin(ang)[:, None, None]
    a, b = x[..., :half], x[..., half:2 * half]
    return torch.cat([a * c - b * s, a * s + b * c, x[..., 2 * half:]], -1)


def _plain(block, w, frames, h, at):
    """The block in plain torch, [T, P, C] frames; returns (x_out, h_out, states)."""
    t, p, _ = frames.shape
    i, n, d = block.inner, block.heads, block.width

    def rms(v, weight):
        return v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6) * weight

    q, k, v, gate = (rms(frames, w["first_w"]) @ w["in_w"].T).split(i, -1)
    pos = at + torch.arange(t)
    q, k, v = _turn(q.reshape(t, p, n, d), pos), _turn(k.reshape(t, p, n, d), pos), v.reshape(t, p, n, d)
    os = []
    for x in range(t):
        h = torch.exp(w["log_decay"])[:, None, None] * h + k[x][..., None] * v[x][..., None, :]
        os.append(d ** -0.5 * (q[x][..., None] * h).sum(-2))
    o = torch.stack(os)
    o = (o - o.mean(-1, keepdim=True)) / torch.sqrt(o.var(-1, unbiased=False, keepdim=True) + 1e-6)
    y = o.reshape(t, p, i) * w["head_w"] + w["head_b"]
    out = (y * torch.nn.functional.silu(gate)) @ w["out_w"].T
    x_out = frames + w["scale"] * rms(out, w["post_w"])
    return x_out, torch.nn.functional.silu(rms(x_out, w["next_w"])), h


def test_block_outputs_states_and_gradients(cuda_device):
    """fp32 block against the plain form in fp64 on the CPU.  Between the two lie
    some 200 roundings of 2**-24 in chains of five products, and a norm of each
    head whose condition is that of a norm of a few values: 1e-4 of each tensor's
    largest value."""
    from causal_conv3d_video_amd.examples.stream_latents import HeadsBlock, HeadsState

    block = HeadsBlock(14, 24, 40, heads=4, dtype=torch.float32, device=DEV, seed=3)
    g = torch.Generator().manual_seed(4)
    frames = torch.randn(7, 14, 24, generator=g)
    dx, dh = torch.randn(7, 14, 24, generator=g), torch.randn(7, 14, 24, generator=g)
    state = HeadsState(block)
    state.h.copy_(torch.randn(state.h.shape, generator=g))
    state.frames += 5
    w = {k: v.double().cpu().requires_grad_() for k, v in block.w.items()}
    f = frames.double().requires_grad_()
    want = _plain(block, w, f, state.h.double().cpu(), 5)
    (want[0] * dx.double()).sum().add((want[1] * dh.double()).sum()).backward()
    kept = {}
    x_out, h_out = block.forward(frames.to(DEV), state, keep=kept)
    df, grads = block.backward(kept, dx.to(DEV), dh.to(DEV))
    assert int(state.frames[0]) == 12

    def near(got, ref, what):
        ref = ref.detach()
        assert float((got.double().cpu() - ref).abs().max()) <= 1e-4 * float(ref.abs().max()), what

    for got, ref, what in zip((x_out, h_out, state.h), want, ("x_out", "h_out", "states")):
        near(got, ref, what)
    near(df, f.grad, "frames")
    assert set(grads) == set(w)
    for k, v in grads.items():
        near(v, w[k].grad, k)


@pytest.mark.parametrize("frames", [[1, 2, 4], [40, 33]])
def test_streamed_chunks_follow_one_call(cuda_device, frames):
    """fp32 chunks against one call, through the decoder's convolution too: the
    block's sums in another order, 2**-24 each, through five products and three
    norms: 1e-4 of the largest value."""
    from causal_conv3d_video_amd.examples.stream_latents import LatentDecoder

    model = LatentDecoder(3, 5, 32, 8, 48, dtype=torch.float32, device=DEV, seed=5, mixer="heads")
    g = torch.Generator().manual_seed(6)
    latents = torch.randn(sum(frames), 3, 5, 32, generator=g).to(DEV)
    whole = model(latents)
    states = model.state.h.clone()
    model.reset()
    parts = torch.cat([model(x) for x in latents.split(frames)])
    assert bool(torch.isfinite(whole).all())
    assert float((parts - whole).abs().max()) <= 1e-4 * float(whole.abs().max())
    assert float((model.state.h - states).abs().max()) <= 1e-4 * float(states.abs().max())


def test_mixers_run_in_bf16(cuda_device):
    from causal_conv3d_video_amd.examples.stream_latents import LatentDecoder, MIXERS

    g = torch.Generator().manual_seed(6)
    latents = torch.randn(7, 6, 10, 32, generator=g).to(torch.bfloat16).to(DEV)
    for mixer in MIXERS:
        model = LatentDecoder(6, 10, 32, 64, 128, device=DEV, seed=5, mixer=mixer)
        out = torch.cat([model(x) for x in latents.split([1, 2, 4])])
        assert out.shape == (7, 6, 10, 64) and bool(torch.isfinite(out).all())
