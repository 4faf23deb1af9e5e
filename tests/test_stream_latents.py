"""The streaming example: its block against a plain torch form of the same
block (outputs, carried states and every gradient), and streamed chunks against
one call."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _plain(block, w, frames, taps, h):
    """The block in plain torch, [T, P, C] frames; returns (x_out, h_out, taps, states)."""
    t, p, _ = frames.shape
    i, r, s, k = block.inner, block.rank, block.states, block.k

    def rms(v, weight):
        return v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6) * weight

    xz = rms(frames, w["first_w"]) @ w["in_w"].T
    x, z = xz[..., :i], xz[..., i:]
    seq = torch.cat([taps.transpose(0, 1), x])
    u = torch.nn.functional.silu(w["conv_b"] + sum(w["conv_w"][j] * seq[j:j + t] for j in range(k)))
    low = u @ w["bc_w"].T
    delta = torch.nn.functional.softplus(low[..., :r] @ w["dt_w"].T + w["dt_bias"])
    ys = []
    for q in range(t):
        b, c = low[q, :, None, r:r + s], low[q, :, None, r + s:]
        h = torch.exp(delta[q][..., None] * w["a"]) * h + (delta[q] * u[q])[..., None] * b
        ys.append(((h * c).sum(-1) + w["d"] * u[q]) * torch.nn.functional.silu(z[q]))
    out = torch.stack(ys) @ w["out_w"].T
    x_out = frames + w["scale"] * rms(out, w["post_w"])
    return x_out, torch.nn.functional.silu(rms(x_out, w["next_w"])), seq[t:].transpose(0, 1), h


def test_block_outputs_states_and_gradients(cuda_device):
    """fp32 block against the plain form in fp64 on the CPU.  Between the two lie
    some 200 roundings of 2**-24 in chains of five products: 1e-4 of each
    tensor's largest value."""
    from causal_conv3d_video_amd.examples.stream_latents import MixerBlock, MixerState

    block = MixerBlock(14, 24, 40, states=16, rank=4, dtype=torch.float32, device=DEV, seed=3)
    g = torch.Generator().manual_seed(4)
    frames = torch.randn(7, 14, 24, generator=g)
    dx, dh = torch.randn(7, 14, 24, generator=g), torch.randn(7, 14, 24, generator=g)
    state = MixerState(block)
    state.taps.copy_(torch.randn(state.taps.shape, generator=g))
    state.h.copy_(torch.randn(state.h.shape, generator=g))
    w = {k: v.double().cpu().requires_grad_() for k, v in block.w.items()}
    f = frames.double().requires_grad_()
    want = _plain(block, w, f, state.taps.double().cpu(), state.h.double().cpu())
    (want[0] * dx.double()).sum().add((want[1] * dh.double()).sum()).backward()
    kept = {}
    x_out, h_out = block.forward(frames.to(DEV), state, keep=kept)
    df, grads = block.backward(kept, dx.to(DEV), dh.to(DEV))

    def near(got, ref, what):
        ref = ref.detach()
        assert float((got.double().cpu() - ref).abs().max()) <= 1e-4 * float(ref.abs().max()), what

    for got, ref, what in zip((x_out, h_out, state.taps, state.h), want, ("x_out", "h_out", "taps", "states")):
        near(got, ref, what)
    near(df, f.grad, "frames")
    assert set(grads) == set(w)
    for k, v in grads.items():
        near(v, w[k].grad, k)


def test_streamed_chunks_follow_one_call(cuda_device):
    """bf16 chunks of 1, 2 and 4 frames against one call over 7.  The block's
    kernels give a frame the same bits either way but for the scan's sums (fp32)
    and the products' (bf16 steps of 2**-8, through four products and two norms):
    4 * 2**-8 of the largest value."""
    from causal_conv3d_video_amd.examples.stream_latents import LatentDecoder

    model = LatentDecoder(6, 10, 32, 64, 48, device=DEV, seed=5)
    g = torch.Generator().manual_seed(6)
    latents = torch.randn(7, 6, 10, 32, generator=g).to(torch.bfloat16).to(DEV)
    whole = model(latents).float()
    states = model.state.h.clone()
    model.reset()
    parts = torch.cat([model(x) for x in latents.split([1, 2, 4])]).float()
    assert bool(torch.isfinite(whole).all())
    assert float((parts - whole).abs().max()) <= 4 * 2.0 ** -8 * float(whole.abs().max())
    assert float((model.state.h - states).abs().max()) <= 4 * 2.0 ** -8 * float(states.abs().max())
