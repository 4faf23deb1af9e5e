"""A temporal mixer over streamed latent frames, ahead of the decoder's cached
causal Conv3D.

Every position of the latent map is a sequence over frames.  One block is

  norm -> projection to (x, z) -> causal_conv1d -> projections to (dt, B, C)
       -> selective_scan -> projection -> norm_join

and norm_join's second norm opens the next block, here the decoder's first
convolution.  Frames arrive in chunks; three states are carried between them,
all in the same manner: the convolution's last taps, the scan's states and the
Conv3D's last frames.  Frames are stored frame by frame ([T][P][C], P
positions) and passed to the operators as their [P, T, C] views, so nothing is
transposed.  ``MixerBlock.backward`` gives the block's gradients.

The other mixer, ``HeadsBlock``, works in heads:

  norm -> projection to (q, k, v, gate) -> rotary positions of q and k
       -> linear_attention -> group_norm of each head, gated -> projection
       -> norm_join

with the heads' states and the frame number carried between chunks.

  python -m causal_conv3d_video_amd.examples.stream_latents [--mixer heads]

streams a 30x52 latent of 384 channels in chunks of 1, 4 and 4 frames, compares
with one call over all frames, and prints the time of a chunk.  Weights are
random.
"""
import argparse
import math

import torch

import causal_conv3d_video_amd as cc3d


def _by_position(x):
    """[T, P, C] as it is stored -> its [P, T, C] view."""
    return x.transpose(0, 1)


class MixerState:
    """What one stream carries from chunk to chunk."""

    def __init__(self, block):
        self.taps = torch.zeros(block.positions, block.k - 1, block.inner, dtype=block.dtype, device=block.device)
        self.spare = torch.empty_like(self.taps)  # cache_out may not be cache_in: the two take turns
        self.h = torch.zeros(block.positions, block.inner, block.states, device=block.device)


class MixerBlock:
    state_type = MixerState

    def __init__(self, positions, channels, inner, states=16, rank=16, taps=4, dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def rn(*shape, scale=1.0, mean=0.0, dtype=dtype):
            return (torch.randn(*shape, generator=g, device=device) * scale + mean).to(dtype)

        self.positions, self.channels, self.inner = positions, channels, inner
        self.states, self.rank, self.k, self.dtype, self.device = states, rank, taps, dtype, device
        self.w = {
            "in_w": rn(2 * inner, channels, scale=channels ** -0.5), "conv_w": rn(taps, inner, scale=taps ** -0.5),
            "conv_b": rn(inner, scale=0.1), "bc_w": rn(rank + 2 * states, inner, scale=inner ** -0.5),
            "dt_w": rn(inner, rank, scale=rank ** -0.5), "out_w": rn(channels, inner, scale=inner ** -0.5),
            # steps between about 0.001 and 0.1
            "dt_bias": torch.empty(inner, device=device).uniform_(math.log(1e-3), math.log(0.1), generator=g),
            "a": -torch.arange(1, states + 1, device=device, dtype=torch.float32).repeat(inner, 1),
            "d": torch.ones(inner, device=device), "first_w": rn(channels, scale=0.1, mean=1.0),
            "post_w": rn(channels, scale=0.1, mean=1.0), "scale": rn(channels, scale=0.05, mean=0.5),
            "next_w": rn(channels, scale=0.1, mean=1.0),
        }
        self._plans = {}

    def plans(self, t):
        """The plans of a chunk of t frames and their workspaces, made once."""
        if t not in self._plans:
            p, rows = self.positions, t * self.positions
            self._plans[t] = got = {
                "first": cc3d.norm_join_plan(cc3d.make_join_desc(rows, self.channels, post=None, pre="rms", dtype=self.dtype)),
                "conv": cc3d.causal_conv1d_plan(cc3d.make_conv1d_desc(p, t, self.inner, self.k, act="silu", dtype=self.dtype)),
                "scan": cc3d.selective_scan_plan(cc3d.make_scan_desc(p, t, self.inner, self.states, dtype=self.dtype)),
                "join": cc3d.norm_join_plan(cc3d.make_join_desc(rows, self.channels, post="rms", pre="rms", act="silu",
                                                                dtype=self.dtype)),
            }
            most = max(plan.info[k] for plan in got.values() for k in ("workspace_bytes", "backward_workspace_bytes"))
            got["space"] = torch.empty(most, dtype=torch.uint8, device=self.device)
        return self._plans[t]

    def _new(self, t, width):
        return torch.empty(t, self.positions, width, dtype=self.dtype, device=self.device)

    def forward(self, frames, state, keep=None):
        """frames [T, P, C] -> (x_out, h_out): the residual stream and the next
        block's normed input.  ``state`` (MixerState) is carried on; ``keep``
        (a dict) receives what ``backward`` needs."""
        t, w, i = frames.shape[0], self.w, self.inner
        p = self.plans(t)
        normed = torch.empty_like(frames)
        cc3d.norm_join_forward(p["first"], None, frames, h_out=normed, pre_w=w["first_w"])
        xz = normed @ w["in_w"].T
        x, z = _by_position(xz[..., :i]), _by_position(xz[..., i:])
        if keep is not None:
            keep.update(frames=frames, normed=normed, xz=xz, taps=state.taps.clone(), h=state.h.clone())
        u = self._new(t, i)
        cc3d.causal_conv1d_forward(p["conv"], x, w["conv_w"], w["conv_b"], _by_position(u), cache_in=state.taps,
                                   cache_out=state.spare)
        state.taps, state.spare = state.spare, state.taps
        low = u @ w["bc_w"].T
        r, s = self.rank, self.states
        dt = low[..., :r] @ w["dt_w"].T
        y = self._new(t, i)
        cc3d.selective_scan_forward(p["scan"], _by_position(u), _by_position(dt), w["a"], _by_position(low[..., r:r + s]),
                                    _by_position(low[..., r + s:]), _by_position(y), d=w["d"], z=z, dt_bias=w["dt_bias"],
                                    h_in=state.h, h_out=state.h, workspace=p["space"])
        out = y @ w["out_w"].T
        x_out, h_out = torch.empty_like(frames), torch.empty_like(frames)
        cc3d.norm_join_forward(p["join"], out, frames, x_out=x_out, h_out=h_out, scale=w["scale"], post_w=w["post_w"],
                               pre_w=w["next_w"])
        if keep is not None:
            keep.update(u=u, low=low, dt=dt, y=y, out=out)
        return x_out, h_out

    def backward(self, kept, dx_out, dh_out):
        """Gradients of the frames and of every weight (a dict) for a chunk
        forwarded with ``keep``; the carried states are taken as given."""
        t, w, i, r, s = dx_out.shape[0], self.w, self.inner, self.rank, self.states
        p = self.plans(t)
        f32 = {"dtype": torch.float32, "device": self.device}
        g = {k: torch.empty(w[k].shape, **f32) for k in ("conv_w", "conv_b", "a", "d", "dt_bias", "first_w", "post_w", "scale",
                                                         "next_w")}

        def rows(v):
            return v.reshape(-1, v.shape[-1])

        dframes, dout = torch.empty_like(dx_out), torch.empty_like(dx_out)
        cc3d.norm_join_backward(p["join"], kept["out"], kept["frames"], dx_out=dx_out, dh=dh_out, scale=w["scale"],
                                post_w=w["post_w"], pre_w=w["next_w"], dy=dout, dresidual=dframes, dscale=g["scale"],
                                dpost_w=g["post_w"], dpre_w=g["next_w"], workspace=p["space"])
        g["out_w"] = rows(dout).T @ rows(kept["y"])
        dy = dout @ w["out_w"]
        dxz, dlow = torch.empty_like(kept["xz"]), torch.empty_like(kept["low"])
        du, ddt = self._new(t, i), self._new(t, i)
        low = kept["low"]
        cc3d.selective_scan_backward(
            p["scan"], _by_position(kept["u"]), _by_position(kept["dt"]), w["a"], _by_position(low[..., r:r + s]),
            _by_position(low[..., r + s:]), _by_position(dy), d=w["d"], z=_by_position(kept["xz"][..., i:]),
            dt_bias=w["dt_bias"], h_in=kept["h"], du=_by_position(du), ddt=_by_position(ddt), da=g["a"],
            db=_by_position(dlow[..., r:r + s]), dc=_by_position(dlow[..., r + s:]), dd=g["d"],
            dz=_by_position(dxz[..., i:]), ddt_bias=g["dt_bias"], workspace=p["space"])
        g["dt_w"] = rows(ddt).T @ rows(low[..., :r])
        dlow[..., :r] = ddt @ w["dt_w"]
        g["bc_w"] = rows(dlow).T @ rows(kept["u"])
        du += dlow @ w["bc_w"]
        cc3d.causal_conv1d_backward(p["conv"], _by_position(kept["xz"][..., :i]), w["conv_w"], w["conv_b"], _by_position(du),
                                    dx=_by_position(dxz[..., :i]), dw=g["conv_w"], db=g["conv_b"], cache_in=kept["taps"],
                                    workspace=p["space"])
        g["in_w"] = rows(dxz).T @ rows(kept["normed"])
        dnormed = dxz @ w["in_w"]
        dfirst = torch.empty_like(dframes)
        cc3d.norm_join_backward(p["first"], None, kept["frames"], dh=dnormed, pre_w=w["first_w"], dresidual=dfirst,
                                dpre_w=g["first_w"], workspace=p["space"])
        return dframes + dfirst, g


class HeadsState:
    """What one stream carries from chunk to chunk."""

    def __init__(self, block):
        self.h = torch.zeros(block.positions, block.heads, block.width, block.width, device=block.device)
        self.frames = torch.zeros(block.positions, dtype=torch.int32, device=block.device)


class HeadsBlock:
    """The mixer in heads of `width` channels: same call, state and gradients as MixerBlock."""

    state_type = HeadsState

    def __init__(self, positions, channels, inner, heads=None, dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def rn(*shape, scale=1.0, mean=0.0, dtype=dtype):
            return (torch.randn(*shape, generator=g, device=device) * scale + mean).to(dtype)

        self.positions, self.channels, self.inner = positions, channels, inner
        self.heads = heads or max(1, inner // 64)
        self.width, self.dtype, self.device = inner // self.heads, dtype, device
        self.w = {
            "in_w": rn(4 * inner, channels, scale=channels ** -0.5), "out_w": rn(channels, inner, scale=inner ** -0.5),
            # memories of 4 to some 100 frames
            "log_decay": torch.log1p(-torch.exp2(torch.linspace(-2, -7, self.heads, device=device))),
            "head_w": rn(inner, scale=0.1, mean=1.0), "head_b": rn(inner, scale=0.1),
            "first_w": rn(channels, scale=0.1, mean=1.0), "post_w": rn(channels, scale=0.1, mean=1.0),
            "scale": rn(channels, scale=0.05, mean=0.5), "next_w": rn(channels, scale=0.1, mean=1.0),
        }
        self._plans = {}

    def plans(self, t):
        """The plans of a chunk of t frames and their workspaces, made once."""
        if t not in self._plans:
            p, rows, h, d = self.positions, t * self.positions, self.heads, self.width
            self._plans[t] = got = {
                "first": cc3d.norm_join_plan(cc3d.make_join_desc(rows, self.channels, post=None, pre="rms", dtype=self.dtype)),
                "rotary": cc3d.rotary_plan(cc3d.make_rotary_desc(p, t, h, h, d, rot=d // 2 * 2, dtype=self.dtype)),
                "linear": cc3d.linear_attention_plan(cc3d.make_linear_attention_desc(p, t, h, d, d, dtype=self.dtype)),
                "heads": cc3d.group_norm_plan(cc3d.make_group_norm_desc(rows, 1, self.inner, h, dtype=self.dtype)),
                "join": cc3d.norm_join_plan(cc3d.make_join_desc(rows, self.channels, post="rms", pre="rms", act="silu",
                                                                dtype=self.dtype)),
            }
            most = max(plan.info[k] for plan in got.values() for k in ("workspace_bytes", "backward_workspace_bytes"))
            got["space"] = torch.empty(most, dtype=torch.uint8, device=self.device)
        return self._plans[t]

    def _new(self, t, width):
        return torch.empty(t, self.positions, width, dtype=self.dtype, device=self.device)

    def _parts(self, x):
        """[T, P, 4 inner] -> the [P, T, inner] views of q, k, v and gate."""
        return [_by_position(v) for v in x.split(self.inner, -1)]

    def forward(self, frames, state, keep=None):
        """frames [T, P, C] -> (x_out, h_out); ``state`` (HeadsState) is carried
        on; ``keep`` (a dict) receives what ``backward`` needs."""
        t, w, i = frames.shape[0], self.w, self.inner
        p = self.plans(t)
        normed = torch.empty_like(frames)
        cc3d.norm_join_forward(p["first"], None, frames, h_out=normed, pre_w=w["first_w"])
        qkvg = normed @ w["in_w"].T
        q, k, v, gate = self._parts(qkvg)
        if keep is not None:
            keep.update(frames=frames, normed=normed, qkvg=qkvg, h=state.h.clone(), at=state.frames.clone())
        # (v and gate are left as they are: q and k turn in their places)
        cc3d.rotary_forward(p["rotary"], q, k, q, k, offsets=state.frames)
        o = self._new(t, i)
        cc3d.linear_attention_forward(p["linear"], q, k, v, _by_position(o), log_decay=w["log_decay"], h_in=state.h,
                                      h_out=state.h, workspace=p["space"])
        state.frames += t
        rows = (t * self.positions, 1, i)
        y, stats = self._new(t, i), torch.empty(rows[0], self.heads, 2, device=self.device)
        cc3d.group_norm_forward(p["heads"], o.view(rows), y.view(rows), w=w["head_w"], b=w["head_b"], stats=stats)
        z = y * torch.nn.functional.silu(qkvg[..., 3 * i:])
        out = z @ w["out_w"].T
        x_out, h_out = torch.empty_like(frames), torch.empty_like(frames)
        cc3d.norm_join_forward(p["join"], out, frames, x_out=x_out, h_out=h_out, scale=w["scale"], post_w=w["post_w"],
                               pre_w=w["next_w"])
        if keep is not None:
            keep.update(o=o, stats=stats, y=y, z=z, out=out)
        return x_out, h_out

    def backward(self, kept, dx_out, dh_out):
        """Gradients of the frames and of every weight (a dict) for a chunk
        forwarded with ``keep``; the carried states are taken as given."""
        t, w, i = dx_out.shape[0], self.w, self.inner
        p = self.plans(t)
        f32 = {"dtype": torch.float32, "device": self.device}
        g = {k: torch.empty(w[k].shape, **f32) for k in ("log_decay", "head_w", "head_b", "first_w", "post_w", "scale", "next_w")}

        def rows(v):
            return v.reshape(-1, v.shape[-1])

        dframes, dout = torch.empty_like(dx_out), torch.empty_like(dx_out)
        cc3d.norm_join_backward(p["join"], kept["out"], kept["frames"], dx_out=dx_out, dh=dh_out, scale=w["scale"],
                                post_w=w["post_w"], pre_w=w["next_w"], dy=dout, dresidual=dframes, dscale=g["scale"],
                                dpost_w=g["post_w"], dpre_w=g["next_w"], workspace=p["space"])
        g["out_w"] = rows(dout).T @ rows(kept["z"])
        dz = dout @ w["out_w"]
        gate = kept["qkvg"][..., 3 * i:]
        s = torch.sigmoid(gate.float())
        dqkvg = torch.empty_like(kept["qkvg"])
        dqkvg[..., 3 * i:] = (dz * kept["y"]).float() * (s * (1 + gate.float() * (1 - s)))
        dy, do = dz * (gate * s.to(self.dtype)), self._new(t, i)
        one = (t * self.positions, 1, i)
        cc3d.group_norm_backward(p["heads"], kept["o"].view(one), dy.view(one), w=w["head_w"], b=w["head_b"],
                                 stats=kept["stats"], dx=do.view(one), dw=g["head_w"], db=g["head_b"], workspace=p["space"])
        q, k, v, _ = self._parts(kept["qkvg"])
        dq, dk, dv, _ = self._parts(dqkvg)
        cc3d.linear_attention_backward(p["linear"], q, k, v, _by_position(do), log_decay=w["log_decay"], h_in=kept["h"], dq=dq,
                                       dk=dk, dv=dv, dlog_decay=g["log_decay"], workspace=p["space"])
        cc3d.rotary_backward(p["rotary"], dq, dk, dq, dk, offsets=kept["at"])
        g["in_w"] = rows(dqkvg).T @ rows(kept["normed"])
        dnormed = dqkvg @ w["in_w"]
        dfirst = torch.empty_like(dframes)
        cc3d.norm_join_backward(p["first"], None, kept["frames"], dh=dnormed, pre_w=w["first_w"], dresidual=dfirst,
                                dpre_w=g["first_w"], workspace=p["space"])
        return dframes + dfirst, g


MIXERS = {"scan": MixerBlock, "heads": HeadsBlock}


class LatentDecoder:
    """The mixer and the decoder's first cached causal Conv3D behind it."""

    def __init__(self, height, width, channels, out_channels, inner, dtype=torch.bfloat16, device="cuda", seed=0, mixer="scan"):
        self.h, self.w_, self.c, self.out = height, width, channels, out_channels
        self.block = MIXERS[mixer](height * width, channels, inner, dtype=dtype, device=device, seed=seed)
        g = torch.Generator(device=device).manual_seed(seed + 1)
        self.weight = (torch.randn(out_channels, 3, 3, 3, channels, generator=g, device=device)
                       * (27 * channels) ** -0.5).to(dtype)
        self.bias = torch.zeros(out_channels, dtype=dtype, device=device)
        self.dtype, self.device = dtype, device
        self._plans = {}
        self.reset()

    def reset(self):
        self.state, self.frames = self.block.state_type(self.block), None

    def __call__(self, latents):
        """latents [T, H, W, C] -> [T, H, W, C_out], carrying every state on."""
        t = latents.shape[0]
        _, mixed = self.block.forward(latents.reshape(t, self.h * self.w_, self.c), self.state)
        x = mixed.reshape(1, t, self.h, self.w_, self.c)
        before = 0 if self.frames is None else self.frames.shape[1]
        if (t, before) not in self._plans:
            self._plans[t, before] = cc3d.causal_conv3d_plan(
                cc3d.make_desc(1, self.c, self.out, self.h, self.w_, t, before, dtype=self.dtype))
        plan = self._plans[t, before]
        shapes = plan.shapes()
        out = torch.empty(shapes["out"], dtype=self.dtype, device=self.device)
        carry = torch.empty(shapes["cache_out"], dtype=self.dtype, device=self.device)
        cc3d.causal_conv3d_forward(plan, x, self.frames, self.weight, self.bias, out, carry)
        self.frames = carry
        return out[0]


def main():
    args = argparse.ArgumentParser()
    args.add_argument("--mixer", choices=sorted(MIXERS), default="scan")
    h, w, c = 30, 52, 384
    model = LatentDecoder(h, w, c, 192, 768, mixer=args.parse_args().mixer)
    g = torch.Generator(device="cuda").manual_seed(7)
    latents = torch.randn(9, h, w, c, generator=g, device="cuda").to(torch.bfloat16)
    whole = model(latents)
    model.reset()
    chunks = [model(part) for part in latents.split([1, 4, 4])]
    off = float((torch.cat(chunks).float() - whole.float()).abs().max())
    print("9 frames in chunks of 1, 4 and 4 against one call: largest difference %.4f beside values of up to %.2f"
          % (off, float(whole.float().abs().max())))
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(3):
        model(latents[5:])
    begin.record()
    for _ in range(20):
        model(latents[5:])
    end.record()
    torch.cuda.synchronize()
    print("a chunk of 4 frames of %dx%d, %d channels: %.3f ms" % (h, w, c, begin.elapsed_time(end) / 20))


if __name__ == "__main__":
    main()
