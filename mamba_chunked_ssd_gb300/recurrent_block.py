"""A block with a gated linear recurrence, for training and for serving, from the library's entry points.

    n -> projection -> x -> causal convolution, SiLU -> gates r | i (projection)
                    -> z                             -> gated linear recurrence, gated by SiLU(z)
      -> projection -> norm, scale, + residual -> norm -> the next block's n

The projections are library matrix products; x, z and r, i stay slices of what
they come out of, and so do their gradients.  ``forward`` runs whole (ragged)
sequences, ``backward`` gives the gradients of all of its inputs and weights,
``step`` runs one token of each sequence; the convolution's last inputs and the
fp32 state are carried from call to call.

Past a row's length n may hold anything: no result has a part of it.  The residual
goes on there as it came (the norms know no lengths), with its own gradient: it and
the gradients that come in have to be finite there.

Run ``python -m mamba_chunked_ssd_gb300.recurrent_block`` for a training step on a ragged batch and
a few decoded tokens on random weights (``--help`` for the sizes).
"""
from __future__ import annotations

import argparse
from dataclasses import dataclass

import torch

from . import binding as bd


@dataclass
class BlockState:
    """What a sequence carries from call to call (of each batch row)."""
    conv: torch.Tensor   # [b, W - 1, channels], dtype of the block
    state: torch.Tensor  # [b, channels] fp32


class RecurrentBlock:
    """Random-initialised block of width ``d_model`` with ``channels`` of recurrence."""

    def __init__(self, d_model, channels, conv_width=4, dtype=torch.bfloat16, device="cuda", seed=0):
        bd.load_library()
        g = torch.Generator(device=device).manual_seed(seed)
        n = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
        self.channels, self.width = channels, conv_width
        w = {"in": n(d_model, 2 * channels) * d_model ** -0.5, "gates": n(channels, 2 * channels) * channels ** -0.5,
             "out": n(channels, d_model) * channels ** -0.5}
        self.w = {k: t.to(dtype) for k, t in w.items()}
        self.w.update(conv=n(channels, conv_width) * conv_width ** -0.5, conv_bias=0.1 * n(channels),
                      A=8 * torch.log(0.9 + 0.099 * torch.rand(channels, generator=g, device=device)),
                      post=1 + 0.1 * n(d_model), scale=torch.full((d_model,), 0.5, device=device),
                      pre=1 + 0.1 * n(d_model))

    def new_state(self, batch) -> BlockState:
        w = self.w["in"]
        return BlockState(torch.zeros(batch, self.width - 1, self.channels, device=w.device, dtype=w.dtype),
                          torch.zeros(batch, self.channels, device=w.device))

    def _norms(self, out, residual):
        w = self.w
        return bd.mamba2_block_norm_fwd(out, residual, post_weight=w["post"], scale=w["scale"], pre_weight=w["pre"])

    def forward(self, n, residual, carried: BlockState | None = None, lengths=None, keep=False):
        """n [b, L, d_model] and the residual stream (fp32 or n's dtype) -> (the next n, the
        next residual, the state after each row's tokens, and with ``keep`` what backward needs)."""
        w, C = self.w, self.channels
        x, z = (n @ w["in"]).split(C, -1)
        u, conv = bd.mamba2_causal_conv_fwd(x, w["conv"], bias=w["conv_bias"], lengths=lengths,
                                            initial_state=carried.conv if carried else None)
        r, i = (u @ w["gates"]).split(C, -1)
        y, state, chunks = bd.mamba2_glr_fwd(u, r, i, w["A"], z=z, lengths=lengths, want_chunk_states=keep,
                                             initial_state=carried.state if carried else None)
        out = y @ w["out"]
        res, nxt = self._norms(out, residual)
        kept = (n, x, z, u, r, i, y, chunks, out, res, carried.conv if carried else None, lengths) if keep else None
        return nxt, res, BlockState(conv, state), kept

    def backward(self, kept, dnext, dres, dafter: BlockState | None = None):
        """Gradients from those of the next n, the next residual and the state after each row's tokens
        (None: zeros): (of n, of the residual, of the carried state, of the weights by name)."""
        w, C = self.w, self.channels
        n, x, z, u, r, i, y, chunks, out, res, conv, lengths = kept
        flat = lambda t: t.flatten(0, -2)  # noqa: E731
        dw = {}
        dout, _, dresidual, dw["post"], dw["scale"], dw["pre"] = bd.mamba2_block_norm_bwd(
            dres, dnext, out, res, post_weight=w["post"], scale=w["scale"], pre_weight=w["pre"])
        dw["out"] = flat(y).T @ flat(dout)
        dproj, dgates = (torch.empty(*u.shape[:-1], 2 * C, dtype=u.dtype, device=u.device) for _ in range(2))
        dx, dz = dproj.split(C, -1)
        dr, di = dgates.split(C, -1)
        du, _, _, _, dw["A"], dstate = bd.mamba2_glr_bwd(dout @ w["out"].T, u, r, i, w["A"], chunks, z=z, lengths=lengths,
                                                         dfinal_state=dafter.state if dafter else None,
                                                         dr=dr, di=di, dz=dz)
        dw["gates"] = flat(u).T @ flat(dgates)
        _, dw["conv"], dw["conv_bias"], dconv = bd.mamba2_causal_conv_bwd(
            du + dgates @ w["gates"].T, x, w["conv"], bias=w["conv_bias"], initial_state=conv, lengths=lengths,
            dfinal_state=dafter.conv if dafter else None, dx=dx)
        if lengths is not None:  # (dproj is 0 past a row's length, but 0 times what is not finite is not)
            past = torch.arange(n.shape[1], device=n.device) >= lengths[:, None]
            n = n.masked_fill(past[..., None], 0)
        dw["in"] = flat(n).T @ flat(dproj)
        return dproj @ w["in"].T, dresidual, BlockState(dconv, dstate), dw

    def step(self, n, residual, carried: BlockState):
        """One token, n and residual [b, d_model] -> (the next n, the next residual); the state is updated in place."""
        w, C = self.w, self.channels
        x, z = (n @ w["in"]).split(C, -1)
        u, _ = bd.mamba2_causal_conv_step(x, w["conv"], state_in=carried.conv, bias=w["conv_bias"], state_out=carried.conv)
        r, i = (u @ w["gates"]).split(C, -1)
        y, _ = bd.mamba2_glr_step(u, r, i, w["A"], z=z, state_in=carried.state, state_out=carried.state)
        res, nxt = self._norms(y @ w["out"], residual)
        return nxt, res


def main(argv=None):
    ap = argparse.ArgumentParser(description="A training step of the block on a ragged batch, and a few decoded tokens.")
    for name, default in (("batch", 2), ("tokens", 300), ("width", 1024), ("channels", 1280), ("decode", 4)):
        ap.add_argument(f"--{name}", type=int, default=default)
    a = ap.parse_args(argv)
    block = RecurrentBlock(a.width, a.channels)
    n = torch.randn(a.batch, a.tokens, a.width, device="cuda").bfloat16()
    res = torch.randn(a.batch, a.tokens, a.width, device="cuda")
    # rows of lengths between L and about half of it
    m = torch.tensor([a.tokens - a.tokens * k // (2 * a.batch + 1) for k in range(a.batch)], dtype=torch.int32, device="cuda")
    nxt, out, carried, kept = block.forward(n, res, lengths=m, keep=True)
    dn, _, _, dw = block.backward(kept, torch.ones_like(nxt), torch.zeros_like(out))
    last = torch.arange(a.batch, device="cuda"), m.long() - 1
    n, res = nxt[last], out[last]
    for _ in range(a.decode):
        n, res = block.step(n, res, carried)
    bd.mamba2_check_device_status()
    print(f"forward and backward {tuple(nxt.shape)}, gradient of {len(dw)} weights, {a.decode} tokens decoded, "
          f"last output's rms {n.float().square().mean().sqrt().item():.3f}")


if __name__ == "__main__":
    main()
