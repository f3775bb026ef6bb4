"""A gated-delta-rule layer for inference, from the library's entry points.

    u -> projection -> [q | k | v] -> causal convolution, SiLU -> gated delta rule
                    -> z, a, b        (g = -A softplus(a + bias), beta = sigmoid(b))
      -> group norm per head, gated by SiLU(z) -> projection

The projections are library matrix products; q, k, v and z stay slices of what
they come out of, since every operator takes a token stride.  ``prefill`` runs
whole (ragged) sequences, ``step`` one token of each; both carry the
convolution's last inputs and the fp32 state, which a later call continues from.

Run ``python -m mamba_chunked_ssd_gb300.gated_delta_layer`` for a ragged batch of
prompts and a few decoded tokens on random weights (``--help`` for the sizes).
"""
from __future__ import annotations

import argparse
from dataclasses import dataclass

import torch

from . import binding as bd


@dataclass
class LayerState:
    """What a sequence carries from call to call (of each batch row)."""
    conv: torch.Tensor   # [b, W - 1, channels of q | k | v], dtype of the layer
    state: torch.Tensor  # [b, nh, S, H] fp32


class GatedDeltaLayer:
    """Random-initialised layer of width ``d_model``: ``nheads`` heads of
    ``headdim`` columns over ``ngroups`` shared q/k groups of ``dstate``."""

    def __init__(self, d_model, nheads, ngroups, headdim, dstate, conv_width=4, dtype=torch.bfloat16, device="cuda",
                 seed=0):
        bd.load_library()
        r = torch.Generator(device=device).manual_seed(seed)
        n = lambda *s: torch.randn(*s, generator=r, device=device)  # noqa: E731
        self.nheads, self.ngroups, self.headdim, self.dstate = nheads, ngroups, headdim, dstate
        self.qk, self.inner, self.width = ngroups * dstate, nheads * headdim, conv_width
        self.channels = 2 * self.qk + self.inner                      # q | k | v
        self.parts = [self.channels, self.inner, nheads, nheads]      # ... | z | a | b
        self.w_in = (n(d_model, sum(self.parts)) * d_model ** -0.5).to(dtype)
        self.w_out = (n(self.inner, d_model) * self.inner ** -0.5).to(dtype)
        self.w_conv, self.b_conv = n(self.channels, conv_width) * conv_width ** -0.5, 0.1 * n(self.channels)
        self.w_norm = 1 + 0.1 * n(self.inner)
        self.A = 1 + 15 * torch.rand(nheads, generator=r, device=device)
        step = torch.exp(torch.rand(nheads, generator=r, device=device) * 4.6 - 6.9)  # 1e-3 .. 0.1
        self.dt_bias = step + torch.log(-torch.expm1(-step))                           # softplus inverse

    def new_state(self, batch) -> LayerState:
        w = self.w_in
        return LayerState(torch.zeros(batch, self.width - 1, self.channels, device=w.device, dtype=w.dtype),
                          torch.zeros(batch, self.nheads, self.dstate, self.headdim, device=w.device))

    def _project(self, u):
        qkv, z, a, b = torch.split(u @ self.w_in, self.parts, -1)
        g = -self.A * torch.nn.functional.softplus(a.float() + self.dt_bias)
        return qkv, z, g, torch.sigmoid(b.float())

    def _qkv(self, x):
        q, k, v = torch.split(x, [self.qk, self.qk, self.inner], -1)
        return (q.unflatten(-1, (self.ngroups, self.dstate)), k.unflatten(-1, (self.ngroups, self.dstate)),
                v.unflatten(-1, (self.nheads, self.headdim)))

    def _finish(self, y, z):
        y = bd.mamba2_group_norm(y.flatten(-2), self.w_norm, self.nheads, z=z, mode="after")
        return y @ self.w_out

    def prefill(self, u, carried: LayerState | None = None, lengths=None):
        """u [b, L, d_model] (lengths [b] int32 for a ragged batch) -> (output
        [b, L, d_model], the state after each row's tokens)."""
        qkv, z, g, beta = self._project(u)
        x, conv = bd.mamba2_causal_conv_fwd(qkv, self.w_conv, bias=self.b_conv, lengths=lengths,
                                            initial_state=carried.conv if carried else None)
        y, state = bd.mamba2_gdr_fwd(*self._qkv(x), g, beta, qk_l2norm=True, lengths=lengths,
                                     initial_state=carried.state if carried else None)
        return self._finish(y, z), LayerState(conv, state)

    def step(self, u, carried: LayerState):
        """u [b, d_model] -> output [b, d_model]; the state is updated in place."""
        qkv, z, g, beta = self._project(u)
        x, _ = bd.mamba2_causal_conv_step(qkv, self.w_conv, state_in=carried.conv, bias=self.b_conv,
                                          state_out=carried.conv)
        y, _ = bd.mamba2_gdr_step(*self._qkv(x), g, beta, state_in=carried.state, qk_l2norm=True,
                                  state_out=carried.state)
        return self._finish(y, z)


def main(argv=None):
    ap = argparse.ArgumentParser(description="A batch of prompts and a few decoded tokens through the layer.")
    for name, default in (("batch", 2), ("tokens", 300), ("width", 1024), ("heads", 16), ("groups", 8),
                          ("headdim", 64), ("dstate", 128), ("decode", 4)):
        ap.add_argument(f"--{name}", type=int, default=default)
    a = ap.parse_args(argv)
    layer = GatedDeltaLayer(a.width, a.heads, a.groups, a.headdim, a.dstate)
    u = torch.randn(a.batch, a.tokens, a.width, device="cuda").bfloat16()
    # rows of every length from L down
    n = torch.tensor([a.tokens - a.tokens * i // (2 * a.batch) for i in range(a.batch)], dtype=torch.int32, device="cuda")
    out, carried = layer.prefill(u, lengths=n)
    token = out[torch.arange(a.batch, device="cuda"), n.long() - 1]
    for _ in range(a.decode):
        token = layer.step(token, carried)
    bd.mamba2_check_device_status()
    print(f"prefill {tuple(out.shape)}, {a.decode} tokens decoded, state {tuple(carried.state.shape)}, "
          f"last output's rms {token.float().square().mean().sqrt().item():.3f}")


if __name__ == "__main__":
    main()
