"""The recurrent block on what a training program hands it: padding that is not finite, and
sequences in segments, whose carried state passes gradients back.

Tolerance of the fp32 block: that of its whole pass, 4e-5 of the largest value (tests of the block beside
this file); a weight's gradient from two segments has the errors of both, each of its own largest value.
"""
import pytest
import torch

import gated_linear_ref as ref
from mamba_chunked_ssd_gb300 import binding as bd
from mamba_chunked_ssd_gb300.recurrent_block import BlockState, RecurrentBlock
from test_gpu_recurrent_block import BF16, FP32, TOL, _lib, close, plain  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [FP32, BF16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_what_lies_past_a_rows_end_is_in_no_gradient(value, dtype):
    b, L, d, C = 3, 70, 40, 64
    block = RecurrentBlock(d, C, dtype=dtype)
    g = torch.Generator().manual_seed(5)
    t = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    n, res, dn, dr = t(b, L, d).to(dtype).cuda(), t(b, L, d).cuda(), t(b, L, d).to(dtype).cuda(), t(b, L, d).cuda()
    lengths = torch.tensor([70, 33, 0], dtype=torch.int32, device="cuda")
    past = (torch.arange(L, device="cuda") >= lengths[:, None])[..., None]
    results = []
    for fill in (0.0, value):
        nxt, out, after, kept = block.forward(n.masked_fill(past, fill), res, lengths=lengths, keep=True)
        gn, gres, gstate, gw = block.backward(kept, dn, dr)
        results.append({"next": nxt, "residual": out, "state": after.state, "conv": after.conv, "n": gn, "res": gres,
                        "dstate": gstate.state, "dconv": gstate.conv, **gw})
    bd.mamba2_check_device_status()
    for name, want in results[0].items():
        assert torch.isfinite(want).all() and torch.equal(results[1][name], want), name


def test_gradients_through_segments():
    """A sequence in two segments, each with its backward pass, against the whole one differentiated in fp64."""
    b, L, d, C, cut = 2, 90, 40, 64, 51
    block = RecurrentBlock(d, C, dtype=FP32)
    g = torch.Generator().manual_seed(6)
    t = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    n, res, dn, dr = t(b, L, d), t(b, L, d), t(b, L, d), t(b, L, d)
    state, dstate = BlockState(t(b, 3, C), t(b, C)), BlockState(t(b, 3, C), t(b, C))
    part = lambda v, k: (v[:, :cut], v[:, cut:])[k].contiguous()  # noqa: E731
    nxt, out, conv, h, leaves = plain(block, n, res, state, None)
    loss = sum((a * ref.f64(v)).sum() for a, v in ((nxt, dn), (out, dr), (conv, dstate.conv), (h, dstate.state)))
    auto = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))

    _, _, middle, first = block.forward(part(n, 0), part(res, 0), state, keep=True)
    _, _, last, second = block.forward(part(n, 1), part(res, 1), middle, keep=True)
    close(last.conv, conv, TOL[FP32], "conv"), close(last.state, h, TOL[FP32], "state")
    gn2, gres2, back, gw2 = block.backward(second, part(dn, 1), part(dr, 1), dstate)
    gn1, gres1, back, gw1 = block.backward(first, part(dn, 0), part(dr, 0), back)
    bd.mamba2_check_device_status()
    for got, name in ((torch.cat([gn1, gn2], 1), "n"), (torch.cat([gres1, gres2], 1), "res"), (back.conv, "conv_state"),
                      (back.state, "state")):
        close(got, auto[name], TOL[FP32], "gradient of " + name)
    for k, v in gw1.items():
        err = ((v + gw2[k]).cpu().double() - auto[k]).abs().max().item()
        most = TOL[FP32] * (v.abs().max() + gw2[k].abs().max()).item()
        assert err <= most, f"gradient of {k}: {err:.3e}, at most {most:.3e}"
