"""The recurrent block on what a training program hands it: padding that is not finite."""
import pytest
import torch

from mamba_chunked_ssd_gb300 import binding as bd
from mamba_chunked_ssd_gb300.recurrent_block import RecurrentBlock
from test_gpu_recurrent_block import BF16, FP32, _lib  # noqa: F401

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
