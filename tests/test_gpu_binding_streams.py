"""Outputs of a call on a stream that is passed come from that stream's memory pool
and hold what a call on the current stream gives."""
import pytest
import torch

from mamba_chunked_ssd_gb300 import binding as bd
from test_gpu_gated_delta import BF16, gdr_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mamba_chunked_ssd_gb300 import build_lib
    build_lib.build()
    bd.load_library()


def pool_stream(t):
    """The stream whose pool a tensor's memory is from."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]


def calls():
    d, h0 = gdr_inputs(2, 40, 4, 2, 64, 128, BF16)
    one = {n: t[:, 0].contiguous() for n, t in d.items()}
    n = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    x, w, s0 = n(2, 40, 64).bfloat16(), n(64, 4), n(2, 3, 64).bfloat16()
    dt, A, B = n(2, 40, 4).abs() * 0.1, -n(4).abs(), d["k"]
    return {
        "gdr_fwd": lambda **k: bd.mamba2_gdr_fwd(**d, initial_state=h0, **k),
        "gdr_step": lambda **k: bd.mamba2_gdr_step(**one, state_in=h0, **k),
        "conv_fwd": lambda **k: bd.mamba2_causal_conv_fwd(x, w, initial_state=s0, **k),
        "conv_step": lambda **k: bd.mamba2_causal_conv_step(x[:, 0].contiguous(), w, state_in=s0, **k),
        "norm": lambda **k: (bd.mamba2_group_norm(x, None, 2, **k),),
        "ssd_fwd": lambda **k: bd.mamba2_ssd_fwd(d["v"], dt, A, B, d["q"], 64, initial_state=h0, **k),
        "ssd_step": lambda **k: bd.mamba2_ssd_step(one["v"], dt[:, 0].contiguous(), A, one["k"], one["q"], state_in=h0, **k),
    }


@pytest.mark.parametrize("name", ["gdr_fwd", "gdr_step", "conv_fwd", "conv_step", "norm", "ssd_fwd", "ssd_step"])
def test_outputs_come_from_the_pool_of_the_stream(name):
    call = calls()[name]
    want = call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = call(stream=s)
    s.synchronize()
    for g, w in zip(got, want):
        assert pool_stream(g) == s.cuda_stream and pool_stream(w) == torch.cuda.current_stream().cuda_stream
        assert torch.equal(g, w)
