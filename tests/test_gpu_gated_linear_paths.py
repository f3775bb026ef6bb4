"""The gated linear recurrence on paths that sizes choose: strips that are left over when every SM has as
many.

Tolerances are those of the parity tests beside this file, on max|err| / max|ref|: a value that
leaves as bf16 is rounded once, by 2^-8 of it at most; the fp32 work before it is within 1e-5; a
sum over tokens or rows within 1e-5 of the sum of its terms' absolute values.
"""
import ctypes

import pytest
import torch

import gated_linear_ref as ref
from mamba_chunked_ssd_gb300 import binding as bd
from test_gpu_gated_linear import BF16, FP32, TOL, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mamba_chunked_ssd_gb300 import build_lib
    build_lib.build()
    bd.load_library()


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# --------------------------------------------------------- left-over strips
LEFT = 24  # strips beyond a whole number to every SM


def left_over(per, gated, dtype, L=1033):
    """Four rows, the last shorter, with `per` strips on every SM and LEFT more; each strip is one of known channels."""
    C = (per * sms() + LEFT) // 4 * 32
    n = gen(per)
    base = {k: n(4, L, 32).to(dtype) for k in ("x", "r", "i", "z", "dy")}
    base["A"], base["h0"], base["df"] = -torch.exp(n(32)), n(4, 32), n(4, 32)
    if not gated:
        base["z"] = None
    lengths = torch.tensor([L, L, L, L - 40], dtype=torch.int32)
    wide = {k: None if t is None else t.cuda().repeat(*[1] * (t.dim() - 1), C // 32) for k, t in base.items()}
    return base, wide, lengths.cuda(), C


def calls(wide, lengths, C):
    """Forward and backward with all their tensors given, and those tensors."""
    x = wide["x"]
    b, L, dt = x.shape[0], x.shape[1], x.dtype
    e = lambda *s, t=dt: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
    fwd = {"y": e(b, L, C), "final_state": e(b, C, t=FP32), "chunk_states": e(b, -(-L // 64), C, t=FP32)}
    bwd = {k: e(b, L, C) for k in ("dx", "dr", "di") + (("dz",) if wide["z"] is not None else ())}
    bwd.update(dA=e(C, t=FP32), dinitial_state=e(b, C, t=FP32))
    ws = e(b * C * 4 + 256, t=torch.uint8)

    def forward(stream=None):
        bd.mamba2_glr_fwd(x, wide["r"], wide["i"], wide["A"], z=wide["z"], initial_state=wide["h0"], lengths=lengths,
                          stream=stream, **fwd)

    def backward(stream=None):
        bd.mamba2_glr_bwd(wide["dy"], x, wide["r"], wide["i"], wide["A"], fwd["chunk_states"], z=wide["z"],
                          dfinal_state=wide["df"], lengths=lengths, workspace=ws, stream=stream, **bwd)

    return forward, backward, {**fwd, **bwd}


LEFT_OVER = [pytest.param(per, gated, dtype, id=f"{per}-{'gated' if gated else 'plain'}-{'bf16' if dtype is BF16 else 'fp32'}")
             for per in (2, 3, 4) for gated in (False, True) for dtype in (BF16, FP32)]


@pytest.mark.parametrize("per,gated,dtype", LEFT_OVER)
def test_glr_left_over_strips_against_fp64(per, gated, dtype):
    base, wide, lengths, C = left_over(per, gated, dtype)
    forward, backward, got = calls(wide, lengths, C)
    forward(), backward()
    bd.mamba2_check_device_status()
    f = {k: ref.f64(t) for k, t in base.items()}
    y, fin, hs = ref.glr(f["x"], f["r"], f["i"], f["A"], f["z"], f["h0"], lengths)
    want, size = ref.glr_grads(f["dy"], f["x"], f["r"], f["i"], f["A"], f["z"], f["h0"], lengths, f["df"])
    want = {**want, "y": y, "final_state": fin, "dinitial_state": want.pop("dinit"),
            "chunk_states": torch.cat([f["h0"][:, None], hs[:, 63:-1:64]], 1)}
    for name, t in got.items():
        w = want[name].cuda()
        err = (t.double() - w.repeat(*[1] * (w.dim() - 1), C // 32)).abs().max().item()
        most = 1e-5 * size.max().item() if name == "dA" else TOL[t.dtype] * w.abs().max().item()
        assert err <= most, f"{name}: {err:.3e}, at most {most:.3e}"


def launches(call):
    """Launches of a call: nodes of the graph that it is captured into."""
    call()
    torch.cuda.synchronize()
    cuda, graph, count = ctypes.CDLL("libcuda.so.1"), ctypes.c_void_p(), ctypes.c_size_t()
    stream = torch.cuda.Stream()
    at = ctypes.c_void_p(stream.cuda_stream)
    assert cuda.cuStreamBeginCapture_v2(at, 1) == 0  # (this thread's calls)
    try:
        call(stream)
    finally:
        assert cuda.cuStreamEndCapture(at, ctypes.byref(graph)) == 0
    assert cuda.cuGraphGetNodes(graph, None, ctypes.byref(count)) == 0
    assert cuda.cuGraphDestroy(graph) == 0
    return count.value


# Blocks of an SM by their shared memory (228 KB, 1 KB of it taken a block) and registers: forward, backward.
BLOCKS = {(BF16, False): (4, 4), (BF16, True): (4, 3), (FP32, False): (4, 3), (FP32, True): (3, 2)}


@pytest.mark.parametrize("per,gated,dtype", LEFT_OVER)
def test_glr_left_over_strips_are_split_where_places_are_filled_less_than_twice(per, gated, dtype):
    """One launch more where strips are more than the blocks that the GPU holds at once."""
    _, wide, lengths, C = left_over(per, gated, dtype)
    forward, backward, _ = calls(wide, lengths, C)
    strips = 4 * (C // 32)
    for call, blocks, least in zip((forward, backward), BLOCKS[dtype, gated], (1, 2)):
        split = blocks * sms() < strips < 2 * blocks * sms()
        assert launches(call) == least + split
