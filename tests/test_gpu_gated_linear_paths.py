"""GPU parity of the gated linear recurrence, the block norm and the gradients on paths that
sizes choose: sequences that four or eight blocks of a cluster share (whole and ragged), strips
that are left over when every SM has as many, and tensors of more than 2^31 elements.

Tolerances are those of the parity tests beside this file, on max|err| / max|ref|: a value that
leaves as bf16 is rounded once, by 2^-8 of it at most; the fp32 work before it is within 1e-5; a
sum over tokens or rows within 1e-5 of the sum of its terms' absolute values.
"""
import ctypes

import pytest
import torch

import gated_linear_ref as ref
from mamba_chunked_ssd_gb300 import binding as bd
from test_gpu_gated_linear import BF16, BOTH, FP32, INF, NAN, TOL, check_glr, gen, glr_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mamba_chunked_ssd_gb300 import build_lib
    build_lib.build()
    bd.load_library()


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# ------------------------------------------------------- clusters of blocks
@BOTH
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("b,L,C", [(1, 1500, 2080), (2, 400, 72), (1, 448, 33), (3, 500, 640)])
def test_glr_clusters_of_four_over_several_steps(b, L, C, gated, dtype):
    """On 152 SMs four blocks share each of these sequences, for two to six steps, the last of
    which has tiles for some of them only (24, 7, 7 and 8 tiles)."""
    d, h0 = glr_inputs(b, L, C, dtype, seed=L + C, gated=gated)
    check_glr(d, h0)


@BOTH
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("L,C", [(700, 37), (400, 128)])
def test_glr_ragged_rows_in_clusters(L, C, gated, dtype):
    """Eight blocks (700 tokens of 2 strips a row) and four (400 tokens of 4): rows without tokens,
    of fewer tiles than blocks, of whole steps and a token more; NaN and infinities past each row's end."""
    lengths = torch.tensor([0, 1, 64, 65, 128, 191, 192, 256, 257, L - 1, L, L + 9, -2], dtype=torch.int32, device="cuda")
    d, h0 = glr_inputs(len(lengths), L, C, dtype, seed=L, gated=gated)
    clean = {k: None if t is None else t.clone() for k, t in d.items()}
    for k, n in enumerate(lengths.clamp(0, L).tolist()):
        for j, name in enumerate(("x", "r", "i", "z")):
            if d[name] is not None:
                d[name][k, n:] = (NAN, INF, -INF, NAN)[j]
    y, fin, grads = check_glr(d, h0, lengths=lengths, clean=clean)
    assert torch.equal(fin[0], h0[0]) and torch.equal(fin[-1], h0[-1])
    for k, n in enumerate(lengths.clamp(0, L).tolist()):
        for t in (y, *(grads[g] for g in grads if g not in ("dA", "dinitial_state"))):
            assert bool((t[k, n:] == 0).all())


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


@pytest.mark.parametrize("gated,dtype", [(False, BF16), (True, FP32)])
def test_glr_left_over_strips_captured_and_replayed(gated, dtype):
    """Both launches of both passes in one graph, replayed on new inputs: what eager calls give, bit for bit."""
    _, wide, lengths, C = left_over(4, gated, dtype)
    forward, backward, got = calls(wide, lengths, C)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    forward(), backward()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        forward(), backward()
    for seed in (1, 2):
        for k in ("x", "r", "i"):
            wide[k].copy_(gen(seed)(*wide[k].shape[:2], 32).to(dtype).repeat(1, 1, C // 32))
        graph.replay()
        torch.cuda.synchronize()
        replayed = {k: t.clone() for k, t in got.items()}
        for t in got.values():
            t.fill_(NAN)
        forward(), backward()
        torch.cuda.synchronize()
        for k, t in got.items():
            assert torch.equal(t, replayed[k]), k


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


# ------------------------------------------------- beyond 32-bit offsets
def big(*shape, last, at):
    """Zeros of bf16 but for the last row's last channels."""
    t = torch.zeros(*shape, dtype=BF16, device="cuda")
    t[at] = last
    return t


def near(got, want, tol, name):
    err, top = (got.double() - want.double()).abs().max().item(), want.double().abs().max().item()
    assert top > 0 and err <= tol * top, f"{name}: {err:.3e} of {top:.3e}"


def need_60_gb():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")


def test_glr_bwd_rows_past_32_bit_offsets():
    need_60_gb()
    b, L, C = 9, 4200, 65536
    n = gen(2)
    last = {k: n(1, L, 64).to(BF16).cuda() for k in ("x", "r", "i", "dy")}
    at = (slice(-1, None), slice(None), slice(-64, None))
    wide = {k: big(b, L, C, last=t, at=at) for k, t in last.items()}
    A = -torch.ones(C, device="cuda")
    _, _, cs = bd.mamba2_glr_fwd(wide["x"], wide["r"], wide["i"], A, want_chunk_states=True, want_final_state=False)
    got = bd.mamba2_glr_bwd(wide["dy"], wide["x"], wide["r"], wide["i"], A, cs)
    _, _, cs1 = bd.mamba2_glr_fwd(last["x"], last["r"], last["i"], A[:64], want_chunk_states=True)
    want = bd.mamba2_glr_bwd(last["dy"], last["x"], last["r"], last["i"], A[:64], cs1)
    for g, w, name in zip(got[:3], want[:3], ("dx", "dr", "di")):
        near(g[at], w, TOL[BF16], name)
        assert bool((g[0] == 0).all()) and bool((g[-1, :, :-64] == 0).all())
    near(got[4][-64:], want[4], 1e-5, "dA")
    near(got[5][-1:, -64:], want[5], 1e-5, "dinit")


def test_conv_bwd_rows_past_32_bit_offsets():
    need_60_gb()
    b, L, C, W = 9, 4200, 65536, 4
    n = gen(3)
    last = {k: n(1, L, 64).to(BF16).cuda() for k in ("x", "dy")}
    at = (slice(-1, None), slice(None), slice(-64, None))
    wide = {k: big(b, L, C, last=t, at=at) for k, t in last.items()}
    weight = n(C, W).cuda()
    dx, dw, _, _ = bd.mamba2_causal_conv_bwd(wide["dy"], wide["x"], weight)
    dx1, dw1, _, _ = bd.mamba2_causal_conv_bwd(last["dy"], last["x"], weight[-64:].contiguous())
    near(dx[at], dx1, TOL[BF16], "dx")
    near(dw[-64:], dw1, 1e-4, "dweight")  # (runs of other lengths: sums of 4200 terms in another order, 1e-5 of their sizes')
    assert bool((dx[0] == 0).all()) and bool((dx[-1, :, :-64] == 0).all()) and bool((dw[:-64] == 0).all())


@pytest.mark.parametrize("rows,C", [(600000, 4096), (75000, 32768)])
def test_block_norm_rows_past_32_bit_offsets(rows, C):
    """One block a row, and the blocks of a cluster; the last three rows are not zero."""
    need_60_gb()
    n = gen(4)
    last = {k: n(3, C).to(BF16).cuda() for k in ("x", "res", "dr", "dy")}
    at = (slice(-3, None),)
    wide = {k: big(rows, C, last=t, at=at) for k, t in last.items()}
    w = {k: 1 + 0.1 * n(C).cuda() for k in ("post_weight", "scale", "pre_weight")}
    out, y = bd.mamba2_block_norm_fwd(wide["x"], wide["res"], **w)
    out1, y1 = bd.mamba2_block_norm_fwd(last["x"], last["res"], **w)
    assert torch.equal(out[at], out1) and torch.equal(y[at], y1) and bool((y[:-3] == 0).all())
    got = bd.mamba2_block_norm_bwd(wide["dr"], wide["dy"], wide["x"], out, **w)
    want = bd.mamba2_block_norm_bwd(last["dr"], last["dy"], last["x"], out1, **w)
    for g, v, name in zip(got, want, ("dx", "dz", "dresidual", "dpost_weight", "dscale", "dpre_weight")):
        if name in ("dx", "dresidual"):
            assert torch.equal(g[at], v) and bool((g[:-3] == 0).all()), name
        elif name != "dz":
            near(g, v, 1e-5, name)
