"""The recurrent block: its operators together, as a program uses them, against the
same block in fp64 on the CPU, differentiated there.

Tolerances: the fp32 block's matrix products run in fp32 on 40 to 128 terms (2^-24 times
their number at most, twice over: 3e-5 of the largest value with the operators' 1e-5); the bf16
block rounds n, proj, u, the gates, y, out and next on the way, each by 2^-8 of it at most:
seven roundings, and as many again on the way back, of which one passes on about as much as it
gets: 14 x 2^-8 = 5.5e-2 of the largest value.
"""
import pytest
import torch

import gated_linear_ref as ref
from mamba_chunked_ssd_gb300 import binding as bd
from mamba_chunked_ssd_gb300.recurrent_block import BlockState, RecurrentBlock, main

pytestmark = pytest.mark.gpu

FP32, BF16 = torch.float32, torch.bfloat16
TOL = {FP32: 3e-5 + 1e-5, BF16: 14 * 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mamba_chunked_ssd_gb300 import build_lib
    build_lib.build()
    bd.load_library()
    tf32 = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    yield
    torch.backends.cuda.matmul.allow_tf32 = tf32


def plain(block, n, res, state, lengths):
    """The block in fp64 with leaves for all inputs and weights."""
    leaf = lambda t: ref.f64(t).requires_grad_()  # noqa: E731
    w = {k: leaf(t) for k, t in block.w.items()}
    n, res, conv, h = leaf(n), leaf(res), leaf(state.conv), leaf(state.state)
    x, z = (n @ w["in"]).split(block.channels, -1)
    u, conv_out = ref.conv(x, w["conv"], w["conv_bias"], True, conv, lengths)
    r, i = (u @ w["gates"]).split(block.channels, -1)
    y, h_out, _ = ref.glr(u, r, i, w["A"], z, h, lengths)
    out, nxt = ref.block_norm(y @ w["out"], res, None, w["post"], w["scale"], w["pre"])
    return nxt, out, conv_out, h_out, {**w, "n": n, "res": res, "conv_state": conv, "state": h}


def close(got, want, tol, name):
    err, top = (got.detach().cpu().double() - want).abs().max().item(), want.abs().max().item()
    assert err <= tol * top, f"{name}: {err:.3e} of {top:.3e}"


@pytest.mark.parametrize("dtype", [FP32, BF16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("ragged", [False, True])
def test_forward_and_backward(ragged, dtype):
    b, L, d, C = 3, 70, 40, 64
    block = RecurrentBlock(d, C, dtype=dtype)
    g = torch.Generator().manual_seed(3)
    t = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    n, res = t(b, L, d).to(dtype).cuda(), t(b, L, d).cuda()
    state = BlockState(t(b, 3, C).to(dtype).cuda(), t(b, C).cuda())
    lengths = torch.tensor([70, 33, 0], dtype=torch.int32, device="cuda") if ragged else None
    if dtype is FP32:
        res = res.to(FP32)
    nxt, out, after, kept = block.forward(n, res, state, lengths=lengths, keep=True)
    want = plain(block, n, res, state, lengths)
    for got, w, name in zip((nxt, out, after.conv, after.state), want, ("next", "residual", "conv", "state")):
        close(got, w, TOL[dtype], name)
    dn, dr = t(b, L, d).to(dtype).cuda(), t(b, L, d).cuda()
    leaves = want[4]
    auto = dict(zip(leaves, torch.autograd.grad((want[0] * ref.f64(dn)).sum() + (want[1] * ref.f64(dr)).sum(),
                                                list(leaves.values()))))
    gn, gres, gstate, gw = block.backward(kept, dn, dr)
    bd.mamba2_check_device_status()
    for got, name in ((gn, "n"), (gres, "res"), (gstate.conv, "conv_state"), (gstate.state, "state"),
                      *((v, k) for k, v in gw.items())):
        close(got, auto[name], TOL[dtype], "gradient of " + name)
    assert set(gw) == set(block.w)


@pytest.mark.parametrize("dtype", [FP32, BF16], ids=["fp32", "bf16"])
def test_decoding_continues_the_whole_sequence(dtype):
    b, L, d, C = 2, 50, 40, 72
    block = RecurrentBlock(d, C, dtype=dtype)
    g = torch.Generator().manual_seed(4)
    n, res = (torch.randn(b, L, d, generator=g).cuda() for _ in range(2))
    n = n.to(dtype)
    whole, whole_res, last, _ = block.forward(n, res)
    part = lambda t, a, c: t[:, a:c].contiguous()  # noqa: E731
    a_n, a_res, carried, _ = block.forward(part(n, 0, 41), part(res, 0, 41))
    ns, rs = [a_n], [a_res]
    for t in range(41, L):
        x, r = block.step(n[:, t].contiguous(), res[:, t].contiguous(), carried)
        ns.append(x[:, None]), rs.append(r[:, None])
    close(torch.cat(ns, 1), whole.cpu().double(), TOL[dtype], "next")
    close(torch.cat(rs, 1), whole_res.cpu().double(), TOL[dtype], "residual")
    close(carried.state, last.state.cpu().double(), TOL[dtype], "state")


def test_the_example_runs(capsys):
    main(["--tokens", "70", "--width", "64", "--channels", "96"])
    assert "tokens decoded" in capsys.readouterr().out
