"""GPU checks of the recurrent block's operators at the ends of its arguments' ranges.

Tolerances are those of the parity tests beside this file, on max|err| / max|ref|: a value that
leaves as bf16 is rounded once, by 2^-8 of it at most; the fp32 work before it is within 1e-5.
"""
import pytest
import torch

import gated_linear_ref as ref
from mamba_chunked_ssd_gb300 import binding as bd
from test_gpu_gated_linear import (BOTH, DTYPES, INF, TOL, check_norm, close, conv_inputs, f64s, gen, glr_inputs,
                                   norm_inputs)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mamba_chunked_ssd_gb300 import build_lib
    build_lib.build()
    bd.load_library()


@BOTH
@pytest.mark.parametrize("gated", [False, True])
def test_glr_gradients_of_decays_beyond_all_exponents(gated, dtype):
    """A at which a is 0 to fp32: the next state has nothing of the last one, and the gate r no part in it.
    Where a is held at e^-87 = 1.6e-38 a token has 87 e^-87 |dh| (|h| + |v|) of dr, with both factors of normal
    numbers below 15 each: below 1e-33; dA is their sum over 140 tokens, by A."""
    b, L, C = 2, 70, 32
    d, h0 = glr_inputs(b, L, C, dtype, seed=9, gated=gated)
    d["A"] = -torch.tensor([1e4, 1e20, 1e30, 1e36, 1e37, 1e38, 3e38, INF]).repeat(C // 8).cuda()
    d["r"] = d["r"].abs()
    y, fin, cs = bd.mamba2_glr_fwd(**d, initial_state=h0, want_chunk_states=True)
    f = {k: ref.f64(t) for k, t in d.items()}
    want = torch.sigmoid(f["i"]) * f["x"]
    if gated:
        want = want * ref.silu(f["z"])
    assert (y.cpu().double() - want).abs().max() <= TOL[dtype] * want.abs().max()
    dy = gen(3)(b, L, C).to(dtype).cuda()
    dx, dr, di, dz, dA, dh = bd.mamba2_glr_bwd(dy, **d, chunk_states=cs, dfinal_state=torch.ones(b, C, device="cuda"))
    bd.mamba2_check_device_status()
    assert dr.abs().max() <= 1e-33 and dA.abs().max() <= 1e-33 and dh.abs().max() <= 1e-33
    assert torch.isfinite(dx).all() and torch.isfinite(di).all()


@BOTH
def test_gates_of_the_lowest_value_are_shut(dtype):
    """z at its dtype's lowest value, as masks have it: SiLU(z) is 0, whatever it meets."""
    b, L, C = 2, 70, 64
    d, h0 = glr_inputs(b, L, C, dtype, seed=11, gated=True)
    h0 *= 8
    d["z"][:, 20:30] = d["z"][1, :, 5::7] = torch.finfo(dtype).min
    shut = d["z"] == torch.finfo(dtype).min
    y, fin, cs = bd.mamba2_glr_fwd(**d, initial_state=h0, want_chunk_states=True)
    f = {k: ref.f64(t) for k, t in d.items()}
    y_ref, fin_ref, _ = ref.glr(**f, init=ref.f64(h0))
    assert bool((y[shut] == 0).all()) and (y.cpu().double() - y_ref).abs().max() <= TOL[dtype] * y_ref.abs().max()
    assert (fin.cpu().double() - fin_ref).abs().max() <= 1e-5 * fin_ref.abs().max()
    dy = gen(3)(b, L, C).to(dtype).cuda()
    dx, dr, di, dz, dA, dh = bd.mamba2_glr_bwd(dy, **d, chunk_states=cs)
    want, size = ref.glr_grads(ref.f64(dy), **f, init=ref.f64(h0))
    for got, k in ((dx, "dx"), (dr, "dr"), (di, "di"), (dz, "dz")):
        assert (got.cpu().double() - want[k]).abs().max() <= TOL[dtype] * want[k].abs().max(), k
    assert bool((dz[shut] == 0).all()) and (dA.cpu().double() - want["dA"]).abs().max() <= 1e-5 * size.max()
    one = {k: t[:, 25].contiguous() if t.dim() == 3 else t for k, t in d.items()}
    y, _ = bd.mamba2_glr_step(**one, state_in=h0)
    assert bool((y == 0).all())


@BOTH
def test_block_norm_gates_of_the_lowest_value_are_shut(dtype):
    d, res, dr, dy = norm_inputs(9, 300, dtype, dtype)
    d["z"][3], d["z"][:, 11::5] = torch.finfo(dtype).min, torch.finfo(dtype).min
    out, y, got = check_norm(d, res, dr, dy)
    shut = d["z"] == torch.finfo(dtype).min
    assert torch.equal(out[shut], res[shut]) and bool((got[1][shut] == 0).all())


@DTYPES
@pytest.mark.parametrize("C", [300, 4608])
def test_block_norm_rows_whose_squares_pass_fp32(C, dtype, rdtype):
    """A sum of squares beyond fp32's largest number is a norm without end: the row's N is 0 and passes no gradient on,
    the residual's own goes through; other rows are as they were."""
    d, res, dr, dy = norm_inputs(6, C, dtype, rdtype, gated=False)
    res[2, 7], d["x"][4, 9] = torch.finfo(rdtype).min, torch.finfo(dtype).min
    dy *= 4
    out, y = bd.mamba2_block_norm_fwd(**d, residual=res)
    dx, _, dres, *weights = bd.mamba2_block_norm_bwd(dr, dy, residual_out=out, **d)
    assert bool((y[2] == 0).all()) and torch.equal(out[4], res[4]) and torch.equal(dres[2], dr[2])
    assert bool((dx[4] == 0).all())
    want, size = ref.block_norm_grads(ref.f64(dr), ref.f64(dy), **f64s(d), out=ref.f64(out))
    rest = [0, 1, 3, 5]
    close(dx[rest], want["dx"][rest], TOL[dtype], size["dx"][rest], name="dx")
    close(dres[rest], want["dresidual"][rest], TOL[rdtype], size["dresidual"][rest], name="dresidual")
    assert all(torch.isfinite(t).all() for t in (dx, dres, *weights))


@BOTH
def test_conv_bwd_activations_of_the_largest_values(dtype):
    """An input at its dtype's lowest value, times weights of both signs: SiLU' is 0 or 1 there, whatever it meets.  (The
    weights' own gradients are products with that input, beyond fp32.)"""
    d, init, dy, dfin = conv_inputs(2, 60, 40, 4, dtype, seed=12)
    d["weight"] = d["weight"] / d["weight"].abs().sum(1, keepdim=True) * 0.9
    d["x"][0, 20], d["x"][1, 33:36, ::3] = torch.finfo(dtype).min, torch.finfo(dtype).min
    dy *= 8
    dx, dw, _, dinit = bd.mamba2_causal_conv_bwd(dy, **d, initial_state=init, dfinal_state=dfin)
    f = f64s(d)
    want, _ = ref.conv_grads(ref.f64(dy), f["x"], f["weight"], f["bias"], init=ref.f64(init), dfinal=ref.f64(dfin))
    close(dx, want["dx"], TOL[dtype], name="dx"), close(dinit, want["dinit"], TOL[dtype], name="dinit")
    clean = [c for c in range(40) if c % 3]
    assert not torch.isnan(dw[clean]).any()
