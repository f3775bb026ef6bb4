"""GPU checks of the gated linear recurrence at the ends of its arguments' ranges.

Tolerances are those of the parity tests beside this file, on max|err| / max|ref|: a value that
leaves as bf16 is rounded once, by 2^-8 of it at most; the fp32 work before it is within 1e-5.
"""
import pytest
import torch

import gated_linear_ref as ref
from mamba_chunked_ssd_gb300 import binding as bd
from test_gpu_gated_linear import BOTH, INF, TOL, gen, glr_inputs

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
