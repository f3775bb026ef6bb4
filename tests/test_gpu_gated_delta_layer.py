"""The gated-delta-rule layer, its operators together as a server runs them:
against the same layer in fp64 on the CPU, prefill then decoding against prefill
alone, and a ragged batch against its rows one by one.

Tolerance on max|err| / max|ref|: the layer rounds to bf16 after the projection,
the convolution, the rule and the norm, and its last product's operands are those
values (2^-9 each, and the rule's three): 7 x 2^-9 < 2e-2.
"""
import numpy as np
import pytest
import torch

import gated_delta_ref as ref
from gpu_helpers import rel_err
from mamba_chunked_ssd_gb300 import binding as bd
from mamba_chunked_ssd_gb300.gated_delta_layer import GatedDeltaLayer, main

pytestmark = pytest.mark.gpu
TOL = 2e-2


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mamba_chunked_ssd_gb300 import build_lib
    build_lib.build()
    bd.load_library()


@pytest.fixture(scope="module", params=[(4, 2, 64, 64), (2, 2, 128, 128)], ids=["h64", "h128"])
def layer(request):
    nh, G, H, S = request.param
    return GatedDeltaLayer(256, nh, G, H, S)


def tokens(b, L, seed=0):
    r = torch.Generator().manual_seed(seed)
    return torch.randn(b, L, 256, generator=r).bfloat16().cuda()


def np64(t):
    return t.detach().cpu().double().numpy()


def in_64_bits(m, u):
    """The layer from its definition (weights and inputs as stored)."""
    w_in, w_out, x = np64(m.w_in), np64(m.w_out), np64(u)
    qkv, z, a, b = np.split(x @ w_in, np.cumsum(m.parts)[:-1], -1)
    t = torch.from_numpy
    c, _ = ref.conv(t(qkv), m.w_conv, m.b_conv)
    q, k, v = np.split(c, [m.qk, 2 * m.qk], -1)
    B, L, _ = x.shape
    g = -np64(m.A) * np.log1p(np.exp(a + np64(m.dt_bias)))
    y, st = ref.gdr(t(q.reshape(B, L, m.ngroups, m.dstate)), t(k.reshape(B, L, m.ngroups, m.dstate)),
                    t(v.reshape(B, L, m.nheads, m.headdim)), t(g), t(1 / (1 + np.exp(-b))), m.dstate ** -0.5, l2norm=True)
    y = ref.norm(t(y.reshape(B, L, -1)), m.nheads, m.w_norm, None, t(z), 1e-5, False, "after")
    return y @ w_out, st


def test_prefill_matches_the_definition(layer):
    u = tokens(2, 90)
    out, carried = layer.prefill(u)
    bd.mamba2_check_device_status()
    want, state = in_64_bits(layer, u)
    assert rel_err(np64(out), want) <= TOL
    assert rel_err(np64(carried.state), state) <= TOL


def test_decoding_continues_a_prefill(layer):
    u = tokens(2, 75, seed=1)
    whole, end = layer.prefill(u)
    _, carried = layer.prefill(u[:, :70].contiguous())
    outs = [layer.step(u[:, t].contiguous(), carried) for t in range(70, 75)]
    assert rel_err(np64(torch.stack(outs, 1)), np64(whole[:, 70:])) <= TOL
    assert rel_err(np64(carried.state), np64(end.state)) <= TOL
    # from nothing: the first token as a step and as a prefill
    first = layer.step(u[:, 0].contiguous(), layer.new_state(2))
    assert rel_err(np64(first), np64(whole[:, 0])) <= TOL


def test_prefill_in_two_calls(layer):
    u = tokens(1, 100, seed=2)
    whole, end = layer.prefill(u)
    a, carried = layer.prefill(u[:, :33].contiguous())
    b, carried = layer.prefill(u[:, 33:].contiguous(), carried)
    assert rel_err(np64(torch.cat([a, b], 1)), np64(whole)) <= TOL
    assert rel_err(np64(carried.state), np64(end.state)) <= TOL
    assert rel_err(np64(carried.conv), np64(end.conv)) <= TOL


def test_ragged_prefill_is_its_rows(layer):
    u = tokens(4, 80, seed=3)
    n = [80, 0, 1, 47]
    out, carried = layer.prefill(u, lengths=torch.tensor(n, dtype=torch.int32, device="cuda"))
    for i, m in enumerate(n):
        if m == 0:
            assert not carried.state[i].any() and not carried.conv[i].any()
            continue
        row, st = layer.prefill(u[i:i + 1, :m].contiguous())
        assert rel_err(np64(out[i, :m]), np64(row[0])) <= TOL
        assert rel_err(np64(carried.state[i]), np64(st.state[0])) <= TOL
        assert torch.isfinite(out[i].float()).all()


def test_the_example_runs(capsys):
    main([])
    assert "4 tokens decoded" in capsys.readouterr().out
