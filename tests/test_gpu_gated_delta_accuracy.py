"""Accuracy of the chunked gated delta rule's outputs, by norm and token by
token (a maximum over a whole tensor hides what a small token loses).

Tolerances, from the arithmetic in bf16 with q, k normalised:
- a result rounded once to bf16 is off by at most 2^-9 of itself; by norm it is
  off by what the fp64 result is when it is rounded (`rounding`);
- before that rounding y is made of two bf16 parts (2^-17) of the state, of the
  corrections and of the scores: 2^-17 of terms a few times y's size on ordinary
  inputs, beside roundings of 1.7e-3 by norm. A hundredth more than the rounding
  alone leaves room for 2.3e-4, eight times as much;
- where a token overwrites values 100 times its own size, the corrections are up
  to 150 times y (keys drawn at random are not quite orthogonal) and P and W are
  each good to 2^-17 of them: 2^-9 + 150 x 2^-16;
- states take 24 bits in what is added to them and two parts in their own
  correction, whose error the correction carries to the state once: below 2^-18
  by norm where states decay.
"""
import numpy as np
import pytest
import torch

import gated_delta_ref as ref
from mamba_chunked_ssd_gb300 import binding as bd
from test_gpu_gated_delta import BF16, gdr_inputs, np64

pytestmark = pytest.mark.gpu

# one head to a block, two, and sizes that are filled up: b, nh, G, H, S
SHAPES = [(1, 4, 2, 128, 128), (1, 4, 2, 64, 128), (10, 16, 4, 64, 128), (1, 4, 1, 128, 64), (10, 16, 8, 64, 64),
          (1, 2, 1, 96, 72), (10, 16, 4, 40, 120)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mamba_chunked_ssd_gb300 import build_lib
    build_lib.build()
    bd.load_library()


def off_by_norm(got, want):
    return np.linalg.norm(got - want) / np.linalg.norm(want)


def rounding(want):
    return off_by_norm(np64(torch.from_numpy(want).to(BF16)), want)


@pytest.mark.parametrize("b,nh,G,H,S", SHAPES)
@pytest.mark.parametrize("decay", [1.0, 0.1])
def test_y_is_the_definitions_rounded_once(b, nh, G, H, S, decay):
    d, h0 = gdr_inputs(b, 200, nh, G, H, S, BF16, seed=H + S, unit=False, decay=decay)
    y, fin = bd.mamba2_gdr_fwd(**d, initial_state=h0, qk_l2norm=True)
    bd.mamba2_check_device_status()
    y_ref, fin_ref = ref.gdr(**d, scale=S ** -0.5, l2norm=True, init=h0)
    assert off_by_norm(np64(y), y_ref) <= 1.01 * rounding(y_ref)
    assert off_by_norm(np64(fin), fin_ref) <= 2.0 ** -18


@pytest.mark.parametrize("b,nh,G,H,S", SHAPES)
def test_y_of_a_token_that_overwrites_a_far_larger_value(b, nh, G, H, S):
    """The same 32 keys in two chunks, asked for as they are written (beta 1, no
    decay), with values that fall by 100 from one to the other."""
    d, _ = gdr_inputs(b, 32, nh, G, H, S, BF16, seed=H * S)
    r = torch.Generator().manual_seed(S)
    k = torch.randn(b, 32, G, S, generator=r).to(BF16).cuda().repeat(1, 2, 1, 1)
    fall = torch.tensor([1.0, 1e-2]).repeat_interleave(32)[None, :, None, None]
    v = (torch.randn(b, 64, nh, H, generator=r) * fall).to(BF16).cuda()
    zeros = torch.zeros(b, 64, nh, device="cuda")
    y, _ = bd.mamba2_gdr_fwd(k, k, v, zeros, zeros + 1, scale=1.0, qk_l2norm=True)
    bd.mamba2_check_device_status()
    y_ref, _ = ref.gdr(k, k, v, zeros, zeros + 1, 1.0, l2norm=True)
    token = np.linalg.norm(np64(y) - y_ref, axis=-1) / np.linalg.norm(y_ref, axis=-1)
    assert token.max() <= 2.0 ** -9 + 150 * 2.0 ** -16


NAN = float("nan")


@pytest.mark.parametrize("b,nh,G,H,S", SHAPES)
@pytest.mark.parametrize("where", [31, 70, 85])
@pytest.mark.parametrize("value,bad", [("k", NAN), ("v", NAN), ("g", NAN), ("beta", NAN), ("v", float("inf"))])
def test_what_is_not_finite_reaches_back_no_further_than_its_16_tokens(b, nh, G, H, S, where, value, bad):
    """The last head's (or group's) token `where`: the tokens before its block of 16
    and the heads of other groups keep their results bit for bit."""
    d, h0 = gdr_inputs(b, 100, nh, G, H, S, BF16, seed=where)
    clean, fin_clean = bd.mamba2_gdr_fwd(**d, initial_state=h0)
    d[value][-1, where, -1] = bad
    y, fin = bd.mamba2_gdr_fwd(**d, initial_state=h0)
    bd.mamba2_check_device_status()
    start = where // 16 * 16
    assert torch.equal(y[-1, :start], clean[-1, :start]) and torch.equal(y[:-1], clean[:-1])
    others = nh - (nh // G if value == "k" else 1)
    assert torch.equal(y[-1, :, :others], clean[-1, :, :others])
    assert torch.equal(fin[-1, :others], fin_clean[-1, :others])
    columns = y[-1, where:, others:]
    assert not torch.isfinite(columns).any()


@pytest.mark.parametrize("b,nh,G,H,S", SHAPES)
@pytest.mark.parametrize("l2norm", [False, True])
@pytest.mark.parametrize("bad", [NAN, float("inf")])
def test_a_query_that_is_not_finite_stays_in_its_token(b, nh, G, H, S, l2norm, bad):
    d, h0 = gdr_inputs(b, 100, nh, G, H, S, BF16, seed=3)
    clean, fin_clean = bd.mamba2_gdr_fwd(**d, initial_state=h0, qk_l2norm=l2norm)
    where, others = 45, nh - nh // G
    d["q"][-1, where, -1, S // 2] = bad
    y, fin = bd.mamba2_gdr_fwd(**d, initial_state=h0, qk_l2norm=l2norm)
    bd.mamba2_check_device_status()
    assert torch.equal(fin, fin_clean)
    assert not torch.isfinite(y[-1, where, others:]).any()
    y[-1, where, others:] = clean[-1, where, others:]
    assert torch.equal(y, clean)
