"""GPU parity of the gated delta rule, the causal convolution and the group
norm against their plain fp64 forms.

Tolerances are on max|err| / max|ref| and follow from the arithmetic:
- y of the gated delta rule in bf16: two products whose left operands and the
  result are each rounded to bf16 once (2^-9 of a term): 3 x 2^-9 < 1e-2;
- states, and everything on the fp32 paths: products of two-part operands
  (2^-17 each, six of them on a chunk's way round the recurrence) or fp32 sums
  of at most 256 terms: 6 x 2^-17 < 1e-4;
- the convolution and the norm: one rounding to bf16 at the end (2^-8 of the
  largest value covers it with the fp32 work before it), or fp32 sums: 1e-5;
- a state that is only copied is exact.
"""
import numpy as np
import pytest
import torch

import gated_delta_ref as ref
from gpu_helpers import Guarded, rel_err
from mamba_chunked_ssd_gb300 import binding as bd

pytestmark = pytest.mark.gpu

TOL_Y = {torch.bfloat16: 1e-2, torch.float32: 1e-4}
TOL_STATE = 1e-4
TOL_ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: 1e-5}
BF16, FP32 = torch.bfloat16, torch.float32
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mamba_chunked_ssd_gb300 import build_lib
    build_lib.build()
    bd.load_library()


def np64(t):
    return t.detach().cpu().double().numpy()


def gdr_inputs(b, L, nh, G, H, S, dtype, seed=0, unit=True, decay=1.0):
    """Keys and queries with a common part, as an activation leaves them."""
    r = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=r)  # noqa: E731
    q, k = (torch.nn.functional.silu(n(b, L, G, S)) for _ in range(2))
    if unit:
        q, k = (x / x.square().sum(-1, keepdim=True).add(1e-6).sqrt() for x in (q, k))
    g = -decay * torch.nn.functional.softplus(n(b, L, nh) - 2)
    return dict(q=q.to(dtype).cuda(), k=k.to(dtype).cuda(), v=n(b, L, nh, H).to(dtype).cuda(), g=g.cuda(),
                beta=torch.sigmoid(n(b, L, nh)).cuda()), (0.3 * n(b, nh, S, H)).cuda()


def check_gdr(d, init, l2norm=False, lengths=None, scale=None, tol_state=TOL_STATE):
    b, L, nh, H = d["v"].shape
    S = d["q"].shape[-1]
    scale = S ** -0.5 if scale is None else scale
    y, fin = Guarded((b, L, nh, H), d["v"].dtype), Guarded((b, nh, S, H), FP32)
    bd.mamba2_gdr_fwd(**d, scale=scale, qk_l2norm=l2norm, initial_state=init, lengths=lengths, y=y.t,
                      final_state=fin.t)
    bd.mamba2_check_device_status()
    assert y.intact() and fin.intact()
    y_ref, fin_ref = ref.gdr(**d, scale=scale, l2norm=l2norm, init=init, lengths=lengths)
    assert rel_err(np64(y.t), y_ref) <= TOL_Y[d["v"].dtype]
    assert rel_err(np64(fin.t), fin_ref) <= tol_state
    return y.t, fin.t


# --------------------------------------------------------- whole sequences
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 63, 64, 65, 128, 129, 200])
def test_gdr_lengths_of_sequences(L, dtype):
    d, h0 = gdr_inputs(2, L, 4, 2, 64, 128, dtype, seed=L)
    check_gdr(d, h0)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("nh,G,H,S", [
    (4, 2, 64, 64), (4, 1, 128, 64), (2, 2, 128, 128), (3, 1, 64, 128), (6, 2, 64, 128), (2, 1, 64, 256),
    (3, 3, 128, 96), (2, 1, 40, 128), (2, 1, 256, 32), (1, 1, 1, 1), (3, 1, 5, 7), (2, 2, 17, 129),
])
def test_gdr_head_layouts(nh, G, H, S, dtype):
    d, h0 = gdr_inputs(2, 137, nh, G, H, S, dtype, seed=H * S)
    check_gdr(d, h0, l2norm=True)


@pytest.mark.parametrize("H", [64, 128, 40])
def test_gdr_without_states(H):
    d, _ = gdr_inputs(1, 150, 2, 1, H, 128, BF16)
    y, none = bd.mamba2_gdr_fwd(**d, want_final_state=False)
    assert none is None
    y_ref, _ = ref.gdr(**d, scale=128 ** -0.5)
    assert rel_err(np64(y), y_ref) <= TOL_Y[BF16]


@pytest.mark.parametrize("H", [64, 128, 40])
@pytest.mark.parametrize("l2norm", [False, True])
def test_gdr_ragged_batch(H, l2norm):
    """Rows of every kind of length (beyond L and below 0 too), with NaN and
    infinities past each row's end: y is 0 there, the state stays."""
    L = 150
    lengths = torch.tensor([0, 1, 63, 64, 65, 100, 128, 149, 150, 999, -7], dtype=torch.int32, device="cuda")
    d, h0 = gdr_inputs(len(lengths), L, 4, 2, H, 128, BF16, unit=not l2norm)
    clean = {n: t.clone() for n, t in d.items()}
    for i, n in enumerate(lengths.clamp(0, L).tolist()):
        for j, t in enumerate(d.values()):
            t[i, n:] = (NAN, float("inf"), -float("inf"), NAN, NAN)[j]
    scale = 128 ** -0.5
    y, fin = bd.mamba2_gdr_fwd(**d, scale=scale, qk_l2norm=l2norm, initial_state=h0, lengths=lengths)
    bd.mamba2_check_device_status()
    y_ref, fin_ref = ref.gdr(**clean, scale=scale, l2norm=l2norm, init=h0, lengths=lengths)
    assert rel_err(np64(y), y_ref) <= TOL_Y[BF16]
    assert rel_err(np64(fin), fin_ref) <= TOL_STATE
    assert torch.equal(fin[0], h0[0]) and torch.equal(fin[-1], h0[-1])
    for i, n in enumerate(lengths.clamp(0, L).tolist()):
        assert bool((y[i, n:] == 0).all())


@pytest.mark.parametrize("b,nh,G,L", [(2, 4, 2, 75), (11, 16, 4, 67), (200, 2, 2, 9), (10, 16, 16, 33)])
@pytest.mark.parametrize("H,S", [(64, 128), (64, 64), (40, 128), (8, 72), (56, 96), (64, 8), (72, 128), (120, 40), (128, 96)])
def test_gdr_sizes_and_numbers_of_heads(b, nh, G, L, H, S):
    """States and heads that are filled up, few heads and enough for two to share
    a block (where a group has two), ragged, with NaN past each row's end."""
    d, h0 = gdr_inputs(b, L, nh, G, H, S, BF16, seed=H + S, unit=False)
    lengths = (torch.arange(b, device="cuda", dtype=torch.int32) * 37 + L) % (L + 1)
    clean = {n: t.clone() for n, t in d.items()}
    for i, n in enumerate(lengths.tolist()):
        for t in d.values():
            t[i, n:] = NAN
    scale = S ** -0.5
    y, fin = Guarded((b, L, nh, H), BF16), Guarded((b, nh, S, H), FP32)
    bd.mamba2_gdr_fwd(**d, scale=scale, qk_l2norm=True, initial_state=h0, lengths=lengths, y=y.t, final_state=fin.t)
    bd.mamba2_check_device_status()
    assert y.intact() and fin.intact()
    y_ref, fin_ref = ref.gdr(**clean, scale=scale, l2norm=True, init=h0, lengths=lengths)
    assert rel_err(np64(y.t), y_ref) <= TOL_Y[BF16]
    assert rel_err(np64(fin.t), fin_ref) <= TOL_STATE


@pytest.mark.parametrize("H", [64, 40])
@pytest.mark.parametrize("case", ["equal_keys", "equal_keys_beta_2", "no_decay", "mixed_decay", "forget_all"])
def test_gdr_hard_inputs_of_many_heads(H, case):
    """The hard inputs below with two heads to a block."""
    d, h0 = gdr_inputs(10, 190, 16, 4, H, 128, BF16, seed=6)
    if case.startswith("equal_keys"):
        d["k"][:] = d["k"][:, :1]
        d["g"] *= 0.01
        d["beta"][:] = 2.0 if case.endswith("2") else 1.0
    if case == "no_decay":
        d["g"][:] = 0
    if case == "mixed_decay":
        d["g"][:, ::3] = 0
        d["g"][:, 1::3] = -90.0
    if case == "forget_all":
        d["g"][:, 100] = -float("inf")
    check_gdr(d, h0, l2norm=case == "equal_keys_beta_2")


def test_gdr_ragged_batch_of_more_rows_than_threads():
    """More rows than a block has threads to order them with."""
    b, L = 1030, 40
    d, h0 = gdr_inputs(b, L, 1, 1, 64, 64, BF16)
    lengths = (torch.arange(b, device="cuda", dtype=torch.int32) * 7) % (L + 1)
    y, fin = bd.mamba2_gdr_fwd(**d, initial_state=h0, lengths=lengths)
    y_ref, fin_ref = ref.gdr(**d, scale=0.125, init=h0, lengths=lengths)
    assert rel_err(np64(y), y_ref) <= TOL_Y[BF16] and rel_err(np64(fin), fin_ref) <= TOL_STATE


@pytest.mark.parametrize("value,where", [("g", 70), ("beta", 70), ("k", 70), ("v", 70)])
def test_gdr_nan_input_shows_from_its_token_on(value, where):
    """A NaN in one head's input leaves the other heads and the tokens before it."""
    d, h0 = gdr_inputs(1, 140, 2, 2, 128, 128, BF16)
    clean, _ = bd.mamba2_gdr_fwd(**d, initial_state=h0)
    d[value][0, where, 1] = NAN
    y, fin = bd.mamba2_gdr_fwd(**d, initial_state=h0)
    assert torch.equal(y[:, :, 0], clean[:, :, 0]) and torch.isfinite(fin[0, 0]).all()
    start = where // 32 * 32  # a chunk's tokens share products with zeros in them
    assert torch.equal(y[:, :start, 1], clean[:, :start, 1])
    assert torch.isnan(y[0, where:, 1]).all() and torch.isnan(fin[0, 1]).all()


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("b,nh,H", [(2, 4, 40), (1, 32, 40), (3, 32, 40), (2, 64, 33)])
@pytest.mark.parametrize("S", [36, 65, 200])
def test_gdr_token_by_token_widths(b, nh, H, S, dtype):
    """Few and many heads (blocks of fewer or more columns), ragged, normalised,
    heads that share q and k, lengths around the tiles' and passes' ends."""
    L = 53
    d, h0 = gdr_inputs(b, L, nh, nh // 4, H, S, dtype, seed=S, unit=False)
    lengths = torch.tensor([L, 0, 34][:b], dtype=torch.int32, device="cuda")
    check_gdr(d, h0, l2norm=True, lengths=lengths)


@pytest.mark.parametrize("nh", [2, 32, 96])
@pytest.mark.parametrize("value", ["g", "beta", "k", "v", "q"])
def test_gdr_token_by_token_nan_input_shows_from_its_token_on(value, nh):
    """Tokens that share a pass over the state: nothing of a later one's NaN
    reaches the ones before it."""
    for where in (20, 21, 22, 23):
        d, h0 = gdr_inputs(1, 40, nh, nh, 40, 32, FP32)
        clean, fin_clean = bd.mamba2_gdr_fwd(**d, initial_state=h0)
        d[value][0, where, 1] = NAN
        y, fin = bd.mamba2_gdr_fwd(**d, initial_state=h0)
        others = [i for i in range(nh) if i != 1]
        assert torch.equal(y[:, :, others], clean[:, :, others]) and torch.equal(fin[0, others], fin_clean[0, others])
        assert torch.equal(y[:, :where, 1], clean[:, :where, 1])
        if value == "q":
            assert torch.isnan(y[0, where, 1]).all() and torch.equal(y[0, where + 1:, 1], clean[0, where + 1:, 1])
            assert torch.equal(fin, fin_clean)
        else:
            assert torch.isnan(y[0, where:, 1]).all() and torch.isnan(fin[0, 1]).all()


def test_gdr_offsets_beyond_32_bits():
    """v and y of more than 2^31 elements: the sequence's end, from the state that
    enters it, against a call on the end alone."""
    L, cut, nh, H = 540_000, 539_700, 64, 64
    r = torch.Generator(device="cuda").manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=r, device="cuda", dtype=BF16)  # noqa: E731
    q, k, v = n(1, L, 1, 64), n(1, L, 1, 64), n(1, L, nh, H)
    g = -torch.rand(1, L, nh, generator=r, device="cuda")
    beta = torch.rand(1, L, nh, generator=r, device="cuda")
    assert v.numel() > 2 ** 31
    y, fin = bd.mamba2_gdr_fwd(q, k, v, g, beta, qk_l2norm=True)
    part = lambda t, s: t[:, s].contiguous()  # noqa: E731
    # decays of e^-0.5 a token on average: nothing is left of what came 1000 tokens before
    a, b = slice(cut - 3000, cut), slice(cut, L)
    _, mid = bd.mamba2_gdr_fwd(*(part(t, a) for t in (q, k, v, g, beta)), qk_l2norm=True)
    y2, fin2 = bd.mamba2_gdr_fwd(*(part(t, b) for t in (q, k, v, g, beta)), qk_l2norm=True, initial_state=mid)
    assert rel_err(np64(y[:, cut:]), np64(y2)) <= TOL_Y[BF16]
    assert rel_err(np64(fin), np64(fin2)) <= TOL_STATE


@pytest.mark.parametrize("H", [64, 128, 40])
def test_gdr_empty_sequences(H):
    d, h0 = gdr_inputs(2, 0, 2, 1, H, 128, BF16)
    y, fin = bd.mamba2_gdr_fwd(**d, initial_state=h0)
    assert y.shape == (2, 0, 2, H) and torch.equal(fin, h0)
    _, fin = bd.mamba2_gdr_fwd(**d)
    assert not fin.any()
    d, _ = gdr_inputs(0, 5, 2, 1, H, 128, BF16)
    y, fin = bd.mamba2_gdr_fwd(**d)
    assert y.shape == (0, 5, 2, H) and fin.shape == (0, 2, 128, H)


@pytest.mark.parametrize("dtype,H", [(BF16, 64), (BF16, 128), (BF16, 48), (FP32, 64)])
@pytest.mark.parametrize("case", ["equal_keys", "equal_keys_beta_2", "no_decay", "strong_decay", "mixed_decay",
                                  "forget_all", "beta_0", "zero_keys"])
def test_gdr_hard_inputs(dtype, H, case):
    """Keys that all agree (the chunk's triangular system at its worst), decays
    from none to total, tokens that write nothing."""
    d, h0 = gdr_inputs(1, 190, 4, 2, H, 128, dtype, seed=5)
    if case.startswith("equal_keys"):
        d["k"][:] = d["k"][:, :1]
        d["g"] *= 0.01
        d["beta"][:] = 2.0 if case.endswith("2") else 1.0
    if case == "no_decay":
        d["g"][:] = 0
    if case == "strong_decay":
        d["g"][:] = -30.0
    if case == "mixed_decay":
        d["g"][:, ::3] = 0
        d["g"][:, 1::3] = -90.0
    if case == "forget_all":
        d["g"][:, 100] = -float("inf")
    if case == "beta_0":
        d["beta"][:] = 0
    if case == "zero_keys":
        d["k"][:] = 0
        d["q"][:, 20] = 0
    # keys of length 1 + 2^-8 (bf16) under beta = 2 let errors grow by (1 + 2^-7) a token
    check_gdr(d, h0, l2norm=case in ("zero_keys", "equal_keys_beta_2"))


def test_gdr_nothing_written_keeps_the_state_exactly():
    d, h0 = gdr_inputs(2, 130, 2, 1, 128, 128, BF16)
    d["g"][:] = 0
    d["beta"][:] = 0
    for H in (128, 64, 40):
        e = dict(d, v=d["v"][..., :H].contiguous())
        s = h0[..., :H].contiguous()
        _, fin = bd.mamba2_gdr_fwd(**e, initial_state=s)
        assert torch.equal(fin, s)


@pytest.mark.parametrize("H", [64, 128])
def test_gdr_split_sequence(H):
    """Two calls joined by the state against one."""
    d, h0 = gdr_inputs(2, 300, 4, 2, H, 128, BF16)
    y, fin = check_gdr(d, h0)
    cut = 171
    a, b = ({n: t[:, s].contiguous() for n, t in d.items()} for s in (slice(0, cut), slice(cut, None)))
    y1, mid = bd.mamba2_gdr_fwd(**a, initial_state=h0)
    y2, end = bd.mamba2_gdr_fwd(**b, initial_state=mid)
    assert rel_err(np64(torch.cat([y1, y2], 1)), np64(y)) <= TOL_Y[BF16]
    assert rel_err(np64(end), np64(fin)) <= TOL_STATE


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_gdr_slices_of_one_tensor(dtype, pad):
    """q, k, v as channel slices of one tensor, at 16-byte boundaries and not."""
    b, L, nh, G, H, S = 2, 100, 4, 2, 64, 128
    d, h0 = gdr_inputs(b, L, nh, G, H, S, dtype)
    parts = [d["q"].flatten(2), d["k"].flatten(2), d["v"].flatten(2)]
    x = torch.cat([parts[0][..., :pad], *parts], -1).contiguous()
    w = [p.shape[-1] for p in parts]
    q, k, v = torch.split(x[..., pad:], w, -1)
    e = dict(d, q=q.unflatten(-1, (G, S)), k=k.unflatten(-1, (G, S)), v=v.unflatten(-1, (nh, H)))
    y1, f1 = bd.mamba2_gdr_fwd(**e, initial_state=h0)
    y2, f2 = bd.mamba2_gdr_fwd(**d, initial_state=h0)
    assert rel_err(np64(y1), np64(y2)) <= TOL_Y[dtype] and rel_err(np64(f1), np64(f2)) <= TOL_STATE


def test_gdr_on_another_stream_and_twice():
    d, h0 = gdr_inputs(2, 333, 4, 2, 128, 128, BF16)
    y1, f1 = bd.mamba2_gdr_fwd(**d, initial_state=h0)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y2, f2 = bd.mamba2_gdr_fwd(**d, initial_state=h0)
    y3, f3 = bd.mamba2_gdr_fwd(**d, initial_state=h0, stream=s)
    s.synchronize()
    assert torch.equal(y1, y2) and torch.equal(f1, f2) and torch.equal(y1, y3) and torch.equal(f1, f3)


def test_gdr_in_a_graph():
    d, h0 = gdr_inputs(1, 200, 4, 2, 128, 128, BF16)
    y, fin = bd.mamba2_gdr_fwd(**d, initial_state=h0)
    y2, fin2 = torch.zeros_like(y), torch.zeros_like(fin)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bd.mamba2_gdr_fwd(**d, initial_state=h0, y=y2, final_state=fin2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(fin, fin2)


# ---------------------------------------------------------------- one token
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("b,nh,G,H,S", [
    (3, 4, 2, 64, 128), (2, 4, 1, 128, 128), (1, 2, 2, 128, 64), (2, 2, 1, 64, 256), (1, 3, 3, 256, 33),
    (2, 3, 1, 5, 7), (1, 1, 1, 1, 1), (2, 2, 1, 33, 200),
])
def test_gdr_step(b, nh, G, H, S, dtype):
    d, h0 = gdr_inputs(b, 1, nh, G, H, S, dtype, unit=False)
    t = {n: x[:, 0].contiguous() for n, x in d.items()}
    y, out = Guarded((b, nh, H), dtype), Guarded((b, nh, S, H), FP32)
    bd.mamba2_gdr_step(**t, state_in=h0, scale=0.2, qk_l2norm=True, y=y.t, state_out=out.t)
    y_ref, h_ref = ref.gdr(**d, scale=0.2, l2norm=True, init=h0)
    assert y.intact() and out.intact()
    assert rel_err(np64(y.t), y_ref[:, 0]) <= (TOL_ROUND[BF16] if dtype == BF16 else 1e-5)
    assert rel_err(np64(out.t), h_ref) <= 1e-5
    st = h0.clone()
    y2, st2 = bd.mamba2_gdr_step(**t, state_in=st, scale=0.2, qk_l2norm=True, state_out=st)
    assert st2 is st and torch.equal(st, out.t) and torch.equal(y2, y.t)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("b,nh,G,H,S", [
    (80, 16, 4, 64, 64), (1301, 1, 1, 40, 128), (650, 1, 1, 128, 96), (330, 2, 2, 100, 200), (3, 4, 2, 8, 128),
    (2, 3, 1, 16, 64), (5, 2, 1, 12, 256), (1, 2, 1, 36, 40),
])
def test_gdr_step_of_many_sequences_and_narrow_heads(b, nh, G, H, S, dtype):
    test_gdr_step(b, nh, G, H, S, dtype)


def test_gdr_step_from_nothing_and_without_decay():
    d, h0 = gdr_inputs(2, 1, 2, 1, 64, 128, BF16)
    t = {n: x[:, 0].contiguous() for n, x in d.items()}
    y, h = bd.mamba2_gdr_step(**t)
    y_ref, h_ref = ref.gdr(**d, scale=128 ** -0.5)
    assert rel_err(np64(y), y_ref[:, 0]) <= TOL_ROUND[BF16] and rel_err(np64(h), h_ref) <= 1e-5
    t["g"].zero_(), t["beta"].zero_()
    _, h = bd.mamba2_gdr_step(**t, state_in=h0)
    assert torch.equal(h, h0)


@pytest.mark.parametrize("H", [64, 128, 40])
def test_gdr_prefill_then_steps(H):
    L, P = 140, 133
    d, h0 = gdr_inputs(2, L, 4, 2, H, 128, BF16)
    _, st = bd.mamba2_gdr_fwd(**{n: t[:, :P].contiguous() for n, t in d.items()}, initial_state=h0)
    ys = [bd.mamba2_gdr_step(**{n: t[:, i].contiguous() for n, t in d.items()}, state_in=st, state_out=st)[0]
          for i in range(P, L)]
    y_ref, fin_ref = ref.gdr(**d, scale=128 ** -0.5, init=h0)
    assert rel_err(np64(torch.stack(ys, 1)), y_ref[:, P:]) <= TOL_Y[BF16]
    assert rel_err(np64(st), fin_ref) <= TOL_STATE


# -------------------------------------------------------------- convolution
def conv_inputs(b, L, C, W, dtype, seed=0):
    r = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=r).cuda()  # noqa: E731
    return n(b, L, C).to(dtype), n(C, W), n(C), n(b, W - 1, C).to(dtype)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("b,L,C,W", [
    (2, 70, 64, 4), (1, 1, 8, 4), (3, 2, 16, 4), (2, 33, 24, 3), (1, 64, 1032, 2), (2, 40, 7, 4), (1, 5, 8, 8),
    (1, 100, 40, 5), (2, 31, 13, 6), (1, 12, 32, 7),
])
def test_conv(b, L, C, W, dtype):
    x, w, bias, s0 = conv_inputs(b, L, C, W, dtype, seed=L)
    y, fin = Guarded((b, L, C), dtype), Guarded((b, W - 1, C), dtype)
    bd.mamba2_causal_conv_fwd(x, w, bias=bias, initial_state=s0, y=y.t, final_state=fin.t)
    y_ref, fin_ref = ref.conv(x, w, bias, True, s0)
    assert y.intact() and fin.intact()
    assert rel_err(np64(y.t), y_ref) <= TOL_ROUND[dtype] and np.array_equal(np64(fin.t), fin_ref)
    y2, none = bd.mamba2_causal_conv_fwd(x, w, silu=False, want_final_state=False)
    assert none is None and rel_err(np64(y2), ref.conv(x, w, None, False)[0]) <= TOL_ROUND[dtype]


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("W", [2, 3, 4, 5, 8])
@pytest.mark.parametrize("C", [820, 822, 823])
def test_conv_channels_in_vectors_of_four_two_and_one(C, W, dtype):
    r = torch.Generator().manual_seed(C + W)
    n = lambda *s: torch.randn(*s, generator=r)  # noqa: E731
    b, L = 2, 150
    x, init = n(b, L, C).to(dtype).cuda(), n(b, W - 1, C).to(dtype).cuda()
    w, bias = n(C, W).cuda() / W, n(C).cuda()
    y, fin = Guarded((b, L, C), dtype), Guarded((b, W - 1, C), dtype)
    bd.mamba2_causal_conv_fwd(x, w, bias=bias, initial_state=init, y=y.t, final_state=fin.t)
    assert y.intact() and fin.intact()
    y_ref, _ = ref.conv(x, w, bias=bias, init=init)
    assert rel_err(np64(y.t), y_ref) <= TOL_ROUND[dtype]
    assert torch.equal(fin.t, x[:, L - W + 1:])


@pytest.mark.parametrize("C", [64, 9])
def test_conv_ragged_batch_with_nan_past_the_ends(C):
    L, W = 50, 4
    lengths = torch.tensor([0, 1, 2, 3, 4, 31, 32, 33, 50, 70, -1], dtype=torch.int32, device="cuda")
    x, w, bias, s0 = conv_inputs(len(lengths), L, C, W, BF16)
    clean = x.clone()
    for i, n in enumerate(lengths.clamp(0, L).tolist()):
        x[i, n:] = NAN
    y, fin = bd.mamba2_causal_conv_fwd(x, w, bias=bias, initial_state=s0, lengths=lengths)
    y_ref, fin_ref = ref.conv(clean, w, bias, True, s0, lengths)
    assert rel_err(np64(y), y_ref) <= TOL_ROUND[BF16] and np.array_equal(np64(fin), fin_ref)


def test_conv_infinite_input_reaches_only_its_window():
    x, w, bias, _ = conv_inputs(1, 20, 8, 4, BF16)
    x[0, 5] = float("inf")
    y, _ = bd.mamba2_causal_conv_fwd(x, w, bias=bias, silu=False)
    finite = torch.isfinite(y[0]).all(-1).tolist()
    assert finite == [not 5 <= t < 9 for t in range(20)]


@pytest.mark.parametrize("off,dtype", [(8, BF16), (3, BF16), (4, FP32), (1, FP32)])
def test_conv_of_a_slice(off, dtype):
    x, w, bias, s0 = conv_inputs(2, 40, 64, 4, dtype)
    wide = torch.zeros(2, 40, 100, device="cuda", dtype=dtype)
    part = wide[..., off:off + 64]
    part.copy_(x)
    out = torch.full((2, 40, 120), 7.0, device="cuda", dtype=dtype)
    y, f = bd.mamba2_causal_conv_fwd(part, w, bias=bias, initial_state=s0, y=out[..., off:off + 64])
    y2, f2 = bd.mamba2_causal_conv_fwd(x, w, bias=bias, initial_state=s0)
    assert torch.equal(y, y2) and torch.equal(f, f2)
    assert bool((out[..., :off] == 7).all()) and bool((out[..., off + 64:] == 7).all())


def test_conv_offsets_beyond_32_bits():
    L, C = 70_000, 32_768
    x = torch.randn(1, L, C, device="cuda", dtype=BF16)
    w = torch.randn(C, 4, device="cuda")
    assert x.numel() > 2 ** 31
    y, fin = bd.mamba2_causal_conv_fwd(x, w)
    tail, _ = bd.mamba2_causal_conv_fwd(x[:, -50:].contiguous(), w, initial_state=x[:, -53:-50].contiguous())
    assert torch.equal(y[:, -50:], tail) and torch.equal(fin, x[:, -3:])


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("b,C,W", [(300, 64, 4), (3, 64, 4), (1, 7, 4), (2, 1032, 3), (2, 8, 2), (1, 16, 8)])
def test_conv_step_continues_a_sequence(b, C, W, dtype):
    x, w, bias, s0 = conv_inputs(b, 12, C, W, dtype)
    _, st = bd.mamba2_causal_conv_fwd(x[:, :5].contiguous(), w, bias=bias, initial_state=s0)
    ys = []
    for t in range(5, 12):
        new, out = bd.mamba2_causal_conv_step(x[:, t].contiguous(), w, state_in=st, bias=bias)
        y, st = bd.mamba2_causal_conv_step(x[:, t].contiguous(), w, state_in=st, bias=bias, state_out=st)
        assert torch.equal(y, new) and torch.equal(st, out)
        ys.append(y)
    y_ref, fin_ref = ref.conv(x, w, bias, True, s0)
    assert rel_err(np64(torch.stack(ys, 1)), y_ref[:, 5:]) <= TOL_ROUND[dtype]
    assert np.array_equal(np64(st), fin_ref)
    y, _ = bd.mamba2_causal_conv_step(x[:, 0].contiguous(), w, silu=False)
    assert rel_err(np64(y), ref.conv(x[:, :1], w, None, False)[0][:, 0]) <= TOL_ROUND[dtype]


# --------------------------------------------------------------------- norm
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("mode", ["none", "silu", "before", "after"])
@pytest.mark.parametrize("rows,groups,size", [
    (5, 4, 64), (3, 3, 128), (9, 2, 33), (1, 1, 1), (2, 1, 4096), (3, 2, 1000), (33, 5, 8), (2, 1, 300), (2, 3, 520),
    (1, 1, 8200), (2, 1, 2049),
])
def test_norm(rows, groups, size, mode, dtype):
    r = torch.Generator().manual_seed(size)
    n = lambda *s: torch.randn(*s, generator=r).cuda()  # noqa: E731
    C = groups * size
    x, w, bias = (n(rows, C) + 0.5).to(dtype), n(C), n(C)
    z = n(rows, C).to(dtype) if mode in ("before", "after") else None
    for mean in (False, True):
        y = Guarded((rows, C), dtype)
        bd.mamba2_group_norm(x, w, groups, z=z, bias=bias, eps=1e-5, subtract_mean=mean, mode=mode, y=y.t)
        assert y.intact()
        want = ref.norm(x, groups, w, bias, z, 1e-5, mean, mode)
        assert rel_err(np64(y.t), want) <= TOL_ROUND[dtype]
    y = bd.mamba2_group_norm(x, None, groups, z=z, mode=mode)
    assert rel_err(np64(y), ref.norm(x, groups, z=z, mode=mode)) <= TOL_ROUND[dtype]


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("mode", ["silu", "before"])
@pytest.mark.parametrize("rows,groups,size", [
    (9001, 1, 520), (4001, 3, 1000), (7001, 3, 100), (2001, 1, 2052), (6007, 1, 1496), (3001, 1, 2056), (2999, 1, 4096), (1501, 1, 8192), (701, 1, 16384),
])
def test_norm_of_many_rows(rows, groups, size, mode, dtype):
    """Every block walks down several rows, of a slice of a wider tensor; a NaN
    stays in its row."""
    r = torch.Generator(device="cuda").manual_seed(size)
    C = groups * size
    wide = (torch.randn(rows, 2 * C + 8, generator=r, device="cuda") + 0.5).to(dtype)
    x, w = wide[:, :C], torch.randn(C, generator=r, device="cuda")
    z = wide[:, C + 8:] if mode == "before" else None
    bad = rows // 2
    wide[bad, 5] = NAN
    y = Guarded((rows, C), dtype)
    bd.mamba2_group_norm(x, w, groups, z=z, mode=mode, subtract_mean=mode == "silu", y=y.t)
    assert y.intact()
    u = x.double() * torch.nn.functional.silu(z.double()) if z is not None else x.double()
    u = u.reshape(rows, groups, size)
    if mode == "silu":
        u = u - u.mean(-1, keepdim=True)
    u = (u / (u.square().mean(-1, keepdim=True) + 1e-5).sqrt()).reshape(rows, C) * w.double()
    want = torch.nn.functional.silu(u) if mode == "silu" else u
    keep = torch.arange(rows, device="cuda") != bad
    assert torch.isnan(y.t[bad, :size]).all() and not torch.isnan(y.t[keep]).any()
    err = (y.t[keep].double() - want[keep]).abs().amax() / want[keep].abs().amax()
    assert float(err) <= TOL_ROUND[dtype]


@pytest.mark.parametrize("size", [32768, 16400])
def test_norm_of_the_largest_groups(size):
    x = torch.randn(2, size, device="cuda").bfloat16()
    z = torch.randn(2, size, device="cuda").bfloat16()
    y = bd.mamba2_group_norm(x, None, 1, z=z, mode="after", subtract_mean=True)
    assert rel_err(np64(y), ref.norm(x, 1, z=z, mode="after", mean=True)) <= TOL_ROUND[BF16]
    odd = bd.mamba2_group_norm(x[:, :size - 1], None, 1)
    assert rel_err(np64(odd), ref.norm(x[:, :size - 1], 1)) <= TOL_ROUND[BF16]


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("size", [17, 65, 129, 257, 513, 1025, 4097, 16383, 32767])
def test_norm_of_odd_groups(size, dtype):
    r = torch.Generator().manual_seed(size)
    x, w = torch.randn(7, 3 * size, generator=r).to(dtype).cuda(), torch.randn(3 * size, generator=r).cuda()
    y = Guarded((7, 3 * size), dtype)
    bd.mamba2_group_norm(x, w, 3, z=x, mode="after", subtract_mean=True, y=y.t)
    assert y.intact()
    assert rel_err(np64(y.t), ref.norm(x, 3, w, None, x, 1e-5, True, "after")) <= TOL_ROUND[dtype]


def test_norm_far_from_zero():
    """A mean far larger than the spread: the squares are of the differences."""
    x = 1000 + torch.randn(4, 512, device="cuda")
    y = bd.mamba2_group_norm(x, None, 2, subtract_mean=True, eps=1e-5)
    # each input's own fp32 rounding (2^-24 of 1000) is exact in both; the mean's is 2^-22 of 1000
    assert rel_err(np64(y), ref.norm(x, 2, mean=True)) <= 1e-3


def test_norm_nan_stays_in_its_group():
    x = torch.randn(3, 256, device="cuda").bfloat16()
    x[1, 70] = NAN
    y = bd.mamba2_group_norm(x, None, 4)
    bad = torch.isnan(y).unflatten(-1, (4, 64)).any(-1)
    assert bad.sum() == 1 and bool(bad[1, 1])
    assert bool(torch.isnan(y[1, 64:128]).all())


@pytest.mark.parametrize("off", [8, 5])
def test_norm_of_slices(off):
    wide = torch.randn(2, 9, 300, device="cuda").bfloat16()
    x, z = wide[..., off:off + 128], wide[..., 150 + off % 8:278 + off % 8]
    y = bd.mamba2_group_norm(x, None, 2, z=z, mode="after")
    y2 = bd.mamba2_group_norm(x.contiguous(), None, 2, z=z.contiguous(), mode="after")
    assert rel_err(np64(y), ref.norm(x, 2, z=z, mode="after")) <= TOL_ROUND[BF16]
    assert rel_err(np64(y2), np64(y)) <= TOL_ROUND[BF16]


def test_norm_offsets_beyond_32_bits():
    rows, C = 540_000, 4096
    x = torch.randn(rows, C, device="cuda", dtype=BF16)
    y = bd.mamba2_group_norm(x, None, 64, z=x, mode="after")
    assert x.numel() > 2 ** 31
    for at in (0, 524_287, 524_288, rows - 1):
        row = x[at:at + 1].contiguous()
        assert torch.equal(y[at:at + 1], bd.mamba2_group_norm(row, None, 64, z=row, mode="after"))


@pytest.mark.parametrize("groups", [1, 2, 3, 7, 33, 100])
def test_norm_row_and_group_counts(groups):
    """Blocks that span several rows, several groups, and parts of either."""
    for rows in (1, 2, 31, 257):
        x = torch.randn(rows, groups * 48, device="cuda").bfloat16()
        y = bd.mamba2_group_norm(x, None, groups)
        assert rel_err(np64(y), ref.norm(x, groups)) <= TOL_ROUND[BF16]


def test_norm_of_no_rows():
    assert bd.mamba2_group_norm(torch.empty(0, 64, device="cuda"), None, 2).shape == (0, 64)
