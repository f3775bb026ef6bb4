"""GPU parity of the gated linear recurrence, the block norm and the gradients
against their plain fp64 forms.

Tolerances are on max|err| / max|ref| and follow from the arithmetic:
- a value that leaves as bf16 is rounded once, by at most half a step: 2^-8 of
  the largest value, on top of the fp32 work before it;
- gates and factors are each within a few 1e-7 of themselves (exponents of up to
  16 rounded to fp32: 16 x 2^-24 = 1e-6 at most), an error of log a is one of log a
  itself, which the memory 1 / (1 - a) of the recurrence turns into the same share of
  h; a result meets at most six of these and sums of a few terms: 1e-5;
- a sum over tokens or rows (a weight's gradient) has the errors of its terms:
  1e-5 of the sum of their absolute values, and so has a gradient through a norm,
  k (q - u mean(q u)): a difference, which with few channels is far smaller than its
  terms, each of them rounded by itself (one channel: it vanishes but for eps);
- a state that is only copied is exact, and so is what a row's end hides.
"""
import pytest
import torch

import gated_linear_ref as ref
from gpu_helpers import Guarded
from mamba_chunked_ssd_gb300 import binding as bd

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
TOL = {BF16: 2.0 ** -8 + 1e-5, FP32: 1e-5}
NAN, INF = float("nan"), float("inf")
BOTH = pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mamba_chunked_ssd_gb300 import build_lib
    build_lib.build()
    bd.load_library()


def close(got, want, tol, size=None, name=""):
    got, want = got.detach().cpu().double(), want.double()
    assert got.shape == want.shape, name
    if not want.numel():
        return
    err = (got - want).abs().max().item()
    top = want.abs().max().item()
    most = tol * max(top, 1e-30) if size is None else (tol - TOL[FP32]) * top + TOL[FP32] * size.max().item()
    assert err <= most, f"{name}: {err:.3e} of {top:.3e}, at most {most:.3e}"


def gen(seed):
    r = torch.Generator().manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=r)


def glr_inputs(b, L, C, dtype, seed=0, gated=False, state=True):
    n = gen(seed)
    d = {"x": n(b, L, C).to(dtype), "r": n(b, L, C).to(dtype), "i": n(b, L, C).to(dtype),
         "A": -torch.exp(1.5 * n(C) - 2), "z": n(b, L, C).to(dtype) if gated else None}
    init = 0.5 * n(b, C) if state else None
    return {k: None if t is None else t.cuda() for k, t in d.items()}, None if init is None else init.cuda()


def f64s(d):
    return {k: ref.f64(t) for k, t in d.items()}


def check_glr(d, init, lengths=None, clean=None, grads=True, seed=1):
    """Forward, chunk states and gradients; `clean`: the inputs without what lies past the rows' ends."""
    b, L, C = d["x"].shape
    dtype, clean = d["x"].dtype, f64s(clean or d)
    nc = -(-L // 64)
    y, fin, cs = Guarded((b, L, C), dtype), Guarded((b, C), FP32), Guarded((b, nc, C), FP32)
    bd.mamba2_glr_fwd(**d, initial_state=init, lengths=lengths, y=y.t, final_state=fin.t, chunk_states=cs.t)
    bd.mamba2_check_device_status()
    assert y.intact() and fin.intact() and cs.intact()
    y_ref, fin_ref, hs = ref.glr(**clean, init=ref.f64(init), lengths=lengths)
    close(y.t, y_ref, TOL[dtype], name="y")
    close(fin.t, fin_ref, TOL[FP32], name="final_state")
    h0 = torch.zeros(b, C, dtype=torch.float64) if init is None else ref.f64(init)
    close(cs.t, torch.cat([h0[:, None], hs[:, 63:-1:64]], 1)[:, :nc], TOL[FP32], name="chunk_states")
    if not grads:
        return
    n = gen(seed)
    dy, dfin = n(b, L, C).to(dtype).cuda(), n(b, C).cuda() if init is not None else None
    dirty = dy.clone()
    for k, m in enumerate(ref.counts(lengths, b, L)):
        dirty[k, m:] = NAN
    outs = {k: Guarded((b, L, C), dtype) for k in ("dx", "dr", "di")}
    if d["z"] is not None:
        outs["dz"] = Guarded((b, L, C), dtype)
    outs["dA"], outs["dinitial_state"] = Guarded((C,), FP32), Guarded((b, C), FP32)
    bd.mamba2_glr_bwd(dirty, **d, chunk_states=cs.t, dfinal_state=dfin, lengths=lengths,
                      **{k: g.t for k, g in outs.items()})
    bd.mamba2_check_device_status()
    assert all(g.intact() for g in outs.values())
    want, size = ref.glr_grads(ref.f64(dy), **clean, init=ref.f64(init), lengths=lengths, dfinal=ref.f64(dfin))
    for k in ("dx", "dr", "di", "dz"):
        if k in want:
            close(outs[k].t, want[k], TOL[dtype], name=k)
    close(outs["dA"].t, want["dA"], TOL[FP32], size, name="dA")
    close(outs["dinitial_state"].t, want["dinit"], TOL[FP32], name="dinit")
    return y.t, fin.t, {k: g.t for k, g in outs.items()}


# --------------------------------------------------- gated linear recurrence
@BOTH
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("L", [1, 2, 7, 8, 9, 63, 64, 65, 127, 128, 129, 200, 513])
def test_glr_lengths_of_sequences(L, gated, dtype):
    d, h0 = glr_inputs(2, L, 72, dtype, seed=L, gated=gated)
    check_glr(d, h0)


@BOTH
@pytest.mark.parametrize("C", [1, 2, 3, 8, 31, 63, 64, 65, 66, 68, 127, 128, 130, 200, 1000])
def test_glr_numbers_of_channels(C, dtype):
    d, h0 = glr_inputs(3, 75, C, dtype, seed=C, gated=C % 2 == 0)
    check_glr(d, h0)


@BOTH
def test_glr_without_states(dtype):
    d, _ = glr_inputs(2, 130, 40, dtype, state=False)
    check_glr(d, None)
    y, none, no_chunks = bd.mamba2_glr_fwd(**d, want_final_state=False)
    assert none is None and no_chunks is None


@BOTH
@pytest.mark.parametrize("b,L,C", [(1, 1500, 64), (1, 1500, 33), (3, 520, 128), (1, 700, 520), (700, 130, 64), (2, 300, 8200)])
def test_glr_few_and_many_strips(b, L, C, dtype):
    """Sequences that a cluster's blocks share, by two, four and eight, and ones that a block walks alone."""
    d, h0 = glr_inputs(b, L, C, dtype, seed=L, gated=L == 1500)
    check_glr(d, h0)


@pytest.mark.parametrize("gated", [False, True])
def test_glr_strips_that_are_left_over(gated):
    """More strips than the GPU takes at once, a few of them left over: those are split between the blocks of
    clusters, beside the others.  Every channel is one of a sequence that is known; a row of them ends early."""
    L, C = 64 * 64 + 9, 32 * 40
    b = 16
    n = gen(3)
    base = {k: n(1, L, 32).cuda() for k in ("x", "r", "i", "z", "dy")}
    A = (-torch.exp(n(32))).cuda()
    wide = {k: t.to(BF16).repeat(b, 1, C // 32).contiguous() for k, t in base.items()}
    lengths = torch.full((b,), L, dtype=torch.int32, device="cuda")
    lengths[-1] = 4000
    z = wide["z"] if gated else None
    y, fin, cs = bd.mamba2_glr_fwd(wide["x"], wide["r"], wide["i"], A.repeat(C // 32), z=z, lengths=lengths,
                                   want_chunk_states=True)
    grads = bd.mamba2_glr_bwd(wide["dy"], wide["x"], wide["r"], wide["i"], A.repeat(C // 32), cs, z=z, lengths=lengths)
    bd.mamba2_check_device_status()
    one = {k: t.to(BF16) for k, t in base.items()}
    for rows, m in ((slice(0, b - 1), L), (slice(b - 1, b), 4000)):
        part = {k: t[:, :m].contiguous() for k, t in one.items()}
        z1 = part["z"] if gated else None
        y1, fin1, cs1 = bd.mamba2_glr_fwd(part["x"], part["r"], part["i"], A, z=z1, want_chunk_states=True)
        want = bd.mamba2_glr_bwd(part["dy"], part["x"], part["r"], part["i"], A, cs1, z=z1)
        close(y[rows, :m], y1.repeat(b, 1, C // 32)[rows].cpu(), TOL[BF16], name="y")
        close(fin[rows], fin1.repeat(b, C // 32)[rows].cpu(), TOL[FP32], name="state")
        for got, w, name in zip(grads[:4], want[:4], ("dx", "dr", "di", "dz")):
            if w is not None:
                close(got[rows, :m], w.repeat(b, 1, C // 32)[rows].cpu(), TOL[BF16], name=name)
                assert bool((got[rows, m:] == 0).all())
        close(grads[5][rows], want[5].repeat(b, C // 32)[rows].cpu(), TOL[FP32], name="dinit")


@BOTH
@pytest.mark.parametrize("C", [64, 37])
@pytest.mark.parametrize("gated", [False, True])
def test_glr_ragged_batch(gated, C, dtype):
    """Rows of every kind of length (beyond L and below 0 too), with NaN and infinities past
    each row's end: outputs are 0 there, the state stays."""
    L = 150
    lengths = torch.tensor([0, 1, 7, 8, 63, 64, 65, 100, 128, 149, 150, 999, -7], dtype=torch.int32, device="cuda")
    d, h0 = glr_inputs(len(lengths), L, C, dtype, gated=gated)
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


@BOTH
def test_glr_slices_of_a_projection(dtype):
    """x, r, i, z side by side in one tensor, and their gradients in another."""
    b, L, C = 2, 100, 96
    n = gen(4)
    wide = n(b, L, 4 * C).to(dtype).cuda()
    x, r, i, z = wide.split(C, -1)
    A, h0 = -torch.rand(C, generator=torch.Generator().manual_seed(1)).cuda(), n(b, C).cuda()
    y, fin, cs = bd.mamba2_glr_fwd(x, r, i, A, z=z, initial_state=h0, want_chunk_states=True)
    same = bd.mamba2_glr_fwd(*(t.contiguous() for t in (x, r, i)), A, z=z.contiguous(), initial_state=h0,
                             want_chunk_states=True)
    assert all(torch.equal(a, c) for a, c in zip((y, fin, cs), same))
    grad = torch.full_like(wide, NAN)
    dx, dr, di, dz = grad.split(C, -1)
    dy = n(b, L, C).to(dtype).cuda()
    got = bd.mamba2_glr_bwd(dy, x, r, i, A, cs, z=z, dx=dx, dr=dr, di=di, dz=dz)
    want = bd.mamba2_glr_bwd(dy, *(t.contiguous() for t in (x, r, i)), A, cs, z=z.contiguous())
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    assert torch.equal(grad, torch.cat(want[:4], -1))


@BOTH
@pytest.mark.parametrize("shift", [1, 2, 4])
def test_glr_rows_on_any_element(shift, dtype):
    """Slices that start on single elements, pairs and fours."""
    b, L, C = 2, 70, 64
    n = gen(5)
    wide = n(3, b, L, C + 8).to(dtype).cuda()
    x, r, i = (t[..., shift:shift + C] for t in wide)
    A = -torch.ones(C, device="cuda")
    got = bd.mamba2_glr_fwd(x, r, i, A)
    want = bd.mamba2_glr_fwd(x.contiguous(), r.contiguous(), i.contiguous(), A)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_glr_far_gates_and_decays():
    """Gates that are fully open or shut, decays from nearly none to all at once: finite
    everywhere, a shut gate keeps the state (to fp32's rounding: a warp takes up its state as
    a t + b of the tokens before, with other roundings than token by token), NaN stays in its
    channel."""
    b, L, C = 1, 70, 64
    d, h0 = glr_inputs(b, L, C, FP32, seed=3)
    d["A"][:8] = torch.tensor([0.0, -1e-30, -1e-10, -1e-4, -50.0, -200.0, -1e4, -1e30])
    d["r"][:, 10:20] = -INF
    d["r"][:, 30:40, 8:16] = 200.0
    d["r"][:, 30:40, 16:24] = -200.0
    d["i"][:, 50:60] = -INF
    y, fin, cs = bd.mamba2_glr_fwd(**d, initial_state=h0, want_chunk_states=True)
    assert torch.isfinite(y).all()
    close(y[:, 10:20], y[:, 9:10].expand(-1, 10, -1).cpu(), TOL[FP32])
    assert torch.equal(y[:, 10:16], y[:, 9:10].expand(-1, 6, -1))  # one warp's tokens
    y_ref, fin_ref, _ = ref.glr(**f64s(d), init=ref.f64(h0))
    close(y, y_ref, TOL[FP32]), close(fin, fin_ref, TOL[FP32])
    dx, dr, di, _, dA, dh = bd.mamba2_glr_bwd(torch.ones_like(y), **d, chunk_states=cs)
    assert all(torch.isfinite(t).all() for t in (dx, dr, di, dh)) and torch.isfinite(dA[1:]).all()
    assert bool(torch.isnan(dA[0]))  # no derivative at A = 0
    assert bool((dr[:, 10:20] == 0).all()) and bool((di[:, 50:60] == 0).all())
    d["r"][0, 40, 5], d["x"][0, 40, 6], d["i"][0, 40, 7] = NAN, NAN, NAN
    y2, fin2, cs2 = bd.mamba2_glr_fwd(**d, initial_state=h0, want_chunk_states=True)
    assert torch.equal(y2[:, :40], y[:, :40]) and torch.isnan(y2[0, 40:, 5:8]).all()
    assert torch.equal(y2[..., 8:], y[..., 8:]) and torch.isnan(fin2[0, 5:8]).all()


def test_glr_small_decays_keep_their_precision():
    """a within 1e-7 .. 1e-3 of 1: sqrt(1 - a^2) is taken without cancellation, and a's
    rounding does not add up over 4000 tokens (a share 2^-24 a token, either way: at most
    4000 x 2^-24 = 2.4e-4 of h, and as the root of their number if they were independent)."""
    d, h0 = glr_inputs(1, 4000, 64, FP32, seed=8)
    d["A"] = -torch.logspace(-7, -3, 64).cuda()
    y, fin, _ = bd.mamba2_glr_fwd(**d, initial_state=h0)
    y_ref, fin_ref, _ = ref.glr(**f64s(d), init=ref.f64(h0))
    close(y, y_ref, 4000 * 2.0 ** -24), close(fin, fin_ref, 4000 * 2.0 ** -24)


def test_glr_rows_past_32_bit_offsets():
    """More than 2^31 elements: the last batch rows' offsets do not fit 32 bits."""
    b, L, C = 9, 4200, 65536
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    x = torch.zeros(b, L, C, dtype=BF16, device="cuda")
    n = gen(2)
    last = {k: n(1, L, 64).to(BF16).cuda() for k in ("x", "r", "i")}
    big = {k: x.clone() for k in ("r", "i")}
    big["x"] = x
    for k, t in last.items():
        big[k][-1:, :, -64:] = t
    A = -torch.ones(C, device="cuda")
    y, fin, cs = bd.mamba2_glr_fwd(big["x"], big["r"], big["i"], A, want_chunk_states=True)
    y1, fin1, cs1 = bd.mamba2_glr_fwd(last["x"], last["r"], last["i"], A[:64])
    close(y[-1:, :, -64:], y1.cpu(), TOL[BF16]), close(fin[-1:, -64:], fin1.cpu(), 1e-5)
    assert bool((y[0] == 0).all())


@BOTH
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("b,C", [(1, 1), (1, 64), (3, 7), (5, 256), (2, 258), (257, 130)])
def test_glr_step(b, C, gated, dtype):
    d, h0 = glr_inputs(b, 1, C, dtype, seed=C, gated=gated)
    one = {k: t[:, 0] if t is not None and t.dim() == 3 else t for k, t in d.items()}
    y, out = Guarded((b, C), dtype), Guarded((b, C), FP32)
    bd.mamba2_glr_step(**one, state_in=h0, state_out=out.t, y=y.t)
    assert y.intact() and out.intact()
    y_ref, fin, _ = ref.glr(**f64s(d), init=ref.f64(h0))
    close(y.t, y_ref[:, 0], TOL[dtype]), close(out.t, fin, TOL[FP32])
    kept = h0.clone()
    y2, same = bd.mamba2_glr_step(**one, state_in=kept, state_out=kept)
    assert same is kept and torch.equal(kept, out.t) and torch.equal(y2, y.t)
    y3, fresh = bd.mamba2_glr_step(**one)
    y_ref, fin, _ = ref.glr(**f64s(d))
    close(y3, y_ref[:, 0], TOL[dtype]), close(fresh, fin, TOL[FP32])


@BOTH
def test_glr_prefill_in_parts_then_steps(dtype):
    """A sequence in two parts and then token by token, as a server runs it, against the whole one."""
    d, h0 = glr_inputs(2, 150, 64, dtype, gated=True)
    whole, last, _ = bd.mamba2_glr_fwd(**d, initial_state=h0)
    part = lambda a, c: {k: t[:, a:c].contiguous() if t.dim() == 3 else t for k, t in d.items()}  # noqa: E731
    y1, h, _ = bd.mamba2_glr_fwd(**part(0, 71), initial_state=h0)
    y2, h, _ = bd.mamba2_glr_fwd(**part(71, 140), initial_state=h)
    ys = [y1, y2]
    for t in range(140, 150):
        y, h = bd.mamba2_glr_step(**{k: v[:, t].contiguous() if v.dim() == 3 else v for k, v in d.items()},
                                  state_in=h, state_out=h)
        ys.append(y[:, None])
    close(torch.cat(ys, 1), whole.cpu(), TOL[dtype]), close(h, last.cpu(), TOL[FP32])


def test_glr_gradient_against_differences():
    """The forward kernel's own differences along random directions (fp32, step 2^-7 with
    errors of its square's size times a third derivative, and 2^-23 x 2^7 x the loss's size of rounding)."""
    d, h0 = glr_inputs(2, 100, 64, FP32, seed=6, gated=True)
    n = gen(7)
    dy, dfin = n(2, 100, 64).cuda(), n(2, 64).cuda()
    _, _, cs = bd.mamba2_glr_fwd(**d, initial_state=h0, want_chunk_states=True)
    dx, dr, di, dz, dA, dh = bd.mamba2_glr_bwd(dy, **d, chunk_states=cs, dfinal_state=dfin)
    grads = {"x": dx, "r": dr, "i": di, "z": dz, "A": dA, "init": dh}

    def loss(v):
        y, fin, _ = bd.mamba2_glr_fwd(v["x"], v["r"], v["i"], v["A"], z=v["z"], initial_state=v["init"])
        return (y.double() * dy).sum() + (fin.double() * dfin).sum()

    at = {**d, "init": h0}
    for name, g in grads.items():
        way = n(*g.shape).cuda() * (0.1 * at["A"].abs() if name == "A" else 1.0)
        e = 2.0 ** -7
        up, down = ({**at, name: at[name] + s * e * way} for s in (1, -1))
        slope = (loss(up) - loss(down)).item() / (2 * e)
        want = (g.double() * way).sum().item()
        scale = (g.double() * way).norm().item() + abs(want)
        assert abs(slope - want) <= 1e-2 * scale, name


# ---------------------------------------------- gradient of the convolution
def conv_inputs(b, L, C, W, dtype, seed=0, bias=True, state=True):
    n = gen(seed)
    d = dict(x=n(b, L, C).to(dtype).cuda(), weight=(n(C, W) * W ** -0.5).cuda(), bias=n(C).cuda() if bias else None)
    return d, n(b, W - 1, C).to(dtype).cuda() if state else None, n(b, L, C).to(dtype).cuda(), \
        n(b, W - 1, C).to(dtype).cuda() if state else None


def check_conv(d, init, dy, dfin, silu=True, lengths=None, clean=None):
    b, L, C = d["x"].shape
    W, dtype = d["weight"].shape[1], d["x"].dtype
    outs = {"dx": Guarded((b, L, C), dtype), "dweight": Guarded((C, W), FP32),
            "dinitial_state": Guarded((b, W - 1, C), dtype)}
    if d["bias"] is not None:
        outs["dbias"] = Guarded((C,), FP32)
    bd.mamba2_causal_conv_bwd(dy, **d, silu=silu, initial_state=init, lengths=lengths, dfinal_state=dfin,
                              **{k: g.t for k, g in outs.items()})
    bd.mamba2_check_device_status()
    assert all(g.intact() for g in outs.values())
    c = f64s(clean or {**d, "dy": dy})
    want, size = ref.conv_grads(c["dy"], c["x"], c["weight"], c["bias"], act=silu, init=ref.f64(init), lengths=lengths,
                                dfinal=ref.f64(dfin))
    close(outs["dx"].t, want["dx"], TOL[dtype], name="dx")
    close(outs["dinitial_state"].t, want["dinit"], TOL[dtype], name="dinit")
    close(outs["dweight"].t, want["dweight"], TOL[FP32], size["dweight"], name="dweight")
    if d["bias"] is not None:
        close(outs["dbias"].t, want["dbias"], TOL[FP32], size["dbias"], name="dbias")
    return {k: g.t for k, g in outs.items()}


@BOTH
@pytest.mark.parametrize("W", [2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("C", [1, 2, 6, 40, 513])
def test_conv_bwd_widths_and_channels(C, W, dtype):
    check_conv(*conv_inputs(2, 45, C, W, dtype, seed=C, bias=C != 6))


@BOTH
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("L", [1, 2, 3, 4, 8, 11, 12, 64, 130, 300, 1100])
def test_conv_bwd_lengths_of_sequences(L, silu, dtype):
    check_conv(*conv_inputs(2, L, 24, 4, dtype, seed=L), silu=silu)


@BOTH
def test_conv_bwd_without_states_and_bias(dtype):
    d, _, dy, _ = conv_inputs(2, 70, 16, 4, dtype, bias=False, state=False)
    check_conv(d, None, dy, None)
    dx, dw, db, ds = bd.mamba2_causal_conv_bwd(dy, d["x"], d["weight"], want_dinitial_state=False)
    assert db is None and ds is None


@BOTH
@pytest.mark.parametrize("W", [2, 4, 7])
def test_conv_bwd_ragged_batch(W, dtype):
    L = 150
    lengths = torch.tensor([0, 1, 2, 3, 5, 64, 75, 149, 150, 400, -3], dtype=torch.int32, device="cuda")
    d, init, dy, dfin = conv_inputs(len(lengths), L, 24, W, dtype)
    clean = {**{k: t.clone() for k, t in d.items()}, "dy": dy.clone()}
    for k, n in enumerate(lengths.clamp(0, L).tolist()):
        d["x"][k, n:], dy[k, n:] = NAN, INF
    outs = check_conv(d, init, dy, dfin, lengths=lengths, clean=clean)
    for k, n in enumerate(lengths.clamp(0, L).tolist()):
        assert bool((outs["dx"][k, n:] == 0).all())
    assert torch.equal(outs["dinitial_state"][0], dfin[0])


@BOTH
@pytest.mark.parametrize("shift", [0, 1, 2, 4])
def test_conv_bwd_slices(shift, dtype):
    b, L, C, W = 2, 90, 32, 4
    n = gen(9)
    wide, dwide = n(b, L, 3 * C).to(dtype).cuda(), n(b, L, 2 * C).to(dtype).cuda()
    x, dy = wide[..., shift:shift + C], dwide[..., shift:shift + C]
    weight = n(C, W).cuda()
    out = torch.full((b, L, 2 * C), NAN, dtype=dtype, device="cuda")
    bd.mamba2_causal_conv_bwd(dy, x, weight, dx=out[..., shift:shift + C])
    want = bd.mamba2_causal_conv_bwd(dy.contiguous(), x.contiguous(), weight)
    close(out[..., shift:shift + C], want[0].cpu(), TOL[dtype])
    assert torch.isnan(out[..., shift + C:]).all() and torch.isnan(out[..., :shift]).all()


def test_conv_bwd_gradient_against_differences():
    """As for the recurrence; without an activation the loss is linear in each."""
    d, init, dy, dfin = conv_inputs(2, 60, 16, 4, FP32, seed=3)
    dx, dw, db, ds = bd.mamba2_causal_conv_bwd(dy, **d, initial_state=init, dfinal_state=dfin)
    at = {**d, "initial_state": init}

    def loss(v):
        y, fin = bd.mamba2_causal_conv_fwd(v["x"], v["weight"], bias=v["bias"], initial_state=v["initial_state"])
        return (y.double() * dy).sum() + (fin.double() * dfin).sum()

    n, e = gen(4), 2.0 ** -7
    for name, g in {"x": dx, "weight": dw, "bias": db, "initial_state": ds}.items():
        way = n(*g.shape).cuda()
        slope = (loss({**at, name: at[name] + e * way}) - loss({**at, name: at[name] - e * way})).item() / (2 * e)
        want = (g.double() * way).sum().item()
        assert abs(slope - want) <= 1e-2 * ((g.double() * way).norm().item() + abs(want)), name


# ------------------------------------------------------------- block norm
DTYPES = pytest.mark.parametrize("dtype,rdtype", [(BF16, BF16), (BF16, FP32), (FP32, FP32)],
                                 ids=["bf16", "bf16_fp32", "fp32"])


def norm_inputs(rows, C, dtype, rdtype, seed=0, gated=True, post=True, pre=True, scale=True):
    n = gen(seed)
    w = lambda on: (1 + 0.1 * n(C)).cuda() if on else None  # noqa: E731
    return dict(x=n(rows, C).to(dtype).cuda(), z=n(rows, C).to(dtype).cuda() if gated else None, post_weight=w(post),
                scale=w(scale), pre_weight=w(pre)), (2 * n(rows, C)).to(rdtype).cuda(), \
        n(rows, C).to(rdtype).cuda(), n(rows, C).to(dtype).cuda()


def check_norm(d, residual, dr, dy, eps=1e-5, post=True, pre=True):
    rows, C = d["x"].shape
    dtype, rdtype = d["x"].dtype, dr.dtype
    out, y = Guarded((rows, C), rdtype), Guarded((rows, C), dtype)
    bd.mamba2_block_norm_fwd(**d, residual=residual, eps=eps, post=post, pre=pre, residual_out=out.t,
                             y=y.t if pre else None)
    assert out.intact() and y.intact()
    out_ref, y_ref = ref.block_norm(**f64s(d), residual=ref.f64(residual), eps=eps, post=post, pre=pre)
    close(out.t, out_ref, TOL[rdtype], name="residual_out")
    if pre:
        close(y.t, y_ref, TOL[dtype], name="y")
    dx, dz, dres = Guarded((rows, C), dtype), Guarded((rows, C), dtype), Guarded((rows, C), rdtype)
    got = bd.mamba2_block_norm_bwd(dr, dy if pre else None, residual_out=out.t if pre else None, **d, eps=eps, post=post,
                                   pre=pre, dx=dx.t, dz=dz.t if d["z"] is not None else None, dresidual=dres.t)
    assert dx.intact() and dz.intact() and dres.intact()
    want, size = ref.block_norm_grads(ref.f64(dr), ref.f64(dy), **f64s(d), out=ref.f64(out.t), eps=eps, post=post,
                                      pre=pre)
    for name, t in zip(("dx", "dz", "dresidual", "dpost_weight", "dscale", "dpre_weight"), got):
        if t is not None:
            close(t, want[name], TOL[t.dtype], size.get(name), name=name)
    return out.t, y.t, got


@DTYPES
@pytest.mark.parametrize("C", [1, 3, 8, 31, 64, 255, 256, 257, 520, 1000, 1024, 2049, 4096, 4097, 4104, 8192, 8200,
                               16384, 20000, 32768])
def test_block_norm_numbers_of_channels(C, dtype, rdtype):
    d, *rest = norm_inputs(5, C, dtype, rdtype, seed=C)
    check_norm(d, *rest)


@DTYPES
@pytest.mark.parametrize("rows,C", [(1, 4096), (2, 40), (37, 1000), (700, 512), (5000, 72), (1300, 4096), (400, 5000),
                                    (3000, 33)])
def test_block_norm_numbers_of_rows(rows, C, dtype, rdtype):
    d, *rest = norm_inputs(rows, C, dtype, rdtype, seed=rows)
    check_norm(d, *rest)


@DTYPES
@pytest.mark.parametrize("rows,C", [(400, 8200), (260, 16400)])
def test_block_norm_rows_of_clusters_captured_and_replayed(rows, C, dtype, rdtype):
    """More rows than clusters at once, each with many exchanges; a replay gives what the calls gave, bit for bit."""
    d, res, dr, dy = norm_inputs(rows, C, dtype, rdtype, seed=C)
    out, y, got = check_norm(d, res, dr, dy)
    names = ("residual_out", "y", "dx", "dz", "dresidual", "dpost_weight", "dscale", "dpre_weight")
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        out2, y2 = bd.mamba2_block_norm_fwd(**d, residual=res)
        got2 = bd.mamba2_block_norm_bwd(dr, dy, residual_out=out2, **d)
    graph.replay()
    torch.cuda.synchronize()
    for name, a, b in zip(names, (out2, y2, *got2), (out, y, *got)):
        assert torch.equal(a, b), name


@DTYPES
@pytest.mark.parametrize("C", [40, 1001, 4608])
@pytest.mark.parametrize("gated,post,pre,scale", [(a, b, c, s) for a in (0, 1) for b in (0, 1) for c in (0, 1)
                                                  for s in (0, 1)])
def test_block_norm_parts(gated, post, pre, scale, C, dtype, rdtype):
    d, *rest = norm_inputs(6, C, dtype, rdtype, gated=gated, post=post, pre=pre, scale=scale)
    check_norm(d, *rest, post=bool(post), pre=bool(pre))


@DTYPES
def test_block_norm_without_weights_and_residual(dtype, rdtype):
    d, _, dr, dy = norm_inputs(9, 200, dtype, rdtype, post=False, pre=False, scale=False)
    out, y, got = check_norm(d, None, dr, dy, eps=0.1)
    assert got[3] is None and got[4] is None and got[5] is None
    dx, dz, none, *_ = bd.mamba2_block_norm_bwd(None, dy, residual_out=out, **d, eps=0.1, want_dresidual=False)
    assert none is None
    want, size = ref.block_norm_grads(None, ref.f64(dy), **f64s(d), out=ref.f64(out), eps=0.1)
    close(dx, want["dx"], TOL[dtype], size["dx"]), close(dz, want["dz"], TOL[dtype])


@DTYPES
def test_block_norm_in_place(dtype, rdtype):
    d, res, dr, dy = norm_inputs(300, 1000, dtype, rdtype)
    out, y = bd.mamba2_block_norm_fwd(**d, residual=res)
    kept = res.clone()
    same, y2 = bd.mamba2_block_norm_fwd(**d, residual=kept, residual_out=kept)
    assert same is kept and torch.equal(kept, out) and torch.equal(y, y2)
    want = bd.mamba2_block_norm_bwd(dr, dy, residual_out=out, **d)
    kept = dr.clone()
    got = bd.mamba2_block_norm_bwd(kept, dy, residual_out=out, **d, dresidual=kept)
    assert got[2] is kept and all(torch.equal(a, c) for a, c in zip(got, want))


@BOTH
@pytest.mark.parametrize("shift", [0, 1, 8])
def test_block_norm_slices(shift, dtype):
    rows, C = 50, 264
    n = gen(11)
    wide = n(rows, 4 * C).to(dtype).cuda()
    x, z = wide[:, shift:shift + C], wide[:, 2 * C + shift:3 * C + shift]
    res, dy = n(rows, C).to(dtype).cuda(), n(rows, C).to(dtype).cuda()
    out, y = bd.mamba2_block_norm_fwd(x, res, z=z)
    flat = bd.mamba2_block_norm_fwd(x.contiguous(), res, z=z.contiguous())
    close(out, flat[0].cpu(), TOL[dtype]), close(y, flat[1].cpu(), TOL[dtype])
    grad = torch.full_like(wide, NAN)
    dx, dz = grad[:, shift:shift + C], grad[:, 2 * C + shift:3 * C + shift]
    bd.mamba2_block_norm_bwd(None, dy, x, out, z=z, dx=dx, dz=dz)
    want = bd.mamba2_block_norm_bwd(None, dy, x.contiguous(), out, z=z.contiguous())
    close(dx, want[0].cpu(), TOL[dtype]), close(dz, want[1].cpu(), TOL[dtype])
    assert torch.isnan(grad[:, C + shift:2 * C + shift]).all()


def test_block_norm_rows_that_are_zero_and_not_finite():
    """A zero row has the factor 1 / sqrt(eps); NaN and infinities stay in their row."""
    d, res, dr, dy = norm_inputs(6, 300, FP32, FP32, gated=False)
    d["x"][1], res[1] = 0, 0
    out, y, got = check_norm(d, res, dr, dy)
    d["x"][3, 7], d["x"][4, 9] = NAN, INF
    out2, y2 = bd.mamba2_block_norm_fwd(**d, residual=res)
    for k in (0, 1, 2, 5):
        assert torch.equal(out2[k], out[k]) and torch.equal(y2[k], y[k])
    assert torch.isnan(y2[3]).all() and torch.isnan(out2[4, 9])


def test_block_norm_gradient_against_differences():
    d, res, dr, dy = norm_inputs(7, 200, FP32, FP32, seed=5)
    out, y = bd.mamba2_block_norm_fwd(**d, residual=res)
    dx, dz, dres, d1, ds, d2 = bd.mamba2_block_norm_bwd(dr, dy, residual_out=out, **d)
    at = {**d, "residual": res}

    def loss(v):
        o, y = bd.mamba2_block_norm_fwd(**v)
        return (o.double() * dr).sum() + (y.double() * dy).sum()

    n, e = gen(4), 2.0 ** -7
    for name, g in {"x": dx, "z": dz, "residual": dres, "post_weight": d1, "scale": ds, "pre_weight": d2}.items():
        way = n(*g.shape).cuda()
        slope = (loss({**at, name: at[name] + e * way}) - loss({**at, name: at[name] - e * way})).item() / (2 * e)
        want = (g.double() * way).sum().item()
        assert abs(slope - want) <= 1e-2 * ((g.double() * way).norm().item() + abs(want)), name


# ------------------------------------------------------------ all of them
def test_gradients_are_the_same_every_time():
    """No sum's order depends on how blocks are scheduled."""
    d, h0 = glr_inputs(3, 700, 200, BF16, gated=True)
    dy = torch.ones_like(d["x"])
    _, _, cs = bd.mamba2_glr_fwd(**d, initial_state=h0, want_chunk_states=True)
    c = conv_inputs(3, 700, 200, 4, BF16)
    nrm = norm_inputs(2000, 512, BF16, FP32)
    runs = []
    for _ in range(4):
        runs.append([*bd.mamba2_glr_bwd(dy, **d, chunk_states=cs),
                     *bd.mamba2_causal_conv_bwd(c[2], **c[0], initial_state=c[1], dfinal_state=c[3]),
                     *bd.mamba2_block_norm_bwd(nrm[2], nrm[3], residual_out=nrm[1], **nrm[0])])
    for other in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], other))


def test_captured_and_replayed_on_new_inputs_on_another_stream():
    """A training step's calls in a graph: replayed on new inputs they give what eager calls give."""
    b, L, C = 2, 200, 128
    d, h0 = glr_inputs(b, L, C, BF16, gated=True)
    weight = torch.randn(C, 4, device="cuda")
    w = torch.rand(C, device="cuda")
    res, dy = torch.randn(b, L, C, device="cuda").to(BF16), torch.randn(b, L, C, device="cuda").to(BF16)

    def step(v):
        x, _ = bd.mamba2_causal_conv_fwd(v["x"], weight)
        y, fin, cs = bd.mamba2_glr_fwd(x, v["r"], v["i"], v["A"], z=v["z"], initial_state=h0, want_chunk_states=True)
        out, n = bd.mamba2_block_norm_fwd(y, res, post_weight=w, scale=w, pre_weight=w)
        gy, _, gres, *gw = bd.mamba2_block_norm_bwd(None, dy, y, out, post_weight=w, scale=w, pre_weight=w)
        gx, gr, gi, gz, gA, gh = bd.mamba2_glr_bwd(gy, x, v["r"], v["i"], v["A"], cs, z=v["z"])
        gx, gweight, _, _ = bd.mamba2_causal_conv_bwd(gx, v["x"], weight)
        return n, fin, gx, gr, gi, gz, gA, gh, gweight, gres, *gw

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step(d)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            got = step(d)
    torch.cuda.current_stream().wait_stream(stream)
    for seed in (5, 6):
        new, _ = glr_inputs(b, L, C, BF16, gated=True, seed=seed)
        for k, t in new.items():
            d[k].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(got, step(new)))


def test_empty_calls():
    e = lambda *s, dt=BF16: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    A, h0 = -torch.ones(8, device="cuda"), torch.randn(2, 8, device="cuda")
    y, fin, cs = bd.mamba2_glr_fwd(e(2, 0, 8), e(2, 0, 8), e(2, 0, 8), A, initial_state=h0, want_chunk_states=True)
    assert torch.equal(fin, h0) and cs.shape == (2, 0, 8)
    *_, dA, dh = bd.mamba2_glr_bwd(y, e(2, 0, 8), e(2, 0, 8), e(2, 0, 8), A, cs, dfinal_state=h0)
    assert torch.equal(dh, h0) and bool((dA == 0).all())
    y, fin, cs = bd.mamba2_glr_fwd(e(0, 5, 8), e(0, 5, 8), e(0, 5, 8), A)
    assert y.shape == (0, 5, 8)
    ds = torch.randn(2, 3, 8, device="cuda").to(BF16)
    dx, dw, db, di = bd.mamba2_causal_conv_bwd(e(2, 0, 8), e(2, 0, 8), torch.ones(8, 4, device="cuda"), dfinal_state=ds)
    assert torch.equal(di, ds) and bool((dw == 0).all())
    out, y = bd.mamba2_block_norm_fwd(e(0, 8), e(0, 8))
    assert out.shape == y.shape == (0, 8)
    w = torch.ones(8, device="cuda")
    *_, d1, dsc, d2 = bd.mamba2_block_norm_bwd(e(0, 8), e(0, 8), e(0, 8), e(0, 8), post_weight=w, scale=w, pre_weight=w)
    assert all(bool((t == 0).all()) for t in (d1, dsc, d2))
