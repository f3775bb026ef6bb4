"""CPU checks of the recurrent block's entry points: what the header declares is
exported and bound, and bad arguments are refused on the host (fake pointers,
never dereferenced: each call fails its checks first).  The fp64 forms that the
GPU tests compare with are pinned by hand-worked values, by differentiating them
and by planted mistakes."""
import ctypes
import math

import pytest
import torch

import gated_linear_ref as ref
from mamba_chunked_ssd_gb300 import binding as bd

OK, INVALID, UNSUPPORTED = 0, 1, 2
NAMES = ["mamba2_block_norm_bwd", "mamba2_block_norm_bwd_workspace_size", "mamba2_block_norm_fwd",
         "mamba2_causal_conv_bwd", "mamba2_causal_conv_bwd_workspace_size", "mamba2_glr_bwd",
         "mamba2_glr_bwd_workspace_size", "mamba2_glr_fwd", "mamba2_glr_step"]


@pytest.fixture(scope="module")
def lib():
    from mamba_chunked_ssd_gb300 import build_lib
    build_lib.build()
    return bd.load_library()


def test_exports_every_declared_function(lib):
    assert bd.header_functions(bd.HEADER_GATED_LINEAR) == NAMES
    for n in NAMES:
        assert hasattr(lib, n)
        assert n.endswith("workspace_size") or callable(getattr(bd, n))


def _p(i, off=0):
    """A fake pointer: apart from every other one, 16-byte aligned but for `off`."""
    return ctypes.c_void_p((i << 36) + off) if i else None


def call(lib, name, shape, order, ptr, defaults, before=(), after=()):
    a = {**defaults, **(ptr or {})}
    return getattr(lib, name)(ctypes.byref(shape), *before, *[a[n] for n in order], *after, None)


GLR = dict(batch=2, seqlen=100, channels=64, x_stride=0, r_stride=0, i_stride=0, z_stride=0, y_stride=0, dtype=1,
           flags=0)


def glr_fwd(lib, ptr=None, **kw):
    order = "x r i z A lengths init y chunks fin".split()
    return call(lib, "mamba2_glr_fwd", bd.mamba2_glr_shape(**{**GLR, **kw}), order + [], ptr,
                {n: _p(k + 1) for k, n in enumerate(order)})


def glr_step(lib, ptr=None, **kw):
    order = "x r i z A init fin y".split()
    return call(lib, "mamba2_glr_step", bd.mamba2_glr_shape(**{**GLR, "seqlen": 1, **kw}), order, ptr,
                {n: _p(k + 1) for k, n in enumerate(order)})


def glr_bwd(lib, ptr=None, grads=None, bytes_=1 << 40, **kw):
    order = "dy x r i z A lengths chunks dfin dx dr di dz dA dinit ws".split()
    g = bd.mamba2_glr_grad_strides(**{**dict(dx_stride=0, dr_stride=0, di_stride=0, dz_stride=0), **(grads or {})})
    return call(lib, "mamba2_glr_bwd", bd.mamba2_glr_shape(**{**GLR, **kw}), order, ptr,
                {n: _p(k + 1) for k, n in enumerate(order)}, before=(ctypes.byref(g),), after=(bytes_,))


@pytest.mark.parametrize("f", [glr_fwd, glr_step, glr_bwd])
@pytest.mark.parametrize("kw,code", [
    (dict(ptr=dict(x=None)), INVALID), (dict(ptr=dict(r=None)), INVALID), (dict(ptr=dict(i=None)), INVALID),
    (dict(ptr=dict(A=None)), INVALID), (dict(ptr=dict(A=_p(30, 4))), INVALID),
    (dict(ptr=dict(x=_p(30, 1))), INVALID),
    (dict(dtype=2), INVALID), (dict(flags=1), INVALID), (dict(batch=-1), INVALID), (dict(channels=0), INVALID),
    (dict(x_stride=63), INVALID), (dict(y_stride=-64), INVALID), (dict(r_stride=1 << 40), UNSUPPORTED),
    (dict(batch=65536), UNSUPPORTED), (dict(channels=(1 << 30) + 1), UNSUPPORTED),
    (dict(batch=9, channels=1 << 30), UNSUPPORTED),
])
def test_glr_refusals(lib, f, kw, code):
    assert f(lib, **kw) == code


@pytest.mark.parametrize("f", [glr_fwd, glr_step])
def test_glr_outputs_over_inputs_are_refused(lib, f):
    assert f(lib, ptr=dict(y=_p(1))) == INVALID        # over x
    assert f(lib, ptr=dict(y=_p(1, 128))) == INVALID
    assert f(lib, ptr=dict(fin=_p(20, 128), y=_p(20))) == INVALID
    assert f(lib, ptr=dict(y=None)) == INVALID


def test_glr_more_refusals(lib):
    assert glr_step(lib, seqlen=2) == INVALID
    assert glr_step(lib, ptr=dict(fin=None)) == INVALID            # the step writes its state
    assert glr_step(lib, ptr=dict(fin=_p(6, 16))) == INVALID       # partly over the state that is read
    assert glr_fwd(lib, ptr=dict(fin=_p(7))) == INVALID            # whole sequences: not in place
    assert glr_fwd(lib, ptr=dict(lengths=_p(30, 2))) == INVALID
    assert glr_fwd(lib, ptr=dict(chunks=_p(30, 8))) == INVALID
    assert glr_fwd(lib, seqlen=(1 << 30) + 1) == UNSUPPORTED
    assert glr_fwd(lib, batch=4096, seqlen=1 << 20, channels=1 << 20) == UNSUPPORTED
    assert glr_fwd(lib, batch=0) == OK
    assert glr_step(lib, batch=0, ptr=dict(x=None, r=None, i=None, y=None)) == OK
    assert lib.mamba2_glr_fwd(None, *[_p(k) for k in range(1, 11)], None) == INVALID


def test_glr_bwd_more_refusals(lib):
    assert glr_bwd(lib, ptr=dict(dy=None)) == INVALID
    assert glr_bwd(lib, ptr=dict(chunks=None)) == INVALID
    assert glr_bwd(lib, ptr=dict(dA=None)) == INVALID
    assert glr_bwd(lib, ptr=dict(dz=None)) == INVALID              # z without its gradient
    assert glr_bwd(lib, ptr=dict(z=None)) == INVALID               # a gradient without z
    assert glr_bwd(lib, ptr=dict(dx=_p(1))) == INVALID             # over dy
    assert glr_bwd(lib, ptr=dict(dr=_p(10))) == INVALID            # over dx
    assert glr_bwd(lib, ptr=dict(dinit=_p(9))) == INVALID          # over dfinal_state
    assert glr_bwd(lib, ptr=dict(ws=None)) == INVALID
    assert glr_bwd(lib, ptr=dict(ws=_p(40, 128))) == INVALID
    shape = bd.mamba2_glr_shape(**GLR)
    need = lib.mamba2_glr_bwd_workspace_size(ctypes.byref(shape))
    assert need >= 2 * 64 * 4 and need % 256 == 0
    assert glr_bwd(lib, bytes_=need - 1) == INVALID
    assert glr_bwd(lib, grads=dict(dx_stride=63)) == INVALID
    assert lib.mamba2_glr_bwd_workspace_size(ctypes.byref(bd.mamba2_glr_shape(**{**GLR, "dtype": 7}))) == 0
    assert lib.mamba2_glr_bwd_workspace_size(None) == 0


def test_slices_side_by_side_do_not_overlap(lib):
    """dx, dr, di in one tensor of rows of 192 channels: refused only where they share elements
    (a refusal for the workspace comes after that for the overlap would)."""
    wide = dict(dx_stride=192, dr_stride=192, di_stride=192)
    side = dict(dx=_p(50), dr=_p(50, 128), di=_p(50, 256), z=None, dz=None)
    shape = bd.mamba2_glr_shape(**{**GLR, "batch": 0})
    need = lib.mamba2_glr_bwd_workspace_size(ctypes.byref(shape))
    assert need == 0
    assert glr_bwd(lib, ptr={**side, "dr": _p(50, 126)}, grads=wide) == INVALID
    assert glr_bwd(lib, ptr={**side, "di": _p(50, 258)}, grads=wide) == INVALID   # its end is over the next row's dx
    assert glr_bwd(lib, ptr={**side, "dr": _p(50, 384 * 3 + 130)}, grads={**wide, "dr_stride": 191}) == INVALID


CONV = dict(batch=2, seqlen=90, channels=64, width=4, x_stride=0, y_stride=0, dtype=1, flags=1)


def conv_bwd(lib, ptr=None, dx_stride=0, bytes_=1 << 40, **kw):
    order = "dy x weight bias lengths init dfin dx dw db dinit ws".split()
    return call(lib, "mamba2_causal_conv_bwd", bd.mamba2_conv_shape(**{**CONV, **kw}), order, ptr,
                {n: _p(k + 1) for k, n in enumerate(order)}, before=(dx_stride,), after=(bytes_,))


@pytest.mark.parametrize("kw,code", [
    (dict(ptr=dict(dy=None)), INVALID), (dict(ptr=dict(x=None)), INVALID), (dict(ptr=dict(weight=None)), INVALID),
    (dict(ptr=dict(dw=None)), INVALID), (dict(ptr=dict(dx=None)), INVALID), (dict(ptr=dict(dx=_p(1))), INVALID),
    (dict(ptr=dict(dx=_p(2, 64))), INVALID), (dict(ptr=dict(dinit=_p(7))), INVALID),
    (dict(ptr=dict(dw=_p(30, 8))), INVALID), (dict(ptr=dict(ws=None)), INVALID), (dict(bytes_=16), INVALID),
    (dict(dx_stride=63), INVALID), (dict(y_stride=5), INVALID), (dict(flags=2), INVALID), (dict(width=1), INVALID),
    (dict(width=9), UNSUPPORTED), (dict(dtype=9), INVALID), (dict(batch=65536), UNSUPPORTED),
    (dict(dx_stride=1 << 40), UNSUPPORTED),
])
def test_conv_bwd_refusals(lib, kw, code):
    assert conv_bwd(lib, **kw) == code


NORM = dict(rows=20, channels=64, x_stride=0, z_stride=0, residual_stride=0, residual_out_stride=0, y_stride=0,
            eps=1e-5, dtype=1, residual_dtype=0, flags=3)


def norm_fwd(lib, ptr=None, **kw):
    order = "x z residual w1 scale w2 out y".split()
    return call(lib, "mamba2_block_norm_fwd", bd.mamba2_block_norm_shape(**{**NORM, **kw}), order, ptr,
                {n: _p(k + 1) for k, n in enumerate(order)})


def norm_bwd(lib, ptr=None, grads=None, bytes_=1 << 40, **kw):
    order = "dout y x z out w1 scale w2 dx dz dres d1 ds d2 ws".split()
    g = bd.mamba2_block_norm_grad_strides(**{**dict(dx_stride=0, dz_stride=0, dresidual_out_stride=0,
                                                    dresidual_stride=0), **(grads or {})})
    return call(lib, "mamba2_block_norm_bwd", bd.mamba2_block_norm_shape(**{**NORM, **kw}), order, ptr,
                {n: _p(k + 1) for k, n in enumerate(order)}, before=(ctypes.byref(g),), after=(bytes_,))


@pytest.mark.parametrize("f", [norm_fwd, norm_bwd])
@pytest.mark.parametrize("kw,code", [
    (dict(ptr=dict(x=None)), INVALID), (dict(ptr=dict(out=None)), INVALID), (dict(ptr=dict(y=None)), INVALID),
    (dict(flags=1), INVALID),                          # y (dy) and pre_weight without the norm before
    (dict(flags=2), INVALID),                          # post_weight without the norm after
    (dict(flags=4), INVALID), (dict(ptr=dict(w1=_p(30, 8))), INVALID), (dict(ptr=dict(x=_p(30, 1))), INVALID),
    (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(dtype=3), INVALID),
    (dict(residual_dtype=3), INVALID), (dict(dtype=0, residual_dtype=1), UNSUPPORTED), (dict(rows=-1), INVALID),
    (dict(channels=0), INVALID), (dict(channels=32769), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED),
    (dict(z_stride=63), INVALID), (dict(x_stride=1 << 40), UNSUPPORTED),
])
def test_block_norm_refusals(lib, f, kw, code):
    assert f(lib, **kw) == code


def test_block_norm_more_refusals(lib):
    assert norm_fwd(lib, ptr=dict(y=_p(1))) == INVALID
    assert norm_fwd(lib, ptr=dict(out=_p(3, 256))) == INVALID                  # partly over the residual
    assert norm_fwd(lib, ptr=dict(out=_p(3)), residual_stride=128) == INVALID  # in place needs one stride
    assert norm_fwd(lib, rows=0) == OK
    assert norm_bwd(lib, ptr=dict(dz=None)) == INVALID
    assert norm_bwd(lib, ptr=dict(z=None)) == INVALID
    assert norm_bwd(lib, ptr=dict(dx=_p(3))) == INVALID
    assert norm_bwd(lib, ptr=dict(dres=_p(5))) == INVALID                      # over the sum that is read
    assert norm_bwd(lib, ptr=dict(ds=_p(12))) == INVALID                       # over another gradient
    assert norm_bwd(lib, bytes_=8) == INVALID
    assert norm_bwd(lib, grads=dict(dx_stride=1)) == INVALID


# -------------------------------------------- what the binding hands over
from test_gated_delta_binding import Gpu, Recorder  # noqa: E402


@pytest.fixture
def rec(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(bd, "load_library", lambda: r)
    monkeypatch.setattr(bd, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(bd, "_current_gpu", lambda: 0, raising=False)
    monkeypatch.setattr(bd, "_workspace_sizes", {})
    return r


def tensors(specs, device, drop):
    return {n: Gpu(*s, device=(device or {}).get(n, 0)) for n, s in specs.items() if n not in drop}


def b_glr_fwd(device=None, drop=(), **kw):
    q = (2, 100, 8)
    return bd.mamba2_glr_fwd(**tensors(dict(x=q, r=q, i=q, A=(8,), z=q, initial_state=(2, 8), y=q, final_state=(2, 8),
                                            chunk_states=(2, 2, 8)), device, drop), **kw)


def b_glr_bwd(device=None, drop=(), **kw):
    q = (2, 100, 8)
    return bd.mamba2_glr_bwd(**tensors(dict(dy=q, x=q, r=q, i=q, A=(8,), chunk_states=(2, 2, 8), z=q, dfinal_state=(2, 8),
                                            dx=q, dr=q, di=q, dz=q, dA=(8,), dinitial_state=(2, 8)), device, drop), **kw)


def b_glr_step(device=None, drop=(), **kw):
    q = (2, 8)
    return bd.mamba2_glr_step(**tensors(dict(x=q, r=q, i=q, A=(8,), z=q, state_in=q, state_out=q, y=q), device, drop), **kw)


def b_conv_bwd(device=None, drop=(), **kw):
    q, s = (2, 9, 8), (2, 3, 8)
    return bd.mamba2_causal_conv_bwd(**tensors(dict(dy=q, x=q, weight=(8, 4), bias=(8,), initial_state=s, dfinal_state=s,
                                                    dx=q, dweight=(8, 4), dbias=(8,), dinitial_state=s), device, drop), **kw)


def b_norm_fwd(device=None, drop=(), **kw):
    q, w = (5, 8), (8,)
    return bd.mamba2_block_norm_fwd(**tensors(dict(x=q, residual=q, z=q, post_weight=w, scale=w, pre_weight=w,
                                                   residual_out=q, y=q), device, drop), **kw)


def b_norm_bwd(device=None, drop=(), **kw):
    q, w = (5, 8), (8,)
    return bd.mamba2_block_norm_bwd(**tensors(dict(dresidual_out=q, dy=q, x=q, residual_out=q, z=q, post_weight=w, scale=w,
                                                   pre_weight=w, dx=q, dz=q, dresidual=q), device, drop), **kw)


BOUND = {"glr_fwd": (b_glr_fwd, "x r i A z initial_state y final_state chunk_states"),
         "glr_bwd": (b_glr_bwd, "dy x r i A chunk_states z dfinal_state dx dr di dz dA dinitial_state"),
         "glr_step": (b_glr_step, "x r i A z state_in state_out y"),
         "conv_bwd": (b_conv_bwd, "dy x weight bias initial_state dfinal_state dx dweight dbias dinitial_state"),
         "norm_fwd": (b_norm_fwd, "x residual z post_weight scale pre_weight residual_out y"),
         "norm_bwd": (b_norm_bwd, "dresidual_out dy x residual_out z post_weight scale pre_weight dx dz dresidual")}


def launches(rec):
    return [c for c in rec.calls if not c[0].endswith("workspace_size")]


@pytest.fixture
def no_memory(monkeypatch):
    """torch.empty as a stand-in for GPU memory, with the stream it was made under."""
    under, made = [], []

    class Under:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            under.append(self.stream)

        def __exit__(self, *a):
            under.pop()

    def empty(*shape, dtype=None, device=None):
        made.append(under[-1] if under else None)
        return Gpu(*shape[0] if len(shape) == 1 and not isinstance(shape[0], int) else shape, dtype=dtype)

    monkeypatch.setattr(torch.cuda, "stream", Under)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch, "empty_like", lambda t, memory_format=None: empty(t.shape, dtype=t.dtype))
    return made


@pytest.mark.parametrize("bound,names", BOUND.values(), ids=BOUND)
def test_tensors_on_another_gpu_are_refused(rec, no_memory, bound, names):
    bound()
    assert len(launches(rec)) == 1
    for name in names.split():
        with pytest.raises(ValueError, match="cuda:"):
            bound(device={name: 1})
    with pytest.raises(ValueError, match="current device"):
        bound(device=dict.fromkeys(names.split(), 1))
    assert len(launches(rec)) == 1


@pytest.mark.parametrize("bound,names", BOUND.values(), ids=BOUND)
def test_outputs_and_workspaces_come_from_the_stream_of_the_call(rec, no_memory, bound, names):
    class Stream:
        cuda_stream, device = 7, torch.device("cuda", 0)

    stream = Stream()
    outputs = "y final_state state_out dx dr di dz dA dinitial_state dweight dbias residual_out dresidual".split()
    drop = [n for n in outputs if n in names.split() and not (bound is b_norm_bwd and n == "residual_out")]
    bound(stream=stream, drop=drop)
    assert no_memory and all(s is stream for s in no_memory)
    assert launches(rec)[0][1][-1] == 7
    count = len(no_memory)
    bound(drop=drop)
    assert no_memory[count:] == [None] * count
    Stream.device = torch.device("cuda", 1)
    with pytest.raises(ValueError, match="stream"):
        bound(stream=Stream())


def test_binding_refuses_wrong_calls(rec, no_memory):
    q = lambda *s, **k: Gpu(*s, **k)  # noqa: E731
    x = q(2, 5, 8)
    A = q(8)
    with pytest.raises(ValueError, match="dimensions"):
        bd.mamba2_glr_fwd(q(5, 8), q(5, 8), q(5, 8), A)
    with pytest.raises(ValueError, match="dimensions"):
        bd.mamba2_glr_step(x, x, x, A)
    with pytest.raises(ValueError):
        bd.mamba2_glr_fwd(x, q(2, 5, 4), x, A)
    with pytest.raises(ValueError):
        bd.mamba2_glr_fwd(x, x, x, q(4))
    with pytest.raises(ValueError):
        bd.mamba2_glr_fwd(x, q(2, 5, 8, dtype=torch.bfloat16), x, A)
    with pytest.raises(ValueError, match="lengths"):
        bd.mamba2_glr_fwd(x, x, x, A, lengths=q(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="chunk_states"):
        bd.mamba2_glr_bwd(x, x, x, x, A, None)
    with pytest.raises(ValueError, match="chunk_states"):
        bd.mamba2_glr_bwd(x, x, x, x, A, q(2, 2, 8))
    with pytest.raises(ValueError, match="dz"):
        bd.mamba2_glr_bwd(x, x, x, x, A, q(2, 1, 8), dz=x)
    with pytest.raises(TypeError):
        h = q(2, 5, 8, dtype=torch.float16)
        bd.mamba2_glr_fwd(h, h, h, A)
    with pytest.raises(ValueError):
        bd.mamba2_causal_conv_bwd(q(2, 4, 8), x, q(8, 4))
    with pytest.raises(ValueError, match="y comes"):
        bd.mamba2_block_norm_fwd(x, pre=False, y=x)
    with pytest.raises(ValueError):
        bd.mamba2_block_norm_fwd(x, q(2, 5, 8, dtype=torch.bfloat16), residual_out=q(2, 5, 8))
    with pytest.raises(ValueError, match="dy and"):
        bd.mamba2_block_norm_bwd(x, None, x, x)
    with pytest.raises(ValueError, match="dy and"):
        bd.mamba2_block_norm_bwd(x, x, x, pre=False)
    with pytest.raises(ValueError, match="workspace"):
        monkey = q(1, dtype=torch.uint8)
        rec.mamba2_glr_bwd_workspace_size = lambda s: 1000
        bd._workspace_sizes.clear()
        bd.mamba2_glr_bwd(x, x, x, x, A, q(2, 1, 8), workspace=monkey)
    with pytest.raises(ValueError, match="CUDA"):
        bd.mamba2_glr_fwd(torch.zeros(2, 5, 8), torch.zeros(2, 5, 8), torch.zeros(2, 5, 8), torch.zeros(8))
    assert launches(rec) == []


def test_an_eps_that_is_a_tensor_counts_by_its_value(rec, no_memory):
    eps, x = torch.tensor(0.5), Gpu(6, 8)
    for value in (0.5, 0.25):
        eps.fill_(value)
        bd.mamba2_block_norm_fwd(x, eps=eps)
    assert [args[0].eps for _, args in launches(rec)] == [0.5, 0.25]


# --------------------------------------------------- the fp64 forms themselves
def n64(seed):
    r = torch.Generator().manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=r, dtype=torch.float64)


def leaves(*ts):
    return [t.clone().requires_grad_() for t in ts]


def test_reference_recurrence_on_hand_worked_values():
    """a = 1/2 at both tokens: h = h0 / 2 + sqrt(3/4) x / 2, twice; a gate of 0 adds nothing."""
    one = torch.zeros(1, 2, 1, dtype=torch.float64)
    x = torch.tensor([[[4.0], [8.0]]], dtype=torch.float64)
    A = torch.tensor([2 * math.log(0.5)], dtype=torch.float64)
    y, fin, _ = ref.glr(x, one, one, A, init=torch.tensor([[6.0]], dtype=torch.float64))
    s = 0.75 ** 0.5
    h1 = 3 + s * 2
    assert torch.allclose(y[0, :, 0], torch.tensor([h1, h1 / 2 + s * 4], dtype=torch.float64))
    y, fin, _ = ref.glr(x, one, one - math.inf, A, init=torch.tensor([[6.0]], dtype=torch.float64), lengths=[1])
    assert y[0, :, 0].tolist() == [3.0, 0.0] and fin.item() == 3.0


def test_gradient_formulas_are_those_of_the_forms():
    n = n64(0)
    b, L, C = 3, 9, 5
    args = leaves(n(b, L, C), n(b, L, C), n(b, L, C), -n(C).abs(), n(b, L, C), n(b, C))
    dy, df, lens = n(b, L, C), n(b, C), [9, 4, 0]
    y, f, _ = ref.glr(*args, lengths=lens)
    auto = torch.autograd.grad((y * dy).sum() + (f * df).sum(), args)
    x, r, i, A, z, h0 = (t.detach() for t in args)
    want, _ = ref.glr_grads(dy, x, r, i, A, z, h0, lens, df)
    for g, k in zip(auto, ("dx", "dr", "di", "dA", "dz", "dinit")):
        assert torch.allclose(g, want[k], rtol=1e-11, atol=1e-12), k
    args = leaves(n(b, L, C), n(C, 4), n(C), n(b, 3, C))
    y, f = ref.conv(args[0], args[1], args[2], True, args[3], lens)
    df = n(b, 3, C)
    auto = torch.autograd.grad((y * dy).sum() + (f * df).sum(), args)
    x, w, bias, h0 = (t.detach() for t in args)
    want, _ = ref.conv_grads(dy, x, w, bias, True, h0, lens, df)
    for g, k in zip(auto, ("dx", "dweight", "dbias", "dinit")):
        assert torch.allclose(g, want[k], rtol=1e-11, atol=1e-12), k
    args = leaves(n(4, C), n(4, C), n(4, C), n(C), n(C), n(C))
    out, y = ref.block_norm(*args)
    dr, dy = n(4, C), n(4, C)
    auto = torch.autograd.grad((out * dr).sum() + (y * dy).sum(), args)
    x, res, z, w1, s, w2 = (t.detach() for t in args)
    want, _ = ref.block_norm_grads(dr, dy, x, out.detach(), z, w1, s, w2)
    for g, k in zip(auto, ("dx", "dresidual", "dz", "dpost_weight", "dscale", "dpre_weight")):
        assert torch.allclose(g, want[k], rtol=1e-11, atol=1e-12), k


def test_forms_against_differences():
    n = n64(1)
    x, r, i, z, h0 = leaves(*(n(1, 4, 3) for _ in range(4)), n(1, 3))
    A = (-n(3).abs()).requires_grad_()
    assert torch.autograd.gradcheck(lambda *a: ref.glr(*a)[:2], (x, r, i, A, z, h0))
    assert torch.autograd.gradcheck(lambda *a: ref.conv(*a), (x, *leaves(n(3, 2), n(3))))
    assert torch.autograd.gradcheck(lambda *a: ref.block_norm(*a), leaves(*(n(2, 3) for _ in range(3)), n(3), n(3), n(3)))


@pytest.mark.parametrize("mistake", ["gate_decays_later", "no_scale_of_inputs", "row_end", "gradient_without_decay_path"])
def test_planted_mistakes_show(mistake):
    n = n64(2)
    x, r, i, A, h0 = n(2, 12, 4), n(2, 12, 4), n(2, 12, 4), -n(4).abs(), n(2, 4)
    y, h, hs = ref.glr(x, r, i, A, init=h0, lengths=[12, 7])
    if mistake == "gate_decays_later":
        y2, h2, _ = ref.glr(x, r.roll(1, 1), i, A, init=h0, lengths=[12, 7])
    elif mistake == "no_scale_of_inputs":
        y2, h2, _ = ref.glr(x / torch.sqrt(-torch.expm1(2 * A * torch.sigmoid(r))), r, i, A, init=h0, lengths=[12, 7])
    elif mistake == "row_end":
        y2, h2, _ = ref.glr(x, r, i, A, init=h0, lengths=[12, 8])
    else:
        dy = n(2, 12, 4)
        g, _ = ref.glr_grads(dy, x, r, i, A, init=h0)
        x2, r2 = leaves(x, r)
        s = torch.sqrt(-torch.expm1(2 * A * torch.sigmoid(r2))).detach()   # as if s did not depend on r
        a, h2, out = torch.exp(A * torch.sigmoid(r2)), h0, 0
        for t in range(12):
            h2 = a[:, t] * h2 + s[:, t] * torch.sigmoid(i[:, t]) * x2[:, t]
            out = out + (h2 * dy[:, t]).sum()
        assert (torch.autograd.grad(out, r2)[0] - g["dr"]).abs().max() > 1e-2
        return
    assert (y - y2).abs().max() > 1e-2 and (h - h2).abs().max() > 1e-3
