"""CPU checks of the gated-delta-rule entry points: what the header declares is
exported and bound, and bad arguments are refused on the host (fake pointers,
never dereferenced: each call fails its checks first).  The fp64 forms that the
GPU tests compare with are pinned by exact cases and by planted mistakes."""
import ctypes

import numpy as np
import pytest
import torch

import gated_delta_ref as ref
from mamba_chunked_ssd_gb300 import binding as bd

OK, INVALID, UNSUPPORTED = 0, 1, 2
NAMES = ["mamba2_causal_conv_fwd", "mamba2_causal_conv_step", "mamba2_gdr_fwd", "mamba2_gdr_step",
         "mamba2_group_norm"]


@pytest.fixture(scope="module")
def lib():
    from mamba_chunked_ssd_gb300 import build_lib
    build_lib.build()
    return bd.load_library()


def test_exports_every_declared_function(lib):
    assert bd.header_functions(bd.HEADER_GATED_DELTA) == NAMES
    for n in NAMES:
        assert hasattr(lib, n) and callable(getattr(bd, n))


def _p(i):
    """A fake pointer: apart from every other one, 16-byte aligned."""
    return ctypes.c_void_p(i << 32) if i else None


def _gdr(lib, step=False, ptr=None, opt=None, **kw):
    d = dict(batch=2, seqlen=1 if step else 40, nheads=4, headdim=64, dstate=128, ngroups=2, chunk_size=64,
             dtype_code=1)
    d.update(kw)
    shape = bd.make_shape(**d)
    o = dict(q_stride=0, k_stride=0, v_stride=0, scale=0.1, l2_eps=1e-6, flags=1, reserved=0)
    o.update(opt or {})
    args = dict(q=_p(1), k=_p(2), v=_p(3), g=_p(4), beta=_p(5), lengths=None, init=_p(6), y=_p(7), out=_p(8))
    args.update(ptr or {})
    a = [ctypes.byref(shape), ctypes.byref(bd.mamba2_gdr_options(**o))] + [args[n] for n in ("q", "k", "v", "g", "beta")]
    if step:
        return lib.mamba2_gdr_step(*a, args["init"], args["out"], args["y"], None)
    return lib.mamba2_gdr_fwd(*a, args["lengths"], args["init"], args["y"], args["out"], None)


def off(i, n):
    return ctypes.c_void_p((i << 32) + n)


@pytest.mark.parametrize("step", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(ptr=dict(q=None)), INVALID),
    (dict(ptr=dict(beta=None)), INVALID),
    (dict(ptr=dict(y=None)), INVALID),
    (dict(ptr=dict(g=off(4, 4))), INVALID),
    (dict(ptr=dict(k=off(2, 1))), INVALID),             # not aligned to an element
    (dict(ptr=dict(y=_p(3))), INVALID),                 # y over v
    (dict(ptr=dict(y=off(6, 64))), INVALID),            # y over the state that is read
    (dict(ptr=dict(out=off(6, 64))), INVALID),          # states partly over one another
    (dict(opt=dict(flags=2)), INVALID),
    (dict(opt=dict(reserved=1)), INVALID),
    (dict(opt=dict(l2_eps=0.0)), INVALID),
    (dict(opt=dict(l2_eps=float("nan"))), INVALID),
    (dict(opt=dict(q_stride=255)), INVALID),            # narrower than G * S
    (dict(opt=dict(v_stride=-8)), INVALID),
    (dict(opt=dict(k_stride=1 << 40)), UNSUPPORTED),
    (dict(nheads=3), INVALID),
    (dict(dtype_code=2), INVALID),
    (dict(headdim=257), UNSUPPORTED),
    (dict(dstate=257), UNSUPPORTED),
    (dict(batch=65536), UNSUPPORTED),
])
def test_gdr_refusals(lib, step, kw, code):
    assert _gdr(lib, step=step, **kw) == code


def test_gdr_more_refusals(lib):
    assert _gdr(lib, step=True, seqlen=2) == INVALID
    assert _gdr(lib, step=True, ptr=dict(out=None)) == INVALID      # the step writes its state
    assert _gdr(lib, ptr=dict(out=_p(6))) == INVALID                # whole sequences: not in place
    assert _gdr(lib, ptr=dict(lengths=off(9, 2))) == INVALID
    assert _gdr(lib, batch=0) == OK                                 # nothing to do
    assert _gdr(lib, step=True, batch=0, ptr=dict(q=None, k=None, v=None)) == OK
    s = bd.make_shape(1, 1, 1, 8, 8, 1, 1, 1)
    assert lib.mamba2_gdr_fwd(ctypes.byref(s), None, *[_p(i) for i in range(1, 10)], None) == INVALID


def _conv(lib, step=False, ptr=None, **kw):
    d = dict(batch=2, seqlen=1 if step else 9, channels=64, width=4, x_stride=0, y_stride=0, dtype=1, flags=1)
    d.update(kw)
    a = dict(x=_p(1), weight=_p(2), bias=_p(3), init=_p(4), y=_p(5), out=_p(6))
    a.update(ptr or {})
    s = ctypes.byref(bd.mamba2_conv_shape(**d))
    if step:
        return lib.mamba2_causal_conv_step(s, a["x"], a["weight"], a["bias"], a["init"], a["out"], a["y"], None)
    return lib.mamba2_causal_conv_fwd(s, a["x"], a["weight"], a["bias"], None, a["init"], a["y"], a["out"], None)


@pytest.mark.parametrize("step", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(ptr=dict(x=None)), INVALID),
    (dict(ptr=dict(weight=None)), INVALID),
    (dict(ptr=dict(y=_p(1))), INVALID),
    (dict(ptr=dict(out=off(4, 16))), INVALID),
    (dict(ptr=dict(init=off(4, 2))), INVALID),
    (dict(width=1), INVALID),
    (dict(width=9), UNSUPPORTED),
    (dict(channels=0), INVALID),
    (dict(x_stride=63), INVALID),
    (dict(flags=2), INVALID),
    (dict(dtype=5), INVALID),
    (dict(batch=-1), INVALID),
    (dict(batch=65536), UNSUPPORTED),
])
def test_conv_refusals(lib, step, kw, code):
    assert _conv(lib, step=step, **kw) == code


def test_conv_more_refusals(lib):
    assert _conv(lib, step=True, seqlen=3) == INVALID
    assert _conv(lib, step=True, ptr=dict(out=None)) == INVALID
    assert _conv(lib, ptr=dict(out=_p(4))) == INVALID
    assert _conv(lib, batch=0) == OK
    assert lib.mamba2_causal_conv_fwd(None, *[_p(i) for i in range(1, 8)], None) == INVALID


def _norm(lib, ptr=None, **kw):
    d = dict(rows=6, channels=128, ngroups=2, x_stride=0, z_stride=0, y_stride=0, eps=1e-5, dtype=1, flags=4,
             reserved=0)
    d.update(kw)
    a = dict(x=_p(1), z=_p(2), weight=_p(3), bias=_p(4), y=_p(5))
    a.update(ptr or {})
    return lib.mamba2_group_norm(ctypes.byref(bd.mamba2_norm_shape(**d)), a["x"], a["z"], a["weight"], a["bias"],
                                 a["y"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(ptr=dict(x=None)), INVALID),
    (dict(ptr=dict(z=None)), INVALID),                  # a gate without z
    (dict(flags=1), INVALID),                           # z without a gate
    (dict(flags=2 | 4), INVALID),
    (dict(flags=4 | 8), INVALID),
    (dict(flags=16), INVALID),
    (dict(ptr=dict(y=_p(1))), INVALID),
    (dict(ptr=dict(y=off(2, 32))), INVALID),
    (dict(ptr=dict(weight=off(3, 8))), INVALID),
    (dict(ngroups=3), INVALID),
    (dict(ngroups=0), INVALID),
    (dict(eps=0.0), INVALID),
    (dict(eps=float("nan")), INVALID),
    (dict(z_stride=100), INVALID),
    (dict(reserved=1), INVALID),
    (dict(rows=-1), INVALID),
    (dict(channels=65538, ngroups=2), UNSUPPORTED),     # 32769 channels to a group
    (dict(rows=1 << 30, channels=8, ngroups=2), UNSUPPORTED),
])
def test_norm_refusals(lib, kw, code):
    assert _norm(lib, **kw) == code


def test_norm_of_no_rows(lib):
    assert _norm(lib, rows=0) == OK
    assert lib.mamba2_group_norm(None, *[_p(i) for i in range(1, 6)], None) == INVALID


def test_binding_refuses_cpu_tensors_and_wrong_layouts():
    x = torch.zeros(2, 8, 4)
    with pytest.raises(ValueError):
        bd.mamba2_causal_conv_fwd(x, torch.zeros(4, 4))
    with pytest.raises(ValueError):
        bd.mamba2_group_norm(x, None, 2)
    with pytest.raises(ValueError):
        bd.mamba2_group_norm(x, None, 2, mode="sideways")
    with pytest.raises((ValueError, TypeError)):
        bd.mamba2_gdr_fwd(x[..., None], x[..., None], x[..., None], x, x)


class _Cuda:
    """A CPU tensor that says it is on the GPU, for the layout rule alone."""
    is_cuda = True

    def __init__(self, t):
        self.t, self.shape = t, t.shape

    def stride(self):
        return self.t.stride()

    def is_contiguous(self):
        return self.t.is_contiguous()


def test_row_strides_of_slices():
    x = torch.zeros(2, 5, 24)
    row = lambda t, inner=1: bd._rows(_Cuda(t), "x", inner)  # noqa: E731
    assert row(x) == 0 and row(x[..., 8:16]) == 24 and row(x[..., 8:16].unflatten(-1, (2, 4)), 2) == 24
    assert row(x[:, :1]) == 120 and row(x[:1, :3, :8]) == 24 and row(x[:1, :3]) == 0
    for bad in (x[:, :3], x[:, ::2], x[..., ::2], x.transpose(0, 1), torch.zeros(1, 1, 24).expand(2, 5, 24)):
        with pytest.raises(ValueError):
            row(bad)


# ---------------------------------------------------- the fp64 forms themselves
def _inputs(b=2, L=12, nh=4, G=2, H=3, S=5, seed=0):
    r = np.random.default_rng(seed)
    t = lambda *s: torch.from_numpy(r.standard_normal(s))  # noqa: E731
    return t(b, L, G, S), t(b, L, G, S), t(b, L, nh, H), -t(b, L, nh).abs(), torch.sigmoid(t(b, L, nh)), t(b, nh, S, H)


def test_reference_gdr_is_the_matrix_product_form():
    """The state after each token as e^g (I - beta k k^T) h + beta k v^T."""
    q, k, v, g, beta, h0 = _inputs()
    y, fin = ref.gdr(q, k, v, g, beta, 0.7, init=h0)
    for b in range(2):
        for h in range(4):
            st = h0[b, h].numpy()
            for t in range(12):
                kt, qt = k[b, t, h // 2].numpy(), q[b, t, h // 2].numpy()
                bt = float(beta[b, t, h])
                st = np.exp(float(g[b, t, h])) * (np.eye(5) - bt * np.outer(kt, kt)) @ st + bt * np.outer(kt, v[b, t, h])
                np.testing.assert_allclose(y[b, t, h], 0.7 * qt @ st, rtol=1e-11, atol=1e-11)
            np.testing.assert_allclose(fin[b, h], st, rtol=1e-11, atol=1e-11)


def test_reference_gdr_reads_back_what_it_wrote():
    """beta = 1 and a unit key: right after the token the state answers v."""
    q, k, v, g, beta, h0 = _inputs(G=4)
    k = k / k.norm(dim=-1, keepdim=True)
    y, _ = ref.gdr(k, k, v, g, torch.ones_like(beta), 1.0, init=h0)
    np.testing.assert_allclose(y, v.numpy(), rtol=1e-11, atol=1e-11)


@pytest.mark.parametrize("mistake", ["no_decay_before_reading", "mask_includes_row_end", "group"])
def test_planted_mistakes_show(mistake):
    q, k, v, g, beta, h0 = _inputs()
    y, h = ref.gdr(q, k, v, g, beta, 1.0, init=h0, lengths=torch.tensor([12, 7]))
    if mistake == "no_decay_before_reading":
        y2, h2 = ref.gdr(q, k, v, torch.zeros_like(g), beta, 1.0, init=h0, lengths=torch.tensor([12, 7]))
    elif mistake == "mask_includes_row_end":
        y2, h2 = ref.gdr(q, k, v, g, beta, 1.0, init=h0, lengths=torch.tensor([12, 8]))
    else:
        y2, h2 = ref.gdr(q.flip(2), k.flip(2), v, g, beta, 1.0, init=h0, lengths=torch.tensor([12, 7]))
    assert np.abs(y - y2).max() > 1e-2 and np.abs(h - h2).max() > 1e-2


def test_reference_conv_and_norm_on_hand_worked_values():
    x = torch.tensor([[[1.0], [2.0], [3.0]]])
    w = torch.tensor([[10.0, 1.0]])
    y, s = ref.conv(x, w, act=False, init=torch.tensor([[[5.0]]]))
    assert y[0, :, 0].tolist() == [51.0, 12.0, 23.0] and s[0, :, 0].tolist() == [3.0]
    y, s = ref.conv(x, w, act=False, lengths=torch.tensor([0]), init=torch.tensor([[[5.0]]]))
    assert y[0, :, 0].tolist() == [0.0] * 3 and s[0, :, 0].tolist() == [5.0]
    y = ref.norm(torch.tensor([[3.0, -3.0, 1.0, 5.0]]), 2, mean=True, eps=0.0)
    np.testing.assert_allclose(y, [[1, -1, -1, 1]])
    y = ref.norm(torch.tensor([[3.0, 4.0]]), 1, eps=0.0, weight=torch.tensor([2.0, 1.0]))
    np.testing.assert_allclose(y, [[6 / 12.5 ** 0.5, 4 / 12.5 ** 0.5]])
