"""Thin Python binding of libmamba2ssd.so (argument marshalling only).

Each function has the name of the C entry point it calls and takes torch
tensors that already live on the GPU; it passes their data pointers, the
shape and the current CUDA stream (or the ``stream`` it is given) to the library
and allocates any missing output with ``torch.empty`` on that stream.  No step of the forward pass runs in Python: if
the library is missing the import fails loudly, there is no fallback.

Layouts and semantics are those of include/mamba2_ssd.h ("Accelerating
Mamba-2 with High-Performance Forward Pass Kernels in NVIDIA CUDA Tile",
§Kernel 1-3) and, for the gated delta rule, the causal convolution and the
group norm, of include/mamba2_gated_delta.h.
"""
from __future__ import annotations

import ctypes
import functools
import operator
import os
import re

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmamba2ssd.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "mamba2_ssd.h")
HEADER_GATED_DELTA = os.path.join(os.path.dirname(_PKG), "include", "mamba2_gated_delta.h")

MAMBA2_F32, MAMBA2_BF16 = 0, 1
MAMBA2_GDR_QK_L2NORM = 1
MAMBA2_CONV_SILU = 1
MAMBA2_NORM_SUBTRACT_MEAN, MAMBA2_NORM_GATE_BEFORE, MAMBA2_NORM_GATE_AFTER, MAMBA2_NORM_SILU = 1, 2, 4, 8
NORM_MODES = {"none": 0, "before": MAMBA2_NORM_GATE_BEFORE, "after": MAMBA2_NORM_GATE_AFTER,
              "silu": MAMBA2_NORM_SILU}
STATUS = {0: "MAMBA2_OK", 1: "MAMBA2_ERR_INVALID_ARG", 2: "MAMBA2_ERR_UNSUPPORTED",
          3: "MAMBA2_ERR_CUDA", 4: "MAMBA2_ERR_TIMEOUT"}


class Mamba2Error(RuntimeError):
    def __init__(self, fn: str, code: int, text: str):
        super().__init__(f"{fn} failed: {text}")
        self.code = code


class mamba2_shape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("nheads", ctypes.c_int64),
                ("headdim", ctypes.c_int64), ("dstate", ctypes.c_int64), ("ngroups", ctypes.c_int64),
                ("chunk_size", ctypes.c_int64), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class mamba2_gdr_options(ctypes.Structure):
    _fields_ = [("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("scale", ctypes.c_float), ("l2_eps", ctypes.c_float), ("flags", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class mamba2_conv_shape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("channels", ctypes.c_int64),
                ("width", ctypes.c_int64), ("x_stride", ctypes.c_int64), ("y_stride", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("flags", ctypes.c_int32)]


class mamba2_norm_shape(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("channels", ctypes.c_int64), ("ngroups", ctypes.c_int64),
                ("x_stride", ctypes.c_int64), ("z_stride", ctypes.c_int64), ("y_stride", ctypes.c_int64),
                ("eps", ctypes.c_float), ("dtype", ctypes.c_int32), ("flags", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libmamba2ssd.so; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with "
                          "`python -m mamba_chunked_ssd_gb300.build_lib` (needs nvcc)")
    lib = ctypes.CDLL(path)
    P, S = ctypes.c_void_p, ctypes.POINTER(mamba2_shape)
    O, V, N = (ctypes.POINTER(t) for t in (mamba2_gdr_options, mamba2_conv_shape, mamba2_norm_shape))
    sig = {
        "mamba2_chunk_cumsum": (ctypes.c_int, [S, P, P, P, P]),
        "mamba2_state_pass": (ctypes.c_int, [S, P, P, P, P, P, P, P, P]),
        "mamba2_chunk_out": (ctypes.c_int, [S, P, P, P, P, P, P, P, P, P]),
        "mamba2_ssd_fwd_workspace_size": (ctypes.c_size_t, [S]),
        "mamba2_ssd_fwd_chunk_size": (ctypes.c_int64, [S]),
        "mamba2_ssd_fwd": (ctypes.c_int, [S, P, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]),
        "mamba2_ssd_fwd_noalloc": (ctypes.c_int, [S, P, P, P, P, P, P, P, P, P, P]),
        "mamba2_ssd_step": (ctypes.c_int, [S, P, P, P, P, P, P, P, P, P, P]),
        "mamba2_gdr_fwd": (ctypes.c_int, [S, O, P, P, P, P, P, P, P, P, P, P]),
        "mamba2_gdr_step": (ctypes.c_int, [S, O, P, P, P, P, P, P, P, P, P]),
        "mamba2_causal_conv_fwd": (ctypes.c_int, [V, P, P, P, P, P, P, P, P]),
        "mamba2_causal_conv_step": (ctypes.c_int, [V, P, P, P, P, P, P, P]),
        "mamba2_group_norm": (ctypes.c_int, [N, P, P, P, P, P, P]),
        "mamba2_selftest_wait_timeout": (ctypes.c_int, [ctypes.c_int64, P]),
        "mamba2_check_device_status": (ctypes.c_int, [P]),
        "mamba2_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "mamba2_version": (ctypes.c_int, []),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
    _lib = lib
    return lib


def header_functions(path: str = HEADER):
    """Names of the functions include/mamba2_ssd.h declares."""
    text = open(path).read()
    return sorted(set(re.findall(r"MAMBA2_API\s+[\w\s\*]+?\b(mamba2_\w+)\s*\(", text)))


def _check(fn: str, rc: int):
    if rc != 0:
        text = load_library().mamba2_status_string(rc).decode()
        raise Mamba2Error(fn, rc, text)


_current_gpu = torch._C._cuda_getDevice


def _ptr(t):
    """A tensor's address, on the current GPU: the launch goes there."""
    if t is None:
        return None
    if t.get_device() != _current_gpu():
        raise ValueError(f"a tensor is on {t.device}, but the current device is cuda:{_current_gpu()}")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if stream.device.index != _current_gpu():
        raise ValueError(f"the stream is on {stream.device}, but the current device is cuda:{_current_gpu()}")
    return ctypes.c_void_p(stream.cuda_stream)


def _new(shape, dtype, device, stream):
    """An output or workspace from the pool of the call's stream: memory that was freed
    on another one may still be in use there."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return MAMBA2_BF16
    if t.dtype == torch.float32:
        return MAMBA2_F32
    raise TypeError(f"unsupported dtype {t.dtype}: x, B, C must be bfloat16 or float32")


def make_shape(batch, seqlen, nheads, headdim, dstate, ngroups, chunk_size, dtype_code) -> mamba2_shape:
    return mamba2_shape(batch, seqlen, nheads, headdim, dstate, ngroups, chunk_size, dtype_code, 0)


def shape_of(x: torch.Tensor, B: torch.Tensor, chunk_size: int) -> mamba2_shape:
    b, L, nh, H = x.shape
    return make_shape(b, L, nh, H, B.shape[3], B.shape[2], int(chunk_size), _dtype_code(x))


def _need(t, name):
    if t is not None and not (t.is_cuda and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous CUDA tensor")


def mamba2_chunk_cumsum(dt, A, chunk_size, G=None, stream=None):
    """Stage 1: G [b, nh, L] fp32 (log2 units)."""
    _need(dt, "dt"), _need(A, "A")
    b, L, nh = dt.shape
    shape = make_shape(b, L, nh, 1, 1, 1, int(chunk_size), MAMBA2_F32)
    if G is None:
        G = _new((b, nh, L), torch.float32, dt.device, stream)
    _check("mamba2_chunk_cumsum", load_library().mamba2_chunk_cumsum(
        ctypes.byref(shape), _ptr(dt), _ptr(A), _ptr(G), _stream(stream)))
    return G


def mamba2_state_pass(x, dt, B, G, chunk_size, initial_state=None, chunk_states=None,
                      final_state=None, want_final_state=True, stream=None):
    """Stage 2: (chunk_states [b, nh, nc, S, H], final_state [b, nh, S, H] or None)."""
    for t, n in ((x, "x"), (dt, "dt"), (B, "B"), (G, "G"), (initial_state, "initial_state")):
        _need(t, n)
    shape = shape_of(x, B, chunk_size)
    nc = -(-shape.seqlen // shape.chunk_size)
    if chunk_states is None:
        chunk_states = _new((shape.batch, shape.nheads, nc, shape.dstate, shape.headdim), x.dtype, x.device, stream)
    if final_state is None and want_final_state:
        final_state = _new((shape.batch, shape.nheads, shape.dstate, shape.headdim), torch.float32, x.device, stream)
    _check("mamba2_state_pass", load_library().mamba2_state_pass(
        ctypes.byref(shape), _ptr(x), _ptr(dt), _ptr(B), _ptr(G), _ptr(initial_state),
        _ptr(chunk_states), _ptr(final_state), _stream(stream)))
    return chunk_states, final_state


def mamba2_chunk_out(x, dt, B, C, G, chunk_states, chunk_size, D=None, y=None, stream=None):
    """Stage 3: y [b, L, nh, H] in x's dtype."""
    for t, n in ((x, "x"), (dt, "dt"), (B, "B"), (C, "C"), (G, "G"), (chunk_states, "chunk_states"),
                 (D, "D")):
        _need(t, n)
    shape = shape_of(x, B, chunk_size)
    if y is None:
        y = _new(x.shape, x.dtype, x.device, stream)
    _check("mamba2_chunk_out", load_library().mamba2_chunk_out(
        ctypes.byref(shape), _ptr(x), _ptr(dt), _ptr(B), _ptr(C), _ptr(D), _ptr(G),
        _ptr(chunk_states), _ptr(y), _stream(stream)))
    return y


def mamba2_ssd_fwd_workspace_size(shape: mamba2_shape) -> int:
    return int(load_library().mamba2_ssd_fwd_workspace_size(ctypes.byref(shape)))


def mamba2_ssd_fwd_chunk_size(shape: mamba2_shape) -> int:
    return int(load_library().mamba2_ssd_fwd_chunk_size(ctypes.byref(shape)))


def mamba2_ssd_fwd(x, dt, A, B, C, chunk_size, D=None, initial_state=None, y=None, final_state=None,
                   want_final_state=True, workspace=None, stream=None):
    """Whole forward pass: (y, final_state or None)."""
    for t, n in ((x, "x"), (dt, "dt"), (A, "A"), (B, "B"), (C, "C"), (D, "D"),
                 (initial_state, "initial_state")):
        _need(t, n)
    shape = shape_of(x, B, chunk_size)
    if y is None:
        y = _new(x.shape, x.dtype, x.device, stream)
    if final_state is None and want_final_state:
        final_state = _new((shape.batch, shape.nheads, shape.dstate, shape.headdim), torch.float32, x.device, stream)
    ws_bytes = mamba2_ssd_fwd_workspace_size(shape)
    if workspace is None:
        workspace = _new(max(ws_bytes, 1), torch.uint8, x.device, stream)
    _check("mamba2_ssd_fwd", load_library().mamba2_ssd_fwd(
        ctypes.byref(shape), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
        _ptr(initial_state), _ptr(y), _ptr(final_state), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))
    return y, final_state


def mamba2_ssd_fwd_noalloc(x, dt, A, B, C, chunk_size, D=None, initial_state=None, y=None,
                           final_state=None, want_final_state=True, stream=None):
    """Whole forward pass with the library's fixed internal scratch (no
    workspace argument; the C entry point allocates nothing).  Missing outputs
    are allocated here, by the caller side, with torch."""
    for t, n in ((x, "x"), (dt, "dt"), (A, "A"), (B, "B"), (C, "C"), (D, "D"),
                 (initial_state, "initial_state")):
        _need(t, n)
    shape = shape_of(x, B, chunk_size)
    if y is None:
        y = _new(x.shape, x.dtype, x.device, stream)
    if final_state is None and want_final_state:
        final_state = _new((shape.batch, shape.nheads, shape.dstate, shape.headdim), torch.float32, x.device, stream)
    _check("mamba2_ssd_fwd_noalloc", load_library().mamba2_ssd_fwd_noalloc(
        ctypes.byref(shape), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
        _ptr(initial_state), _ptr(y), _ptr(final_state), _stream(stream)))
    return y, final_state


def mamba2_ssd_step(x, dt, A, B, C, state_in=None, D=None, state_out=None, y=None, stream=None):
    """One decode step: x [b, nh, H], dt [b, nh], B, C [b, G, S], state
    [b, nh, S, H] fp32.  Returns (y [b, nh, H], state_out).  Pass
    state_out=state_in to update the state in place."""
    for t, n in ((x, "x"), (dt, "dt"), (A, "A"), (B, "B"), (C, "C"), (D, "D"),
                 (state_in, "state_in"), (state_out, "state_out")):
        _need(t, n)
    b, nh, H = x.shape
    shape = make_shape(b, 1, nh, H, B.shape[2], B.shape[1], 1, _dtype_code(x))
    if y is None:
        y = _new(x.shape, x.dtype, x.device, stream)
    if state_out is None:
        state_out = _new((b, nh, B.shape[2], H), torch.float32, x.device, stream)
    _check("mamba2_ssd_step", load_library().mamba2_ssd_step(
        ctypes.byref(shape), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
        _ptr(state_in), _ptr(state_out), _ptr(y), _stream(stream)))
    return y, state_out


# The gated-delta-rule entry points are also called once a token, where the host
# call is the time: they pass plain integers (ctypes makes the pointers), ask for
# the raw stream, check a tensor's layout in as few attribute reads as will do, and
# keep the structures that describe a call's sizes (never its tensors: what may come
# as one, a scale, an eps or a number of groups, is a number before it is looked up).
_raw_stream = torch._C._cuda_getCurrentRawStream


def _at(t):
    return None if t is None else t.data_ptr()


def _on(stream, gpu):
    if stream is None:
        return _raw_stream(gpu)
    if stream.device.index != gpu:
        raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{gpu}")
    return stream.cuda_stream


def _rows(t, name, inner):
    """Stride from row to row of a tensor whose last ``inner`` dimensions are
    packed and whose leading ones form one run of rows, e.g. a channel slice of
    a contiguous [b, L, C] tensor (0: packed, as in the C interface)."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.is_contiguous():
        return 0
    shape, st = t.shape, t.stride()
    lead, want = len(shape) - inner, 1
    for d in range(len(shape) - 1, lead - 1, -1):
        if shape[d] != 1 and st[d] != want:
            raise ValueError(f"{name}: the last {inner} dimension(s) must be packed")
        want *= shape[d]
    row = None
    for d in range(lead - 1, -1, -1):
        if shape[d] == 1:
            continue
        if row is None:
            row = run = st[d]
        elif st[d] != run:
            raise ValueError(f"{name}: its rows must be one run with one stride")
        run *= shape[d]
    if row is None:
        return want
    if row < want:
        raise ValueError(f"{name}: its rows overlap")
    return row


def _gpu(t, name):
    """The index of a tensor's GPU, which has to be the current one: the launch goes there."""
    gpu = t.get_device()
    if gpu < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if gpu != _current_gpu():
        raise ValueError(f"{name} is on cuda:{gpu}, but the current device is cuda:{_current_gpu()}")
    return gpu


def _want(t, name, dtype, shape, gpu):
    """A contiguous tensor of this dtype and shape on this GPU (or None)."""
    if t is None or (t.dtype is dtype and t.shape == shape and t.get_device() == gpu and t.is_contiguous()):
        return
    raise ValueError(f"{name} must be a contiguous tensor on cuda:{gpu}, {dtype} {tuple(shape)}, "
                     f"not {t.dtype} {tuple(t.shape)} on {t.device} with strides {t.stride()}")


def _like(t, given, name, stream=None):
    """The output for an input's dtype, shape and GPU: the given one, checked, or a new one."""
    if given is None and stream is None:
        return torch.empty_like(t, memory_format=torch.contiguous_format)
    if given is None:
        return _new(t.shape, t.dtype, t.device, stream)
    if given.dtype is not t.dtype or given.shape != t.shape or given.get_device() != t.get_device():
        raise ValueError(f"{name} must be {t.dtype} {tuple(t.shape)} on {t.device}, "
                         f"not {given.dtype} {tuple(given.shape)} on {given.device}")
    return given


_gdr_shape = functools.lru_cache(maxsize=1024)(lambda *a: mamba2_shape(*a))
_gdr_options = functools.lru_cache(maxsize=1024)(lambda *a: mamba2_gdr_options(*a))
_conv_shape = functools.lru_cache(maxsize=1024)(lambda *a: mamba2_conv_shape(*a))
_norm_shape = functools.lru_cache(maxsize=1024)(lambda *a: mamba2_norm_shape(*a))


def _gdr_args(q, k, v, g, beta, scale, qk_l2norm, l2_eps):
    """The shape and options of a gated-delta-rule call, its state's shape and its GPU; checks q, k, v, g, beta."""
    vs, qs, dt = v.shape, q.shape, v.dtype
    if len(vs) not in (3, 4):
        raise ValueError(f"v must have the dimensions (batch, [tokens,] heads, headdim), not {tuple(vs)}")
    rows, nh = vs[:-1], vs[-2]
    if qs != k.shape or len(qs) != len(vs) or qs[:-2] != vs[:-2]:
        raise ValueError(f"q and k must be {tuple(vs[:-2])} + (groups, state): got {tuple(qs)}, {tuple(k.shape)}")
    if q.dtype is not dt or k.dtype is not dt:
        raise TypeError("q, k and v must have one dtype")
    gpu = _gpu(v, "v")
    if q.get_device() != gpu or k.get_device() != gpu:
        raise ValueError(f"q and k must be on {v.device} as v is, not on {q.device} and {k.device}")
    _want(g, "g", torch.float32, rows, gpu), _want(beta, "beta", torch.float32, rows, gpu)
    S = qs[-1]
    shape = _gdr_shape(vs[0], vs[1] if len(vs) == 4 else 1, nh, vs[-1], S, qs[-2], 64, _dtype_code(v), 0)
    opt = _gdr_options(_rows(q, "q", 2), _rows(k, "k", 2), _rows(v, "v", 2),
                       S ** -0.5 if scale is None else float(scale), float(l2_eps),
                       MAMBA2_GDR_QK_L2NORM if qk_l2norm else 0, 0)
    return shape, opt, (vs[0], nh, S, vs[-1]), gpu


def mamba2_gdr_fwd(q, k, v, g, beta, scale=None, qk_l2norm=False, l2_eps=1e-6, initial_state=None, lengths=None,
                   y=None, final_state=None, want_final_state=True, stream=None):
    """The gated delta rule over whole sequences: (y [b, L, nh, H], final_state
    [b, nh, S, H] fp32 or None).  q, k [b, L, G, S] and v [b, L, nh, H] may be
    slices of a wider tensor; g (log decay), beta [b, L, nh] fp32; scale
    defaults to S ** -0.5; lengths [b] int32 or None."""
    shape, opt, state, gpu = _gdr_args(q, k, v, g, beta, scale, qk_l2norm, l2_eps)
    _want(initial_state, "initial_state", torch.float32, state, gpu)
    _want(lengths, "lengths", torch.int32, state[:1], gpu)
    if y is not None:
        _want(y, "y", v.dtype, v.shape, gpu)
    y = _like(v, y, "y", stream)
    if final_state is not None:
        _want(final_state, "final_state", torch.float32, state, gpu)
    elif want_final_state:
        final_state = _new(state, torch.float32, v.device, stream)
    rc = load_library().mamba2_gdr_fwd(shape, opt, _at(q), _at(k), _at(v), _at(g), _at(beta), _at(lengths),
                                       _at(initial_state), _at(y), _at(final_state), _on(stream, gpu))
    if rc:
        _check("mamba2_gdr_fwd", rc)
    return y, final_state


def mamba2_gdr_step(q, k, v, g, beta, state_in=None, scale=None, qk_l2norm=False, l2_eps=1e-6, state_out=None, y=None,
                    stream=None):
    """One token of the gated delta rule: q, k [b, G, S], v [b, nh, H], g, beta
    [b, nh], state [b, nh, S, H] fp32.  Returns (y [b, nh, H], state_out).  Pass
    state_out=state_in to update the state in place."""
    shape, opt, state, gpu = _gdr_args(q, k, v, g, beta, scale, qk_l2norm, l2_eps)
    _want(state_in, "state_in", torch.float32, state, gpu)
    if y is not None:
        _want(y, "y", v.dtype, v.shape, gpu)
    y = _like(v, y, "y", stream)
    if state_out is None:
        state_out = _new(state, torch.float32, v.device, stream)
    elif state_out is not state_in:
        _want(state_out, "state_out", torch.float32, state, gpu)
    rc = load_library().mamba2_gdr_step(shape, opt, _at(q), _at(k), _at(v), _at(g), _at(beta), _at(state_in),
                                        _at(state_out), _at(y), _on(stream, gpu))
    if rc:
        _check("mamba2_gdr_step", rc)
    return y, state_out


def mamba2_causal_conv_fwd(x, weight, bias=None, silu=True, initial_state=None, lengths=None, y=None,
                           final_state=None, want_final_state=True, stream=None):
    """Depthwise causal convolution over time: x [b, L, C] (may be a channel
    slice), weight [C, W] and bias [C] fp32, states [b, W - 1, C] in x's dtype.
    Returns (y [b, L, C], final_state or None)."""
    b, L, C = x.shape
    W, gpu = weight.shape[-1], _gpu(x, "x")
    _want(weight, "weight", torch.float32, (C, W), gpu), _want(bias, "bias", torch.float32, (C,), gpu)
    _want(initial_state, "initial_state", x.dtype, (b, W - 1, C), gpu)
    _want(lengths, "lengths", torch.int32, (b,), gpu)
    y = _like(x, y, "y", stream)
    if final_state is not None:
        _want(final_state, "final_state", x.dtype, (b, W - 1, C), gpu)
    elif want_final_state:
        final_state = _new((b, W - 1, C), x.dtype, x.device, stream)
    shape = _conv_shape(b, L, C, W, _rows(x, "x", 1), _rows(y, "y", 1), _dtype_code(x),
                        MAMBA2_CONV_SILU if silu else 0)
    rc = load_library().mamba2_causal_conv_fwd(shape, _at(x), _at(weight), _at(bias), _at(lengths), _at(initial_state),
                                               _at(y), _at(final_state), _on(stream, gpu))
    if rc:
        _check("mamba2_causal_conv_fwd", rc)
    return y, final_state


def mamba2_causal_conv_step(x, weight, state_in=None, bias=None, silu=True, state_out=None, y=None, stream=None):
    """One token of the convolution: x [b, C], state [b, W - 1, C] in x's dtype.
    Returns (y [b, C], state_out); state_out=state_in updates in place."""
    b, C = x.shape
    W, gpu = weight.shape[-1], _gpu(x, "x")
    state = (b, W - 1, C)
    _want(weight, "weight", torch.float32, (C, W), gpu), _want(bias, "bias", torch.float32, (C,), gpu)
    _want(state_in, "state_in", x.dtype, state, gpu)
    y = _like(x, y, "y", stream)
    if state_out is None:
        state_out = _new(state, x.dtype, x.device, stream)
    elif state_out is not state_in:
        _want(state_out, "state_out", x.dtype, state, gpu)
    shape = _conv_shape(b, 1, C, W, _rows(x, "x", 1), _rows(y, "y", 1), _dtype_code(x),
                        MAMBA2_CONV_SILU if silu else 0)
    rc = load_library().mamba2_causal_conv_step(shape, _at(x), _at(weight), _at(bias), _at(state_in), _at(state_out),
                                                _at(y), _on(stream, gpu))
    if rc:
        _check("mamba2_causal_conv_step", rc)
    return y, state_out


def mamba2_group_norm(x, weight, ngroups, z=None, bias=None, eps=1e-5, subtract_mean=False, mode="none", y=None,
                      stream=None):
    """Group norm of each row of x [.., C] over its ngroups groups of channels:
    mode "none", "silu" (SiLU of the result), "before" or "after" (a gate
    SiLU(z) before or after the norm).  weight, bias [C] fp32 or None."""
    C, gpu = x.shape[-1], _gpu(x, "x")
    _want(weight, "weight", torch.float32, (C,), gpu), _want(bias, "bias", torch.float32, (C,), gpu)
    flags = NORM_MODES.get(mode)
    if flags is None:
        raise ValueError(f"mode must be one of {sorted(NORM_MODES)}, not {mode!r}")
    if z is not None:
        _like(x, z, "z")
    y = _like(x, y, "y", stream)
    shape = _norm_shape(x.numel() // C if C else 0, C, operator.index(ngroups), _rows(x, "x", 1),
                        0 if z is None else _rows(z, "z", 1), _rows(y, "y", 1), float(eps), _dtype_code(x),
                        flags | MAMBA2_NORM_SUBTRACT_MEAN if subtract_mean else flags, 0)
    rc = load_library().mamba2_group_norm(shape, _at(x), _at(z), _at(weight), _at(bias), _at(y), _on(stream, gpu))
    if rc:
        _check("mamba2_group_norm", rc)
    return y


def mamba2_selftest_wait_timeout(limit_ns: int, stream=None):
    """Enqueue the bounded-wait self-test kernel (see the header); the next
    mamba2_check_device_status then raises with MAMBA2_ERR_TIMEOUT."""
    _check("mamba2_selftest_wait_timeout",
           load_library().mamba2_selftest_wait_timeout(int(limit_ns), _stream(stream)))


def mamba2_check_device_status(stream=None):
    """Synchronises the stream and raises if a kernel reported a timeout."""
    _check("mamba2_check_device_status", load_library().mamba2_check_device_status(_stream(stream)))


def mamba2_version() -> int:
    return int(load_library().mamba2_version())
