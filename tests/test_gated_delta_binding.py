"""CPU checks of what the binding of the gated-delta-rule operators hands to the
library: stand-ins for GPU tensors and a library that records its arguments."""
import pytest
import torch

from mamba_chunked_ssd_gb300 import binding as bd


class Gpu:
    """A CPU tensor that says it is on a GPU."""
    is_cuda = True

    def __init__(self, *shape, dtype=torch.float32, device=0):
        self.t, self.dtype, self.index = torch.zeros(*shape, dtype=dtype), dtype, device
        self.shape, self.device = self.t.shape, torch.device("cuda", device)

    def get_device(self):
        return self.index

    def __getattr__(self, name):  # stride, is_contiguous, data_ptr, numel
        return getattr(self.t, name)


class Recorder:
    """Every entry point: keeps its name and arguments and answers MAMBA2_OK."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    rec = Recorder()
    monkeypatch.setattr(bd, "load_library", lambda: rec)
    monkeypatch.setattr(bd, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(bd, "_current_gpu", lambda: 0, raising=False)
    return rec


def gdr(step=False, lead=None, device=None, drop=(), **kw):
    """A call of the rule with every tensor given but those in `drop`; `device` puts
    single ones on other GPUs."""
    lead = ((2,) if step else (2, 5)) if lead is None else lead
    at = lambda name, *s: Gpu(*s, device=(device or {}).get(name, 0))  # noqa: E731
    t = {"q": at("q", *lead, 2, 16), "k": at("k", *lead, 2, 16), "v": at("v", *lead, 4, 8),
         "g": at("g", *lead, 4), "beta": at("beta", *lead, 4)}
    b = lead[0] if lead else 4
    first, last = ("state_in", "state_out") if step else ("initial_state", "final_state")
    t.update({"y": at("y", *lead, 4, 8), first: at(first, b, 4, 16, 8), last: at(last, b, 4, 16, 8)})
    t = {n: x for n, x in t.items() if n not in drop}
    return (bd.mamba2_gdr_step if step else bd.mamba2_gdr_fwd)(**t, **kw)


@pytest.mark.parametrize("step", [False, True])
def test_a_scale_that_is_a_tensor_counts_by_its_value(lib, step):
    """A tensor that is changed between two calls: the second call has its new value."""
    scale, eps = torch.tensor(0.5), torch.tensor(1e-6)
    gdr(step, scale=scale, l2_eps=eps, qk_l2norm=True)
    scale.fill_(3.0), eps.fill_(0.25)
    gdr(step, scale=scale, l2_eps=eps, qk_l2norm=True)
    first, second = (args[1] for _, args in lib.calls)
    assert (first.scale, second.scale, second.l2_eps) == (0.5, 3.0, 0.25)


def test_an_eps_that_is_a_tensor_counts_by_its_value(lib):
    eps, x = torch.tensor(0.5), Gpu(6, 8)
    for value in (0.5, 0.25):
        eps.fill_(value)
        bd.mamba2_group_norm(x, None, 2, eps=eps, y=Gpu(6, 8))
    assert [args[0].eps for _, args in lib.calls] == [0.5, 0.25]


def test_a_number_of_groups_that_is_a_tensor_counts_by_its_value(lib):
    groups, x = torch.tensor(2), Gpu(6, 8)
    for value in (2, 4):
        groups.fill_(value)
        bd.mamba2_group_norm(x, None, groups, y=Gpu(6, 8))
    assert [args[0].ngroups for _, args in lib.calls] == [2, 4]
    with pytest.raises(TypeError):
        bd.mamba2_group_norm(x, None, 2.0, y=Gpu(6, 8))


@pytest.mark.parametrize("step", [False, True])
@pytest.mark.parametrize("lead", [(), (2, 3, 5)])
def test_tensors_with_too_few_or_too_many_dimensions_are_refused(lib, step, lead):
    """With two dimensions heads would be taken for batch rows (and read behind the
    tensors' ends); with five all but one token of a row would be left out."""
    with pytest.raises(ValueError, match="dimensions"):
        gdr(step, lead=lead)
    assert lib.calls == []


@pytest.mark.parametrize("step", [False, True])
def test_a_single_token_with_and_without_its_dimension(lib, step):
    gdr(step, lead=(3,)), gdr(step, lead=(3, 1))
    for _, args in lib.calls:
        assert (args[0].batch, args[0].seqlen, args[0].nheads) == (3, 1, 4)


def conv(step=False, device=None, drop=(), **kw):
    b, C, W = 2, 8, 4
    at = lambda name, *s: Gpu(*s, device=(device or {}).get(name, 0))  # noqa: E731
    first, last = ("state_in", "state_out") if step else ("initial_state", "final_state")
    lead = (b,) if step else (b, 5)
    t = {"x": at("x", *lead, C), "weight": at("weight", C, W), "bias": at("bias", C), "y": at("y", *lead, C),
         first: at(first, b, W - 1, C), last: at(last, b, W - 1, C)}
    t = {n: x for n, x in t.items() if n not in drop}
    return (bd.mamba2_causal_conv_step if step else bd.mamba2_causal_conv_fwd)(**t, **kw)


def norm(device=None, drop=(), **kw):
    at = lambda name, *s: Gpu(*s, device=(device or {}).get(name, 0))  # noqa: E731
    return bd.mamba2_group_norm(at("x", 6, 8), at("weight", 8), 2, z=at("z", 6, 8), bias=at("bias", 8),
                                y=None if "y" in drop else at("y", 6, 8), mode="after", **kw)


CALLS = {"gdr_fwd": (gdr, "q k v g beta y initial_state final_state"),
         "gdr_step": (lambda **kw: gdr(True, **kw), "q k v g beta y state_in state_out"),
         "conv_fwd": (conv, "x weight bias y initial_state final_state"),
         "conv_step": (lambda **kw: conv(True, **kw), "x weight bias y state_in state_out"),
         "norm": (norm, "x weight bias z y")}


@pytest.mark.parametrize("call,names", CALLS.values(), ids=CALLS)
def test_tensors_on_another_gpu_are_refused(lib, monkeypatch, call, names):
    """One tensor on another GPU than the rest, and all of them on another one than
    the current: a launch would get addresses that are not its device's."""
    call()
    assert len(lib.calls) == 1
    for name in names.split():
        with pytest.raises(ValueError, match="cuda:"):
            call(device={name: 1})
    with pytest.raises(ValueError, match="current device"):
        call(device=dict.fromkeys(names.split(), 1))
    assert len(lib.calls) == 1
    monkeypatch.setattr(bd, "_current_gpu", lambda: 1)
    call(device=dict.fromkeys(names.split(), 1))
    assert len(lib.calls) == 2


@pytest.mark.parametrize("call", [c for c, _ in CALLS.values()], ids=CALLS)
def test_a_stream_of_another_gpu_is_refused(lib, call):
    class Stream:
        cuda_stream, device = 7, torch.device("cuda", 0)
    call(stream=Stream())
    assert lib.calls[0][1][-1] == 7
    Stream.device = torch.device("cuda", 1)
    with pytest.raises(ValueError, match="stream"):
        call(stream=Stream())


def test_lengths_on_another_gpu_are_refused(lib):
    for call in (gdr, conv):
        call(lengths=Gpu(2, dtype=torch.int32))
        with pytest.raises(ValueError, match="lengths"):
            call(lengths=Gpu(2, dtype=torch.int32, device=1))


@pytest.mark.parametrize("call", [c for c, _ in CALLS.values()], ids=CALLS)
def test_outputs_that_are_not_given_come_from_the_stream_of_the_call(lib, monkeypatch, call):
    """Memory from the current stream's pool may still be in use there, and a kernel
    on another stream does not wait for that."""
    class Stream:
        cuda_stream, device = 7, torch.device("cuda", 0)

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
    outputs = ("y", "final_state", "state_out")
    stream = Stream()
    call(stream=stream, drop=outputs)
    assert made and all(s is stream for s in made) and not under
    count = len(made)
    call(drop=outputs)
    assert made[count:] == [None] * count
