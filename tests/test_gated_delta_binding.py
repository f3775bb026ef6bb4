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
    return rec


def gdr(step=False, lead=None, device=None, **kw):
    """A call of the rule with every tensor given; `device` puts single ones on other GPUs."""
    lead = ((2,) if step else (2, 5)) if lead is None else lead
    at = lambda name, *s: Gpu(*s, device=(device or {}).get(name, 0))  # noqa: E731
    t = {"q": at("q", *lead, 2, 16), "k": at("k", *lead, 2, 16), "v": at("v", *lead, 4, 8),
         "g": at("g", *lead, 4), "beta": at("beta", *lead, 4)}
    b = lead[0] if lead else 4
    first, last = ("state_in", "state_out") if step else ("initial_state", "final_state")
    t.update({"y": at("y", *lead, 4, 8), first: at(first, b, 4, 16, 8), last: at(last, b, 4, 16, 8)})
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
