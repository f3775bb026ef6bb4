"""CPU checks of what the binding of the state-space entry points hands to the
library, with stand-ins for GPU tensors."""
import pytest
import torch

from mamba_chunked_ssd_gb300 import binding as bd
from test_gated_delta_binding import Gpu, lib  # noqa: F401


class Stream:
    def __init__(self, device=0):
        self.cuda_stream, self.device = 7, torch.device("cuda", device)


def tensors(names, device):
    b, L, nh, H, G, S, T = 2, 8, 4, 8, 2, 16, 4
    shapes = {"x": (b, L, nh, H), "dt": (b, L, nh), "A": (nh,), "B": (b, L, G, S), "C": (b, L, G, S), "D": (nh,),
              "G": (b, nh, L), "chunk_states": (b, nh, L // T, S, H), "y": (b, L, nh, H), "workspace": (64,),
              **dict.fromkeys(("initial_state", "final_state", "state_in", "state_out"), (b, nh, S, H))}
    return {n: Gpu(*shapes[n], device=device.get(n, 0)) for n in names}


CALLS = {"mamba2_chunk_cumsum": "dt A G",
         "mamba2_state_pass": "x dt B G initial_state chunk_states final_state",
         "mamba2_chunk_out": "x dt B C G chunk_states D y",
         "mamba2_ssd_fwd": "x dt A B C D initial_state y final_state workspace",
         "mamba2_ssd_fwd_noalloc": "x dt A B C D initial_state y final_state",
         "mamba2_ssd_step": "x dt A B C D state_in state_out y"}


@pytest.mark.parametrize("name", CALLS)
def test_tensors_and_streams_of_another_gpu_are_refused(lib, monkeypatch, name):  # noqa: F811
    names = CALLS[name].split()

    def call(device={}, stream=Stream()):
        t = tensors(names, device)
        if name == "mamba2_ssd_step":  # one token: no sequence dimension
            for n in ("x", "dt", "B", "C", "y"):
                t[n].t = t[n].t[:, 0].contiguous()
                t[n].shape = t[n].t.shape
        else:
            t["chunk_size"] = 4
        getattr(bd, name)(**t, stream=stream)
        return sum(n == name for n, _ in lib.calls)

    assert call() == 1
    for n in names:
        with pytest.raises(ValueError, match="cuda:"):
            call({n: 1})
    with pytest.raises(ValueError, match="cuda:"):
        call(dict.fromkeys(names, 1))
    with pytest.raises(ValueError, match="stream"):
        call(stream=Stream(1))
    monkeypatch.setattr(bd, "_current_gpu", lambda: 1)
    assert call(dict.fromkeys(names, 1), Stream(1)) == 2


@pytest.mark.parametrize("name", CALLS)
def test_outputs_and_workspace_that_are_not_given_come_from_the_stream_of_the_call(lib, monkeypatch, name):  # noqa: F811
    under, made, stream = [], [], Stream()

    class Under:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            under.append(self.s)

        def __exit__(self, *a):
            under.pop()

    real = torch.empty

    def empty(shape, dtype=None, device=None):
        made.append(under[-1] if under else None)
        t = Gpu(1)
        t.t = real(shape, dtype=dtype)
        return t

    out = {"mamba2_chunk_cumsum": ["G"], "mamba2_state_pass": ["chunk_states", "final_state"], "mamba2_chunk_out": ["y"],
           "mamba2_ssd_fwd": ["y", "final_state", "workspace"], "mamba2_ssd_fwd_noalloc": ["y", "final_state"],
           "mamba2_ssd_step": ["y", "state_out"]}[name]
    t = tensors([n for n in CALLS[name].split() if n not in out], {})
    if name == "mamba2_ssd_step":
        for n in ("x", "dt", "B", "C"):
            t[n].t = t[n].t[:, 0].contiguous()
            t[n].shape = t[n].t.shape
    else:
        t["chunk_size"] = 4
    monkeypatch.setattr(torch.cuda, "stream", Under)
    monkeypatch.setattr(torch, "empty", empty)
    getattr(bd, name)(**t, stream=stream)
    assert made == [stream] * len(out) and not under
