"""CPU checks of what the binding of the recurrent block's operators says of a wrong call."""
import pytest
import torch

from mamba_chunked_ssd_gb300 import binding as bd
from test_gated_delta_binding import Gpu, Recorder


@pytest.fixture
def rec(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(bd, "load_library", lambda: r)
    monkeypatch.setattr(bd, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(bd, "_current_gpu", lambda: 0, raising=False)
    return r


@pytest.mark.parametrize("wrong", [Gpu(2, 5, 4), Gpu(2, 5, 8, dtype=torch.bfloat16), Gpu(2, 5, 8, device=1)])
def test_a_wrong_gradient_of_y_is_named_as_it_was_given(rec, wrong):
    x, A = Gpu(2, 5, 8), Gpu(8)
    with pytest.raises(ValueError, match="^dy must be"):
        bd.mamba2_glr_bwd(wrong, x, x, x, A, Gpu(2, 1, 8))
    with pytest.raises(ValueError, match="^y must be"):
        bd.mamba2_glr_fwd(x, x, x, A, y=wrong)
    rows = Gpu(2, 5, 9)
    rows.t = rows.t[..., ::2][..., :4]
    rows.shape = rows.t.shape
    q = Gpu(2, 5, 4)
    with pytest.raises(ValueError, match="^dy: "):
        bd.mamba2_glr_bwd(rows, q, q, q, Gpu(4), Gpu(2, 1, 4))
    assert rec.calls == []
