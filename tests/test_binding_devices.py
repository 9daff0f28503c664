"""The calls that take torch tensors refuse those of another device than the current one, before any launch (with
stand-ins: a tensor is asked where it is, and nothing else)."""
import pytest


class Tensor:
    is_cuda = True

    def __init__(self, device):
        self.device = device

    def get_device(self):
        return self.device


@pytest.mark.parametrize("current", [0, 1])
def test_tensors_of_another_device_are_refused(monkeypatch, current):
    import activation_sparse_transformer_gb300 as tw
    tw._setup()
    monkeypatch.setattr(tw, "_device", lambda: current)
    other = 1 - current
    tw._on_device(Tensor(current), None, Tensor(current))
    tw._on_device(None)
    for tensors in ((Tensor(other),), (Tensor(current), Tensor(other)), (None, Tensor(current), Tensor(2), Tensor(current))):
        with pytest.raises(ValueError, match="current device is"):
            tw._on_device(*tensors)
    with pytest.raises(ValueError, match="CUDA"):
        tw._on_device(Tensor(current), Tensor(-1))


def test_the_norm_looks_at_every_tensor(monkeypatch):
    """Its own look at the devices is written out; each argument on another device is found."""
    import inspect

    import activation_sparse_transformer_gb300 as tw
    import torch
    tw._setup()
    monkeypatch.setattr(tw, "_device", lambda: 0)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: int(getattr(t, "elsewhere", 0)))
    bf, f32 = torch.bfloat16, torch.float32
    new = {k: torch.zeros((4, 64), dtype=bf) for k in ("x", "y", "x_out", "h")}
    new.update({k: torch.ones(64, dtype=bf) for k in ("w_post", "gate", "w_pre")})
    new.update({k: torch.zeros(4, dtype=f32) for k in ("row_gate", "rstd_post", "rstd_pre")})
    given = inspect.signature(tw.twell_block_norm).parameters
    assert set(new) == set(given) - {"skip_scale", "branch_scale", "eps", "stream"}
    for k in new:
        new[k].elsewhere = 1
        with pytest.raises(ValueError, match="a tensor on device 1, the current device is 0"):
            tw.twell_block_norm(**new)
        new[k].elsewhere = 0
