"""The norms' and the AdamW step's calls run with their tensors' device current, on that device's current
stream, whichever device the caller has current (a stand-in for the binding and for two devices)."""

import contextlib
import types

import pytest
import torch

import precision_gemm_amd as P
from precision_gemm_amd import _binding


class On1(torch.Tensor):
    """A tensor that says it is on device 1."""
    device = property(lambda self: torch.device("cuda", 1))


def _step(x):
    opt = types.SimpleNamespace(tiles=x, group_first=x, state_bits=32, steps=x, workspace=x)
    return P.adamw_step(opt, x)


CALLS = {"layer_norm": lambda x: P.layer_norm(x), "layer_norm_backward": lambda x: P.layer_norm_backward(x, x), "adamw_step": _step}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("current", [0, 1])
def test_device_of_the_tensors(monkeypatch, name, current):
    state, seen = {"device": current}, []

    @contextlib.contextmanager
    def device(index):
        was, state["device"] = state["device"], index
        try:
            yield
        finally:
            state["device"] = was

    class Binding:
        def __getattr__(self, call):
            return lambda *args: seen.append((call, state["device"], args[-1])) or "outputs"

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(_binding, "binding", Binding)
    monkeypatch.setattr(_binding, "_raw_stream", lambda index: 100 + index)
    monkeypatch.setattr(_binding, "_current_device", lambda: state["device"])
    x = torch.zeros(2, 64).as_subclass(On1)
    assert CALLS[name](x) == "outputs"
    assert seen == [(name, 1, 101)] and state["device"] == current


def test_status_is_raised(monkeypatch):
    monkeypatch.setattr(_binding, "binding", lambda: types.SimpleNamespace(layer_norm=lambda *a: 2))
    with pytest.raises(RuntimeError, match="lora_layer_norm failed with status 2"):
        P.layer_norm(torch.zeros(2, 64))


class Large(torch.Tensor):
    """A tensor that says it is on device 1, and has no memory behind it."""
    device = property(lambda self: torch.device("cuda", 1))
    is_cuda = property(lambda self: True)


@pytest.mark.parametrize("n, group, n_groups, match", [
    (2**32 + 64, 0, 1, "values"),             # of which 32 bits hold 64
    (2**31 - 4096, 0, 1, "values"),
    (64, 2**32, 1, "group"),                  # of which they hold 0
    (64, 0, 2**32 + 1, "n_groups"),
])
def test_numbers_behind_32_bits(n, group, n_groups, match):
    x = torch.empty(n, dtype=torch.float32, device="meta").as_subclass(Large)
    with pytest.raises(ValueError, match=match):
        P.AdamW([P.AdamWTensor(x, x, group)], n_groups)
