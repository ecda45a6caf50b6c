"""The attention block's calls run with their tensors' device current, on that device's current
stream, whichever device the caller has current (a stand-in for the binding and for two devices)."""

import contextlib

import pytest
import torch

import precision_gemm_amd as P
from precision_gemm_amd import attention


class On1(torch.Tensor):
    """A tensor that says it is on device 1."""
    device = property(lambda self: torch.device("cuda", 1))


CALLS = {
    "qk_norm_rope": lambda x: P.qk_norm_rope(x, None, 1, 1, 64),
    "qk_norm_rope_backward": lambda x: P.qk_norm_rope_backward(None, None, x, x, x),
    "rope_append_kv": lambda x: P.rope_append_kv(x, None, x, x, x, 1),
    "tree_mask": lambda x: P.tree_mask(x, x, 1),
    "tree_attention": lambda x: P.tree_attention(x, x, x, x, x, x, 1),
}


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
    monkeypatch.setattr(attention, "_c", Binding)
    monkeypatch.setattr(attention, "_raw_stream", lambda index: 100 + index)
    monkeypatch.setattr(attention, "_current_device", lambda: state["device"], raising=False)
    x = torch.zeros(2, 64).as_subclass(On1)
    assert CALLS[name](x) == "outputs"
    assert seen == [(name, 1, 101)] and state["device"] == current
