"""Calls of the compiled binding ``_step.so`` (csrc_step/binding.cpp) on the stream and device of
their tensors."""

from __future__ import annotations

import importlib
import os

import torch

from ._lib import HERE, check, lib

_binding = None
_raw_stream = torch._C._cuda_getCurrentRawStream  # current_stream() wraps it in an object: 2 us a call
_current_device = torch._C._cuda_getDevice


def binding():
    global _binding
    if _binding is None:
        lib()  # says how to build what is missing
        if not os.path.exists(os.path.join(HERE, "_step.so")):
            raise RuntimeError(f"{HERE}/_step.so is not built; run `python -m precision_gemm_amd.build`")
        _binding = importlib.import_module("precision_gemm_amd._step")
    return _binding


def call(name: str, on, *args):
    """The binding's call ``name`` on the current stream of the device of tensor ``on``, with that
    device current: the handle of a default stream is 0 on every device.  (What is no device tensor
    the binding refuses.)  Returns the outputs; the binding returns the library's status where it is
    an error."""
    f = getattr(binding(), name)
    index = on.device.index if isinstance(on, torch.Tensor) else None
    if index is None:
        result = f(*args, 0)
    elif index == _current_device():
        result = f(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            result = f(*args, _raw_stream(index))
    if type(result) is int:
        check("lora_" + name, result)
    return result
