"""An AdamW step over many tenants' adapters at once (lora_adamw_step of include/lora_lowp.h): from
the gradients that ``lora_backward`` leaves to the adapters in the forms that the layer and its
backward read, in a few launches for all tensors.

Each tensor belongs to a group, a tenant, with its own rates, step count and gradient norm.  Master
copies are float32; states float32, or 8 bits with a scale for each 64 values.  A step writes its
buffers in place, without autograd's version counters.
"""

from __future__ import annotations

import ctypes
from dataclasses import dataclass

import numpy as np
import torch

from ._binding import call
from ._lib import AdamWTensorStruct, check, lib
from .ops import Adapters, BackwardAdapters, Grads, a_rows, rank_pad

LORA_ADAMW_NOT_FINITE = 1
_KIND = {"plain": 0, "A": 1, "B": 2}
_BLOCK = 64
_MOST_VALUES = 2**31 - 4097  # lora_adamw_tensor


def _int32(n: int) -> bool:  # ctypes keeps the low bits of what is larger
    return -2**31 <= n < 2**31


@dataclass
class AdamWTensor:
    """One tensor of a step.  ``param`` and ``grad`` float32 of one shape; ``kind`` "A" ([K, r]), "B"
    ([r, N]) or "plain" (any shape).  ``copy`` (bf16, of that shape) and, for A and B, ``pack`` (At or
    Bt of :func:`pack_adapter`) and ``pack_bwd`` (Ar or Bop of :func:`pack_adapters_bwd`) receive the
    updated values if given.  States ``m`` and ``v`` are made, as zeros, where they are None: float32 of
    that shape, or float8_e4m3fn with ``m_scale`` and ``v_scale`` float32 [ceil(values / 64)] (m = code *
    scale, sqrt(v) = code * scale)."""

    param: torch.Tensor
    grad: torch.Tensor
    group: int = 0
    kind: str = "plain"
    copy: torch.Tensor | None = None
    pack: torch.Tensor | None = None
    pack_bwd: torch.Tensor | None = None
    m: torch.Tensor | None = None
    v: torch.Tensor | None = None
    m_scale: torch.Tensor | None = None
    v_scale: torch.Tensor | None = None


def adamw_adapters(ad: Adapters, grads: Grads, bw: BackwardAdapters | None = None, group0: int = 0) -> list:
    """The tensors of one projection's adapters: adapter a in group ``group0 + a``, master copies made
    from ``ad.A`` and ``ad.B``.  A step updates those, ``ad``'s packed forms and, if given, ``bw``'s."""
    out = []
    for a, (A, B) in enumerate(zip(ad.A, ad.B)):
        out.append(AdamWTensor(A.float(), grads.dA[a], group0 + a, "A", A, ad.At[a], bw.Ar[a] if bw else None))
        out.append(AdamWTensor(B.float(), grads.dB[a], group0 + a, "B", B, ad.Bt[a], bw.Bop[a] if bw else None))
    return out


def _check(t: torch.Tensor, name: str, dtype, numel: int, dev) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if t.numel() != numel:
        raise ValueError(f"{name} must have {numel} values, got {t.numel()}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


class AdamW:
    """The tensors of a step with their states, cut into tiles once (lora_adamw_plan); the handle of
    :func:`adamw_step`.  ``steps`` int32 [n_groups] holds the steps that each group has made (zeros if
    not given).  The handle holds the addresses of its tensors' buffers, and keeps their memory for as long
    as it lives: gradients are written into those (``lora_backward`` does), and what a field or a tensor
    of ``tensors`` is given in their place afterwards is not seen (a new handle is needed for it, as for
    adapters that are packed into new buffers).
    Calls on one handle must be ordered on one stream: they share its states and workspace."""

    def __init__(self, tensors: list, n_groups: int, *, state_bits: int = 32, steps: torch.Tensor | None = None):
        if state_bits not in (32, 8):
            raise ValueError("state_bits must be 32 or 8")
        if not _int32(n_groups):
            raise ValueError(f"n_groups must be an int32, got {n_groups}")
        if not tensors:
            raise ValueError("a step needs a tensor at least")
        self.tensors, self.n_groups, self.state_bits = list(tensors), int(n_groups), state_bits
        if not isinstance(self.tensors[0].param, torch.Tensor) or not self.tensors[0].param.is_cuda:
            raise ValueError("param must be a device tensor")
        dev = self.device = self.tensors[0].param.device
        # memory whose addresses the plan holds: the tensors' fields are the caller's, who may replace them
        self._memory = []
        structs = (AdamWTensorStruct * len(self.tensors))()
        for t, s in zip(self.tensors, structs):
            self._fill(t, s, dev)
        n_tiles = ctypes.c_int64()
        plan = lambda tiles, first: check("lora_adamw_plan", lib().lora_adamw_plan(  # noqa: E731
            structs, len(self.tensors), self.n_groups, state_bits, ctypes.byref(n_tiles), tiles, first))
        plan(None, None)
        tiles = np.zeros((n_tiles.value, ctypes.sizeof(AdamWTensorStruct) + 8), np.uint8)
        first = np.zeros(self.n_groups + 1, np.int32)
        plan(tiles.ctypes.data_as(ctypes.c_void_p), first.ctypes.data_as(ctypes.c_void_p))
        up = lambda a: torch.from_numpy(a).to(dev)  # noqa: E731
        self.tiles, self.group_first = up(tiles), up(first)
        if steps is None:
            steps = torch.zeros(self.n_groups, dtype=torch.int32, device=dev)
        _check(steps, "steps", torch.int32, self.n_groups, dev)
        self.steps = steps
        self.workspace = torch.zeros(max(16, int(lib().lora_adamw_workspace_bytes(n_tiles.value, self.n_groups))),
                                     dtype=torch.uint8, device=dev)

    def _fill(self, t: AdamWTensor, s, dev) -> None:
        if t.kind not in _KIND:
            raise ValueError('kind must be "A", "B" or "plain"')
        n = t.param.numel()
        if n > _MOST_VALUES:
            raise ValueError(f"param has {n} values, and {_MOST_VALUES} at most are taken: give it in parts")
        if not _int32(t.group):
            raise ValueError(f"there is no group {t.group}")
        if t.kind == "plain":
            rows, cols = 1, n
            packs = (0, 0)
        else:
            if t.param.dim() != 2:
                raise ValueError("param must be [K, r] or [r, N]")
            rows, cols = t.param.shape
            r, side = (cols, rows) if t.kind == "A" else (rows, cols)
            packs = (a_rows(r) * side, rank_pad(r) * side) if t.kind == "A" else (rank_pad(r) * side, a_rows(r) * side)
        s.param, s.grad = _check(t.param, "param", torch.float32, n, dev), _check(t.grad, "grad", torch.float32, n, dev)
        if t.grad.shape != t.param.shape:
            raise ValueError("grad must have the shape of param")
        held = torch.float32 if self.state_bits == 32 else torch.float8_e4m3fn
        if t.m is None:
            t.m = torch.zeros(t.param.shape, dtype=torch.uint8 if self.state_bits == 8 else held, device=dev).view(held)
        if t.v is None:
            t.v = torch.zeros(t.param.shape, dtype=torch.uint8 if self.state_bits == 8 else held, device=dev).view(held)
        s.m, s.v = _check(t.m, "m", held, n, dev), _check(t.v, "v", held, n, dev)
        if self.state_bits == 8:
            blocks = -(-n // _BLOCK)
            if t.m_scale is None:
                t.m_scale = torch.zeros(blocks, dtype=torch.float32, device=dev)
            if t.v_scale is None:
                t.v_scale = torch.zeros(blocks, dtype=torch.float32, device=dev)
            s.m_scale = _check(t.m_scale, "m_scale", torch.float32, blocks, dev)
            s.v_scale = _check(t.v_scale, "v_scale", torch.float32, blocks, dev)
        elif t.m_scale is not None or t.v_scale is not None:
            raise ValueError("m_scale and v_scale are for states in 8 bits")
        if t.copy is not None:
            s.copy = _check(t.copy, "copy", torch.bfloat16, n, dev)
        for name, b, size in (("pack", t.pack, packs[0]), ("pack_bwd", t.pack_bwd, packs[1])):
            if b is not None:
                if not size:
                    raise ValueError(f"{name} is for A and B")
                setattr(s, name, _check(b, name, torch.bfloat16, size, dev))
        self._memory += [b.untyped_storage() for b in (t.param, t.grad, t.m, t.v, t.m_scale, t.v_scale, t.copy, t.pack, t.pack_bwd)
                         if b is not None]
        s.rows, s.cols, s.group, s.kind = rows, cols, t.group, _KIND[t.kind]


def adamw_step(opt: AdamW, hyper: torch.Tensor, *, active: torch.Tensor | None = None, clip: bool = False,
               grad_norm: torch.Tensor | None = None, status: torch.Tensor | None = None):
    """One step of every active group (lora_adamw_step).  ``hyper`` float64 [n_groups, 6]: rate, beta1,
    beta2, eps, weight decay, largest gradient norm (0: not clipped); ``active`` int32 [n_groups], 0
    for a group that is left as it is (a tenant without tokens in the batch).  With ``clip`` the groups'
    gradient norms are taken: gradients are clipped by them, a group whose norm is not finite is left as
    it was (LORA_ADAMW_NOT_FINITE in ``status``, int32 [1]), and the norms are returned, float32
    [n_groups] (in ``grad_norm`` if given); without it gradients are taken as they are, and None is
    returned.  Apart from the norms the call allocates nothing, and can be captured in a HIP graph."""
    return call("adamw_step", opt.tiles, opt.tiles, opt.group_first, opt.state_bits, hyper, active, opt.steps, clip,
                grad_norm, status, opt.workspace)
