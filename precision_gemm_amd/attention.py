"""The attention block of include/lora_lowp.h on torch device tensors: head norms with rotation,
the append to a paged cache, and attention for drafted trees.

The arguments are checked and marshalled by a compiled binding (csrc_attn/binding.cpp), built
with the library by ``precision_gemm_amd.build``.  Every call enqueues on the current stream of
its tensors' device, whichever device is current, and synchronises nothing.  They are no operations
of autograd: outputs have no graph, whatever requires gradients among the inputs (the gradients of
:func:`qk_norm_rope` are :func:`qk_norm_rope_backward`; the attention has none here), and buffers and
caches are written without autograd's version counters.
"""

from __future__ import annotations

import importlib
import math
import os

import torch

from ._lib import HERE, check, lib

LORA_KV_BF16 = 0
LORA_KV_FP8_E4M3 = 1
LORA_ATTN_BAD_POSITION = 1
LORA_ATTN_BAD_SLOT = 2
LORA_ATTN_BAD_PAGE = 4
LORA_ATTN_BAD_LENGTH = 8
LORA_ATTN_BAD_PARENT = 16

_binding = None
_raw_stream = torch._C._cuda_getCurrentRawStream  # current_stream() wraps it in an object: 2 us a call
_current_device = torch._C._cuda_getDevice


def _c():
    global _binding
    if _binding is None:
        lib()  # says how to build what is missing
        if not os.path.exists(os.path.join(HERE, "_attn.so")):
            raise RuntimeError(f"{HERE}/_attn.so is not built; run `python -m precision_gemm_amd.build`")
        _binding = importlib.import_module("precision_gemm_amd._attn")
    return _binding


def _call(name: str, on, *args):
    """The binding's call ``name`` on the current stream of the device of tensor ``on``, with that
    device current: the handle of a default stream is 0 on every device.  (What is no device tensor
    the binding refuses.)  Returns the outputs; the binding returns the library's status where it is
    an error."""
    f = getattr(_c(), name)
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


def rope_table(max_pos: int, rot: int, theta: float = 10000.0, device="cuda") -> torch.Tensor:
    """The rotation table of the calls below, float32 [max_pos, rot]: for each position the
    rot / 2 cosines of position * theta^(-2 i / rot), then the sines.  Computed once, in 64 bits."""
    f = theta ** (-torch.arange(rot // 2, dtype=torch.float64) * 2.0 / rot)
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * f[None, :]
    return torch.cat([a.cos(), a.sin()], 1).to(torch.float32).to(device)


def qk_norm_rope(qkv: torch.Tensor, positions: torch.Tensor | None, n_q: int, n_kv: int, head_dim: int, *, cos_sin=None,
                 q_weight=None, k_weight=None, eps: float = 1e-6, interleaved: bool = False, q_out=None, k_out=None,
                 status=None):
    """Norms of the query and key heads and their rotation (lora_qk_norm_rope).  ``qkv`` bf16
    [T, (n_q + 2 n_kv) head_dim], rows of any stride; ``cos_sin`` from :func:`rope_table` (None: no
    rotation), ``q_weight`` and ``k_weight`` float32 [head_dim] (None: no norm).  Returns ``(q, k)``,
    bf16 [T, n_q, head_dim] and [T, n_kv, head_dim], in ``q_out`` and ``k_out`` if given (which may
    be the heads' own places in ``qkv``); without a graph of autograd."""
    return _call("qk_norm_rope", qkv, qkv, positions, n_q, n_kv, head_dim, cos_sin, q_weight, k_weight, eps, interleaved,
                 q_out, k_out, status)


def qk_norm_rope_backward_workspace_bytes(T: int, head_dim: int) -> int:
    """Bytes of the workspace lora_qk_norm_rope_backward needs when there are weights."""
    return int(lib().lora_qk_norm_rope_backward_workspace_bytes(T, head_dim))


def qk_norm_rope_backward(qkv: torch.Tensor | None, positions: torch.Tensor | None, dq: torch.Tensor, dk: torch.Tensor,
                          dv: torch.Tensor | None, *, cos_sin=None, q_weight=None, k_weight=None, eps: float = 1e-6,
                          interleaved: bool = False, dqkv=None, dq_weight=None, dk_weight=None, workspace=None,
                          status=None):
    """Gradients of :func:`qk_norm_rope` (lora_qk_norm_rope_backward): ``dq`` bf16 [T, n_q, D] and
    ``dk`` [T, n_kv, D] -> ``(dqkv, dq_weight, dk_weight)``: bf16 [T, (n_q + 2 n_kv) D], the dY of
    :func:`lora_backward`, and float32 [D] (None without weights).  ``dv`` is copied to its place;
    with ``dv=None`` those columns of ``dqkv`` are left as they are (so ``dqkv`` has to be given).
    Output buffers and the workspace may be passed in; then the call allocates nothing."""
    return _call("qk_norm_rope_backward", dq, qkv, positions, dq, dk, dv, cos_sin, q_weight, k_weight, eps, interleaved, dqkv,
                 dq_weight, dk_weight, workspace, status)


def rope_append_kv(qkv: torch.Tensor, positions: torch.Tensor | None, slots: torch.Tensor, k_cache: torch.Tensor,
                   v_cache: torch.Tensor, n_q: int, *, cos_sin=None, q_weight=None, k_weight=None, eps: float = 1e-6,
                   interleaved: bool = False, k_scale=None, v_scale=None, q_out=None, status=None) -> torch.Tensor:
    """Keys and values of ``qkv`` into a paged cache (lora_rope_append_kv), the norm and rotation
    of :func:`qk_norm_rope` applied on the way; returns the queries, bf16 [T, n_q, D].  ``k_cache``
    and ``v_cache`` [pages, kv heads, page size, D], bfloat16 or float8_e4m3fn (then ``k_scale`` and
    ``v_scale`` float32 [kv heads]); ``slots`` int32 [T], page * page size + offset (negative: not
    stored)."""
    return _call("rope_append_kv", qkv, qkv, positions, slots, k_cache, v_cache, n_q, cos_sin, q_weight, k_weight, eps,
                 interleaved, k_scale, v_scale, q_out, status)


def tree_mask(parents: torch.Tensor, q_indptr: torch.Tensor, max_q: int, *, status=None) -> torch.Tensor:
    """Masks of drafted trees from their parents (lora_tree_mask): ``parents`` int32 [T] (index
    among the sequence's own drafted tokens, -1: none) -> int64 [T, ceil(max_q / 64)]."""
    return _call("tree_mask", parents, parents, q_indptr, max_q, status)


def tree_attention_workspace_bytes(n_q: int, n_kv: int, head_dim: int, max_q: int) -> int:
    """Bytes of the workspace lora_tree_attention needs for any batch of such heads."""
    return int(lib().lora_tree_attention_workspace_bytes(n_q, n_kv, head_dim, max_q))


def tree_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
                   kv_len: torch.Tensor, q_indptr: torch.Tensor, max_q: int, *, tree_mask=None, scale=None, k_scale=None,
                   v_scale=None, out=None, lse=None, workspace=None, status=None):
    """Attention over a paged cache for the tokens just appended to it (lora_tree_attention).

    ``q`` bf16 [T, n_q, D]; ``page_table`` int32 [B, max pages], ``kv_len`` int32 [B] (the drafted
    tokens included), ``q_indptr`` int32 [B + 1], ``max_q`` at least every sequence's drafted tokens;
    ``tree_mask`` int64 or uint64 [T, words] (None: in order).  Returns ``(out, lse)``, bf16
    [T, n_q, D] and float32 [T, n_q]; rows that no sequence has are 0 and -inf.  With ``workspace``
    (uint8, any content, at least :func:`tree_attention_workspace_bytes`; calls that overlap in time
    need their own), ``out`` and ``lse`` passed in the call allocates nothing.  The outputs have no graph of autograd."""
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    return _call("tree_attention", q, q, k_cache, v_cache, page_table, kv_len, q_indptr, max_q, tree_mask, scale, k_scale,
                 v_scale, out, lse, workspace, status)
