"""Python binding of the attention block of include/lora_lowp.h, on torch device tensors:
head norms with rotation, the append to a paged cache, and attention for drafted trees.

Argument marshalling only, as in :mod:`precision_gemm_amd.ops`.  Every call enqueues on the
current stream of its tensors' device and synchronises nothing.
"""

from __future__ import annotations

import math

import torch

from ._lib import check, lib

LORA_KV_BF16 = 0
LORA_KV_FP8_E4M3 = 1
LORA_ATTN_BAD_POSITION = 1
LORA_ATTN_BAD_SLOT = 2
LORA_ATTN_BAD_PAGE = 4
LORA_ATTN_BAD_LENGTH = 8
LORA_ATTN_BAD_PARENT = 16

_BF16, _F32, _I32, _I64, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8
_KV_FMT = {torch.bfloat16: LORA_KV_BF16, torch.float8_e4m3fn: LORA_KV_FP8_E4M3}


def _stream(dev: torch.device) -> int:
    return torch.cuda.current_stream(dev).cuda_stream


def _need(t: torch.Tensor, name: str, dtype, shape: tuple, dev: torch.device) -> int:
    """Address of a dense device tensor of this type and shape."""
    if t.dtype is not dtype:
        raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _opt(t, name, dtype, shape, dev) -> int | None:
    return None if t is None else _need(t, name, dtype, shape, dev)


def _rows(t: torch.Tensor, name: str, width: int, T: int, dev: torch.device) -> tuple:
    """Address and row stride of bf16 rows [T, width] (or [T, heads, D]) whose values are
    dense within a row."""
    if t.dtype is not _BF16:
        raise ValueError(f"{name} must have dtype torch.bfloat16, got {t.dtype}")
    if t.device != dev or dev.type != "cuda":
        raise ValueError(f"{name} must be a device tensor on {dev}")
    if t.dim() < 2 or t.shape[0] != T or t.shape[1:].numel() != width:
        raise ValueError(f"{name} must be {T} rows of {width} values, got {list(t.shape)}")
    st = t.stride()
    if T and (st[-1] != 1 or (t.dim() == 3 and t.shape[1] > 1 and st[1] != t.shape[2]) or t.dim() > 3):
        raise ValueError(f"{name} must be dense within each row")
    return t.data_ptr(), st[0] if T > 1 else width


def _rope(positions, cos_sin, q_weight, k_weight, T, D, dev) -> tuple:
    """(positions, cos_sin, max_pos, rot, q_weight, k_weight) as the C ABI takes them."""
    if (q_weight is None) != (k_weight is None):
        raise ValueError("q_weight and k_weight go together")
    if cos_sin is None:
        mp = rot = 0
        pos = cs = None
    else:
        if cos_sin.dim() != 2:
            raise ValueError("cos_sin must be [positions, rot]")
        mp, rot = cos_sin.shape
        cs = _need(cos_sin, "cos_sin", _F32, (mp, rot), dev)
        pos = _need(positions, "positions", _I32, (T,), dev)
    return (pos, cs, mp, rot, _opt(q_weight, "q_weight", _F32, (D,), dev), _opt(k_weight, "k_weight", _F32, (D,), dev))


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
    be the heads' own places in ``qkv``)."""
    T, D, dev = qkv.shape[0], head_dim, qkv.device
    src, ld = _rows(qkv, "qkv", (n_q + 2 * n_kv) * D, T, dev)
    pos, cs, mp, rot, qw, kw = _rope(positions, cos_sin, q_weight, k_weight, T, D, dev)
    if q_out is None:
        q_out = torch.empty((T, n_q, D), dtype=_BF16, device=dev)
    if k_out is None:
        k_out = torch.empty((T, n_kv, D), dtype=_BF16, device=dev)
    qo, ldq = _rows(q_out, "q_out", n_q * D, T, dev)
    ko, ldk = _rows(k_out, "k_out", n_kv * D, T, dev)
    st = lib().lora_qk_norm_rope(src, ld, pos, T, n_q, n_kv, D, cs, mp, rot, interleaved, qw, kw, eps, qo, ldq, ko, ldk,
                                 _opt(status, "status", _I32, (1,), dev), _stream(dev))
    if st:
        check("lora_qk_norm_rope", st)
    return q_out, k_out


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
    T, n_q, D = dq.shape
    n_kv, dev = dk.shape[1], dq.device
    if dev.type != "cuda":
        raise ValueError("dq must be a device tensor")
    width = (n_q + 2 * n_kv) * D
    g = (_need(dq, "dq", _BF16, (T, n_q, D), dev), _need(dk, "dk", _BF16, (T, n_kv, D), dev),
         _opt(dv, "dv", _BF16, (T, n_kv, D), dev))
    pos, cs, mp, rot, qw, kw = _rope(positions, cos_sin, q_weight, k_weight, T, D, dev)
    src, ld = (None, width) if q_weight is None else _rows(qkv, "qkv", width, T, dev)
    if dqkv is None:
        if dv is None:
            raise ValueError("without dv, dqkv has to be given (its value columns are not written)")
        dqkv = torch.empty((T, width), dtype=_BF16, device=dev)
    dst, ldd = _rows(dqkv, "dqkv", width, T, dev)
    ws, wsb, dqw, dkw = None, 0, None, None
    if q_weight is not None:
        if dq_weight is None:
            dq_weight = torch.empty(D, dtype=_F32, device=dev)
        if dk_weight is None:
            dk_weight = torch.empty(D, dtype=_F32, device=dev)
        dqw, dkw = _need(dq_weight, "dq_weight", _F32, (D,), dev), _need(dk_weight, "dk_weight", _F32, (D,), dev)
        if workspace is None:
            workspace = torch.empty(max(16, qk_norm_rope_backward_workspace_bytes(T, D)), dtype=_U8, device=dev)
        wsb = workspace.numel()
        ws = _need(workspace, "workspace", _U8, (wsb,), dev)
    st = lib().lora_qk_norm_rope_backward(src, ld, pos, *g, T, n_q, n_kv, D, cs, mp, rot, interleaved, qw, kw, eps, dst,
                                          ldd, dqw, dkw, _opt(status, "status", _I32, (1,), dev), ws, wsb, _stream(dev))
    if st:
        check("lora_qk_norm_rope_backward", st)
    return dqkv, (dq_weight if dqw else None), (dk_weight if dkw else None)


def _cache(k_cache, v_cache, k_scale, v_scale, dev) -> tuple:
    """(format, k, v, k_scale, v_scale, n_pages, n_kv, page_size, D) of a paged cache."""
    fmt = _KV_FMT.get(k_cache.dtype)
    if fmt is None or k_cache.dim() != 4:
        raise ValueError("k_cache must be [pages, kv heads, page size, head_dim] in bfloat16 or float8_e4m3fn")
    n_pages, n_kv, page, D = k_cache.shape
    k = _need(k_cache, "k_cache", k_cache.dtype, k_cache.shape, dev)
    v = _need(v_cache, "v_cache", k_cache.dtype, k_cache.shape, dev)
    if fmt == LORA_KV_BF16:
        if k_scale is not None or v_scale is not None:
            raise ValueError("k_scale and v_scale are for an 8-bit cache")
        return fmt, k, v, None, None, n_pages, n_kv, page, D
    if k_scale is None or v_scale is None:
        raise ValueError("an 8-bit cache needs k_scale and v_scale")
    return (fmt, k, v, _need(k_scale, "k_scale", _F32, (n_kv,), dev), _need(v_scale, "v_scale", _F32, (n_kv,), dev),
            n_pages, n_kv, page, D)


def rope_append_kv(qkv: torch.Tensor, positions: torch.Tensor | None, slots: torch.Tensor, k_cache: torch.Tensor,
                   v_cache: torch.Tensor, n_q: int, *, cos_sin=None, q_weight=None, k_weight=None, eps: float = 1e-6,
                   interleaved: bool = False, k_scale=None, v_scale=None, q_out=None, status=None) -> torch.Tensor:
    """Keys and values of ``qkv`` into a paged cache (lora_rope_append_kv), the norm and rotation
    of :func:`qk_norm_rope` applied on the way; returns the queries, bf16 [T, n_q, D].  ``k_cache``
    and ``v_cache`` [pages, kv heads, page size, D], bfloat16 or float8_e4m3fn (then ``k_scale`` and
    ``v_scale`` float32 [kv heads]); ``slots`` int32 [T], page * page size + offset (negative: not
    stored)."""
    T, dev = qkv.shape[0], qkv.device
    fmt, k, v, ks, vs, n_pages, n_kv, page, D = _cache(k_cache, v_cache, k_scale, v_scale, dev)
    src, ld = _rows(qkv, "qkv", (n_q + 2 * n_kv) * D, T, dev)
    pos, cs, mp, rot, qw, kw = _rope(positions, cos_sin, q_weight, k_weight, T, D, dev)
    if q_out is None:
        q_out = torch.empty((T, n_q, D), dtype=_BF16, device=dev)
    qo, ldq = _rows(q_out, "q_out", n_q * D, T, dev)
    st = lib().lora_rope_append_kv(src, ld, pos, _need(slots, "slots", _I32, (T,), dev), T, n_q, n_kv, D, cs, mp, rot,
                                   interleaved, qw, kw, eps, qo, ldq, fmt, k, v, ks, vs, n_pages, page,
                                   _opt(status, "status", _I32, (1,), dev), _stream(dev))
    if st:
        check("lora_rope_append_kv", st)
    return q_out


def tree_mask(parents: torch.Tensor, q_indptr: torch.Tensor, max_q: int, *, status=None) -> torch.Tensor:
    """Masks of drafted trees from their parents (lora_tree_mask): ``parents`` int32 [T] (index
    among the sequence's own drafted tokens, -1: none) -> int64 [T, ceil(max_q / 64)]."""
    T, dev = parents.shape[0], parents.device
    if dev.type != "cuda":
        raise ValueError("parents must be a device tensor")
    B, words = q_indptr.shape[0] - 1, max(1, (max_q + 63) // 64)
    mask = torch.empty((T, words), dtype=_I64, device=dev)
    st = lib().lora_tree_mask(_need(parents, "parents", _I32, (T,), dev), _need(q_indptr, "q_indptr", _I32, (B + 1,), dev),
                              B, T, max_q, words, mask.data_ptr(), _opt(status, "status", _I32, (1,), dev), _stream(dev))
    if st:
        check("lora_tree_mask", st)
    return mask


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
    [T, n_q, D] and float32 [T, n_q].  With ``workspace`` (uint8, any content, at least
    :func:`tree_attention_workspace_bytes`; calls that overlap in time need their own), ``out`` and
    ``lse`` passed in the call allocates nothing."""
    T, n_q, D = q.shape
    dev = q.device
    fmt, k, v, ks, vs, n_pages, n_kv, page, Dc = _cache(k_cache, v_cache, k_scale, v_scale, dev)
    if Dc != D:
        raise ValueError(f"q has heads of {D} values, the cache of {Dc}")
    src, ldq = _rows(q, "q", n_q * D, T, dev)
    B = kv_len.shape[0]
    if page_table.dim() != 2:
        raise ValueError("page_table must be [sequences, max pages]")
    mp = page_table.shape[1]
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    mask, words = None, 0
    if tree_mask is not None:
        if tree_mask.dtype not in (_I64, torch.uint64) or tree_mask.dim() != 2:
            raise ValueError("tree_mask must be int64 or uint64 [tokens, words]")
        words = tree_mask.shape[1]
        mask = _need(tree_mask, "tree_mask", tree_mask.dtype, (T, words), dev)
    if out is None:
        out = torch.empty((T, n_q, D), dtype=_BF16, device=dev)
    if lse is None:
        lse = torch.empty((T, n_q), dtype=_F32, device=dev)
    if workspace is None:
        workspace = torch.empty(max(16, tree_attention_workspace_bytes(n_q, n_kv, D, max_q)), dtype=_U8, device=dev)
    wsb = workspace.numel()
    st = lib().lora_tree_attention(src, ldq, fmt, k, v, ks, vs, n_pages, page,
                                   _need(page_table, "page_table", _I32, (B, mp), dev), mp,
                                   _need(kv_len, "kv_len", _I32, (B,), dev),
                                   _need(q_indptr, "q_indptr", _I32, (B + 1,), dev), B, T, max_q, n_q, n_kv, D, mask, words,
                                   scale, _need(out, "out", _BF16, (T, n_q, D), dev), _need(lse, "lse", _F32, (T, n_q), dev),
                                   _opt(status, "status", _I32, (1,), dev), _need(workspace, "workspace", _U8, (wsb,), dev),
                                   wsb, _stream(dev))
    if st:
        check("lora_tree_attention", st)
    return out, lse
