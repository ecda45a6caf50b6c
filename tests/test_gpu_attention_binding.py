"""Errors of the attention block's Python calls that come only with tensors on a device."""

import pytest

pytestmark = pytest.mark.gpu


def _rope(T=3, n_q=2, n_kv=1, D=64):
    import torch
    qkv = torch.zeros((T, (n_q + 2 * n_kv) * D), dtype=torch.bfloat16, device="cuda")
    return qkv, torch.zeros(T, dtype=torch.int32, device="cuda"), n_q, n_kv, D


@pytest.mark.parametrize("value", ["a tensor", "an array"])
def test_interleaved_has_to_be_a_truth_value(value):
    """What has no truth value is refused by name (it passed as False, with Python's error left set)."""
    import numpy as np
    import torch
    import precision_gemm_amd as P
    print("[case] interleaved", value, flush=True)
    what = torch.ones(2) if value == "a tensor" else np.ones(2)
    qkv, pos, n_q, n_kv, D = _rope()
    cs = P.rope_table(4, D)
    with pytest.raises(ValueError, match="interleaved"):
        P.qk_norm_rope(qkv, pos, n_q, n_kv, D, cos_sin=cs, interleaved=what)
    dq, dk = (torch.zeros((3, n, D), dtype=torch.bfloat16, device="cuda") for n in (n_q, n_kv))
    with pytest.raises(ValueError, match="interleaved"):
        P.qk_norm_rope_backward(qkv, pos, dq, dk, dk, cos_sin=cs, interleaved=what)
    cache = torch.zeros((1, n_kv, 16, D), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="interleaved"):
        P.rope_append_kv(qkv, pos, pos, cache, cache.clone(), n_q, cos_sin=cs, interleaved=what)
    q, _ = P.qk_norm_rope(qkv, pos, n_q, n_kv, D, cos_sin=cs, interleaved=np.bool_(True))
    assert q.shape == (3, n_q, D)


def test_out_of_memory():
    """Buffers that do not fit raise torch's own error, as every allocation of its does."""
    import torch
    import precision_gemm_amd as P
    print("[case] out of memory", flush=True)
    total = torch.cuda.mem_get_info()[1]
    q = torch.zeros((16384, 8, 256), dtype=torch.bfloat16, device="cuda")
    cache = torch.zeros((1, 1, 16, 256), dtype=torch.bfloat16, device="cuda")
    one, two = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (1, 2))
    torch.cuda.empty_cache()
    try:
        torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (8 << 20)) / total)
        with pytest.raises(torch.cuda.OutOfMemoryError):
            P.tree_attention(q, cache, cache, one.view(1, 1), one, two, 1)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
