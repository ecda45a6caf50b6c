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
