"""The handle of an AdamW step keeps the memory that it writes to, whatever becomes of the caller's tensors."""

import gc

import pytest

pytestmark = pytest.mark.gpu


def _tensor(P, torch, bits, r=16, K=65536):
    t = P.AdamWTensor(torch.ones((K, r), device="cuda"), torch.ones((K, r), device="cuda"), 0, "A")
    t.copy, t.pack, t.pack_bwd = (torch.zeros((K, r), dtype=torch.bfloat16, device="cuda") for _ in range(3))
    return t


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("way", ["field", "data"])
def test_replaced_tensors(way, bits):
    """Fields that are given other tensors, and tensors that are given other memory: the handle goes on with
    what it was made of, which no later tensor is given meanwhile."""
    import torch
    import precision_gemm_amd as P
    print("[case] handle", way, bits, flush=True)
    t = _tensor(P, torch, bits)
    opt = P.AdamW([t], 1, state_bits=bits)
    fields = ["param", "grad", "copy", "pack", "pack_bwd", "m", "v"] + (["m_scale", "v_scale"] if bits == 8 else [])
    at = {getattr(t, f).data_ptr(): getattr(t, f).untyped_storage().nbytes() for f in fields}
    for f in fields:
        old = getattr(t, f)
        if way == "field":
            setattr(t, f, torch.zeros(old.shape, device="cuda").to(old.dtype))
        else:
            old.data = torch.zeros(old.shape, device="cuda").to(old.dtype)
        del old
    gc.collect()
    # memory that is free would be handed out again here
    later = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in at.values() for _ in range(4)]
    for x in later + [getattr(t, f) for f in fields]:
        assert not any(p <= x.data_ptr() < p + n for p, n in at.items()), "a buffer of the handle was given away"
    h = torch.tensor([[0.1, 0.9, 0.99, 1e-8, 0.0, 0.0]], dtype=torch.float64, device="cuda")
    P.adamw_step(opt, h)
    torch.cuda.synchronize()
    assert all((x == 7).all() for x in later)
    assert not any(getattr(t, f).float().any() for f in fields)


def test_memory_goes_with_the_handle():
    import torch
    import precision_gemm_amd as P
    gc.collect()
    before = torch.cuda.memory_allocated()
    opt = P.AdamW([_tensor(P, torch, 32)], 1)
    assert torch.cuda.memory_allocated() > before
    del opt
    gc.collect()
    assert torch.cuda.memory_allocated() == before
