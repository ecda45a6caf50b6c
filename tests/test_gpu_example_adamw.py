"""The example's training by AdamW: it runs, the call leaves the adapters packed as their masters are, the
tenant without tokens is as it was, and the first step is the oracle's."""

import importlib.util
import os

import numpy as np
import pytest

from oracle import step as S

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("attention_block_example", os.path.join(ROOT, "examples", "attention_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("bits", [32, 8])
def test_training_by_adamw(bits):
    import torch
    import precision_gemm_amd as P
    print("[case] example adamw", bits, flush=True)
    ex = _example()
    block = ex.AttentionBlock(256, 4, 2, 64, [5, 16, 33], max_pos=128, train=True)
    lens = [40, 7, 33]
    x, target, _ = ex.training_batch(block, lens, 3)
    ids = torch.tensor([b % 2 * 2 for b, n in enumerate(lens) for _ in range(n)], dtype=torch.int32, device="cuda")  # 0 and 2
    parts = [(p.A + p.B, p.ad.A + p.ad.B) for p in (block.qkv, block.o)]
    before = [[m.clone() for m in p.A + p.B] for p in (block.qkv, block.o)]
    weights = [block.q_weight.clone(), block.k_weight.clone()]
    _, grads, _ = ex.train_step(block, x, target, ids, lens)
    losses, opt = ex.train_adamw(block, x, target, ids, lens, steps=1, rate=1e-3, state_bits=bits)
    assert opt.steps.tolist() == [1, 0, 1, 1] and np.isfinite(losses).all()
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    norms = np.zeros(4)
    for name in ("qkv", "o"):
        for a in range(3):
            norms[a] += sum((f64(grads[name + k][a]) ** 2).sum() for k in ("_A", "_B"))
    norms[3] = (f64(grads["q_weight"]) ** 2).sum() + (f64(grads["k_weight"]) ** 2).sum()
    norms = np.sqrt(norms)

    def check(now, was, g, group):
        # the update is rate g / (|g| + eps) at the first step: 2^-20 of the rate, p's own rounding 2^-22
        g = f64(g) * S.clip_factor(norms[group], 1.0)
        want, _, _ = S.adamw(f64(was), g, 0 * g, 0 * g, 1, 1e-3, 0.9, 0.999, 1e-8, 0.01)
        tol = 2.0 ** -22 * np.abs(want) + 2.0 ** -19 * 1e-3
        assert (np.abs(f64(now) - want) <= tol).all(), group

    for (masters, copies), was, name in zip(parts, before, ("qkv", "o")):
        for k in range(6):
            a = k % 3
            if a == 1:
                assert torch.equal(masters[k], was[k])
            else:
                check(masters[k], was[k], grads[name + ("_A" if k < 3 else "_B")][a], a)
            assert torch.equal(copies[k], masters[k].bfloat16())
    check(block.q_weight, weights[0], grads["q_weight"], 3)
    check(block.k_weight, weights[1], grads["k_weight"], 3)
    for p in (block.qkv, block.o):
        fresh = P.Adapters([a.bfloat16() for a in p.A], [b.bfloat16() for b in p.B], torch.ones(3, device="cuda"))
        fbw = P.pack_adapters_bwd(fresh)
        for a in range(3):
            assert torch.equal(p.ad.At[a], fresh.At[a]) and torch.equal(p.ad.Bt[a], fresh.Bt[a])
            assert torch.equal(p.bw.Ar[a], fbw.Ar[a]) and torch.equal(p.bw.Bop[a], fbw.Bop[a])
    losses, opt = ex.train_adamw(block, x, target, ids, lens, steps=3, state_bits=bits)
    assert len(losses) == 3 and np.isfinite(losses).all() and opt.steps.tolist() == [3, 0, 3, 3]
