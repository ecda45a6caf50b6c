"""AdamW steps on gradients that are no numbers, infinite, or finite with a square that is not: what becomes
of the value itself, and that no other value is touched, over two steps and bit by bit with the definition in
numpy's float32 (``by_definition``).

In 8 bits a moment, or a root, that is not finite is held as the code of NaN and is nothing to its block's
scale, which is that of the block's finite values.  A block's scale is what couples its 64 values, so a
finite moment that is far above its neighbours' still takes their codes to 0 (never to no number).
"""

import numpy as np
import pytest

from test_gpu_adamw import F, _blocks, _codes, _coefficients, _np, Case

pytestmark = pytest.mark.gpu

# each tensor's places of a bad gradient: alone in its block, twice, at a block's ends, a whole block, and in
# the last, part filled block of a vector
SHAPES = [("plain", 1, 200, 0), ("A", 128, 8, 0), ("B", 8, 128, 1), ("plain", 1, 4096, 1), ("A", 64, 5, 2), ("plain", 1, 130, 2)]
BAD = [[5, 70, 100, 199], [0, 63, 64, 700], [77, 130, 1023], list(range(640, 704)) + [64 * 20, 64 * 20 + 63, 4095], [319], []]
VALUES = {"nan": np.nan, "inf": np.inf, "-inf": -np.inf, "1e20": 1e20, "-1e20": -1e20, "3e38": 3e38}


def _held(x, floor):
    """Codes (as the values they stand for) and scales of float32 values in 8 bits."""
    b = _blocks(x)
    fine = np.isfinite(b)
    most = np.where(fine, np.abs(b), F(0)).max(1, keepdims=True)
    most = np.where(most >= F(2.0 ** -100), most, F(0))
    with np.errstate(all="ignore"):
        inv = np.where(most > 0, F(1) / most * F(448), F(0)).astype(F)
        q = b * inv
        if floor:
            q = np.where((b > 0) & (most > 0), np.maximum(q, F(2.0 ** -9)), q)
    q = np.where(fine, np.clip(q, F(-448), F(448)), F(np.nan))
    return _codes(q).ravel()[:x.size].reshape(x.shape), (most * F(1 / F(448))).ravel()


def by_definition(b, step, h, norm, bits):
    b1, n1, b2, n2, eps, rb, keep, rate, clip = _coefficients(step, h, norm)
    p, g, m, v, ms, vs = (b[k] for k in ("p", "g", "m", "v", "ms", "vs"))
    with np.errstate(all="ignore"):
        if norm is not None:
            g = g * clip
        if bits == 8:
            m = m * np.repeat(ms, 64)[:m.size].reshape(m.shape)
            r = v * np.repeat(vs, 64)[:v.size].reshape(v.shape)
            v = r * r
        m = m * b1 + g * n1
        v = v * b2 + (g * g) * n2
        root = np.sqrt(v)
        p = p * keep - (m / (root * rb + eps)) * rate
    if bits == 8:
        (m, ms), (v, vs) = _held(m, False), _held(root, True)
    return dict(p=p, m=m, v=v, ms=ms, vs=vs)


def _check(c, before, clip):
    norms = c.norms(before, None)
    for i, (t, b, now) in enumerate(zip(c.tensors, before, c.values())):
        h = c.hyper[t.group]
        want = by_definition(b, int(c.steps[t.group]), h, norms[t.group] if clip else None, c.bits)
        for k, w in want.items():
            if w is not None:
                same = (now[k] == w) | (np.isnan(now[k]) & np.isnan(w))
                assert same.all(), f"tensor {i}: {k} differs in {(~same).sum()} of {same.size}"


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("beta1", [0.9, 0.0])
@pytest.mark.parametrize("bad,clip", [(b, c) for b, v in VALUES.items() for c in ((False, True) if np.isfinite(v) else (False,))])
def test_no_other_value_is_touched(bad, clip, beta1, bits):
    """Also with norms, where the largest norm of 0 takes finite gradients as they are (with others a group
    makes no step)."""
    import torch
    print("[case] overflow", bad, clip, beta1, bits, flush=True)
    c = Case(SHAPES, 3, bits, 11)
    c.hyper[:, 1], c.hyper[:, 5] = beta1, 0.0
    c.hyper_dev.copy_(torch.from_numpy(c.hyper))
    for t, at in zip(c.tensors, BAD):
        t.grad.flatten()[at] = VALUES[bad]
    for k in range(3):
        before = c.values()
        c.step(clip=clip)
        c.steps += 1
        _check(c, before, clip)
        for t, at in zip(c.tensors, BAD):
            for f in (t.param, t.m, t.v):  # nothing but the bad values themselves is no number
                off = (~torch.isfinite(f.detach().float().flatten())).nonzero().flatten().tolist()
                assert set(off) <= set(at), (k, off)
            assert bits == 32 or (torch.isfinite(t.m_scale).all() and torch.isfinite(t.v_scale).all())
            fine = torch.ones(t.param.numel(), dtype=torch.bool, device="cuda")
            fine[at] = False
            if t.copy is not None:
                assert torch.equal(t.copy.flatten()[fine], t.param.flatten()[fine].bfloat16())
        g = np.random.default_rng(k)
        for t in c.tensors:  # gradients that are finite from here on
            t.grad.copy_(torch.from_numpy(g.standard_normal(tuple(t.grad.shape)).astype(F) * F(0.01)))


def test_block_of_nothing_else():
    """Blocks whose only value that is not 0 is no number: all others stay 0 and step by their own gradients."""
    import torch
    import precision_gemm_amd as P
    print("[case] overflow alone", flush=True)
    t = P.AdamWTensor(torch.ones(192, device="cuda"), torch.zeros(192, device="cuda"))
    t.grad[3], t.grad[64:128] = float("inf"), float("nan")
    opt = P.AdamW([t], 1, state_bits=8)
    h = torch.tensor([[0.1, 0.9, 0.99, 1e-8, 0.0, 0.0]], dtype=torch.float64, device="cuda")
    P.adamw_step(opt, h)
    m = _np(t.m)
    assert np.isnan(m[3]) and np.isnan(m[64:128]).all() and not m[:3].any() and not m[4:64].any() and not m[128:].any()
    assert not t.m_scale.any() and not t.v_scale.any()
    t.grad.fill_(0.5)
    P.adamw_step(opt, h)
    bad = ~torch.isfinite(t.param)
    assert bad[3] and bad[64:128].all() and int(bad.sum()) == 65
    assert (t.param[4:64] < 1).all()
