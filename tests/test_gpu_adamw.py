"""GPU parity of the AdamW step with the fp64 oracle, and bit by bit with its definition in fp32.

The step rounds every product and sum on its own, so its results are those of the same line in numpy's
float32, where sqrt and division are correctly rounded too (`_by_definition`); coefficients are taken in
float64 and rounded once, and 8-bit codes are torch's e4m3fn conversion.  Only the coefficients could
differ, by a last bit of a 64-bit power, which leaves their rounding to fp32 as it is at the step counts
used here.

Tolerances against 64 bits (v = 2^-24, half a step of fp32): a term of m or v has at most the roundings of
its coefficient, of the clipping (coefficient and product), of two products and the sum: 6 v < 2^-21 of
the terms' magnitudes.  The update is rate m / (sqrt(v) c + eps): 2^-21 of v is half of that of its root,
and six more roundings: 2^-20 of the update, and 2^-21 of m's terms in its place; p keeps 3 v of itself.
8-bit states: half a step of e4m3 is 2^-4 of the value, or 2^-10 of the block's unit below 2^-6 of it (for
a root that is kept from 0: 2^-9).
"""

import numpy as np
import pytest

from oracle import step as S

pytestmark = pytest.mark.gpu

F = np.float32


def _torch():
    import torch
    return torch


def _np(t):
    return t.detach().float().cpu().numpy()


def _codes(x):
    """float32 values to e4m3fn and back."""
    torch = _torch()
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.float8_e4m3fn).float().numpy()


def _blocks(x):
    return np.concatenate([x.ravel(), np.zeros(-x.size % 64, x.dtype)]).reshape(-1, 64)


def _held(x, floor):
    """Codes (as the values they stand for) and scales of float32 values in 8 bits."""
    b = _blocks(x)
    most = np.abs(b).max(1, keepdims=True)
    most = np.where(most >= F(2.0 ** -100), most, F(0))
    with np.errstate(divide="ignore"):
        inv = np.where(most > 0, F(1) / most * F(448), F(0)).astype(F)
    q = b * inv
    if floor:
        q = np.where((b > 0) & (most > 0), np.maximum(q, F(2.0 ** -9)), q)
    return _codes(np.clip(q, F(-448), F(448))).ravel()[:x.size].reshape(x.shape), (most * F(1 / F(448))).ravel()


def _coefficients(step, h, norm):
    rate, b1, b2, eps, decay, largest = h
    c = 1.0 if norm is None or largest <= 0 else min(1.0, largest / (norm + 1e-6))
    return [F(v) for v in (b1, 1 - b1, b2, 1 - b2, eps, 1 / np.sqrt(1 - b2 ** step), 1 - rate * decay, rate / (1 - b1 ** step), c)]


def _by_definition(p, g, m, v, ms, vs, step, h, norm, bits):
    b1, n1, b2, n2, eps, rb, keep, rate, clip = _coefficients(step, h, norm)
    if norm is not None:
        g = g * clip
    if bits == 8:
        m = m * np.repeat(ms, 64)[:m.size].reshape(m.shape)
        r = v * np.repeat(vs, 64)[:m.size].reshape(m.shape)
        v = r * r
    m = m * b1 + g * n1
    v = v * b2 + (g * g) * n2
    root = np.sqrt(v)
    p = p * keep - (m / (root * rb + eps)) * rate
    if bits == 8:
        (m, ms), (v, vs) = _held(m, False), _held(root, True)
    return p, m, v, ms, vs


class Case:
    """Tensors (kind, rows, cols, group) with random values, and their handle."""

    def __init__(self, shapes, n_groups, bits, seed, packs=True, steps=None, gstd=0.01):
        torch = _torch()
        import precision_gemm_amd as P
        rng = np.random.default_rng(seed)
        self.bits, self.P = bits, P
        f = lambda a: torch.from_numpy(np.ascontiguousarray(a, F)).cuda()  # noqa: E731
        ts = []
        for kind, rows, cols, group in shapes:
            n = (rows, cols)
            p, g = rng.standard_normal(n).astype(F) * F(0.02), rng.standard_normal(n).astype(F) * F(gstd)
            m, root = rng.standard_normal(n).astype(F) * F(0.003), np.abs(rng.standard_normal(n)).astype(F) * F(0.01)
            t = P.AdamWTensor(f(p), f(g), group, kind)
            if bits == 8:
                (mq, ms), (vq, vs) = _held(m, False), _held(root, True)
                t.m, t.v = f(mq).to(torch.float8_e4m3fn), f(vq).to(torch.float8_e4m3fn)
                t.m_scale, t.v_scale = f(ms), f(vs)
            else:
                t.m, t.v = f(m), f(root * root)
            if kind == "plain":
                t.copy = torch.zeros(n, dtype=torch.bfloat16, device="cuda") if packs and rows * cols % 3 else None
            elif packs:
                r, side = (cols, rows) if kind == "A" else (rows, cols)
                t.copy = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
                sizes = (P.a_rows(r), P.rank_pad(r)) if kind == "A" else (P.rank_pad(r), P.a_rows(r))
                # whole buffers are written, the padding ranks too
                t.pack, t.pack_bwd = (torch.full((s, side), 7.0, dtype=torch.bfloat16, device="cuda") for s in sizes)
            ts.append(t)
        self.tensors = ts
        self.hyper = np.stack([rng.uniform(1e-4, 1e-2, n_groups), np.full(n_groups, 0.9), rng.choice([0.95, 0.999], n_groups),
                               np.full(n_groups, 1e-8), rng.uniform(0, 0.1, n_groups), rng.uniform(0.1, 3.0, n_groups)], 1)
        self.steps = np.asarray(rng.integers(0, 50, n_groups) if steps is None else steps, np.int32)
        self.opt = P.AdamW(ts, n_groups, state_bits=bits, steps=torch.from_numpy(self.steps.copy()).cuda())
        self.hyper_dev = torch.from_numpy(self.hyper).cuda()

    def values(self):
        return [dict(p=_np(t.param), g=_np(t.grad), m=_np(t.m), v=_np(t.v), ms=None if t.m_scale is None else _np(t.m_scale),
                     vs=None if t.v_scale is None else _np(t.v_scale)) for t in self.tensors]

    def norms(self, values, active):
        sums = np.zeros(len(self.hyper))
        for t, v in zip(self.tensors, values):
            sums[t.group] += (v["g"].astype(np.float64) ** 2).sum()
        return np.sqrt(sums) * (np.ones(len(sums)) if active is None else np.asarray(active) != 0)

    def step(self, active=None, clip=False, **kw):
        torch = _torch()
        act = None if active is None else torch.tensor(active, dtype=torch.int32, device="cuda")
        return self.P.adamw_step(self.opt, self.hyper_dev, active=act, clip=clip, **kw)

    def check(self, before, norms, active, clip):
        """The step from ``before`` to what the tensors hold now."""
        torch = _torch()
        on = [True] * len(self.hyper) if active is None else [a != 0 for a in active]
        for i, (t, b, now) in enumerate(zip(self.tensors, before, self.values())):
            what = f"tensor {i} ({t.kind} {tuple(t.param.shape)}, group {t.group})"
            if not on[t.group]:
                for k in b:
                    assert np.array_equal(b[k], now[k]) if b[k] is not None else now[k] is None, (what, k)
                continue
            step, h = int(self.steps[t.group]), self.hyper[t.group]
            norm = norms[t.group] if clip else None
            p, m, v, ms, vs = _by_definition(b["p"], b["g"], b["m"], b["v"], b["ms"], b["vs"], step, h, norm, self.bits)
            for k, want in (("m", m), ("v", v), ("ms", ms), ("vs", vs), ("p", p)):
                if want is not None:
                    assert np.array_equal(now[k], want), f"{what}: {k} differs in {(now[k] != want).sum()} of {want.size}"
            self._check64(b, now, step, h, norm, what)
            if t.copy is not None:
                assert torch.equal(t.copy, t.param.bfloat16()), what
        self._check_packs(on)

    def _check64(self, b, now, step, h, norm, what):
        rate, b1, b2, eps, decay, largest = h
        d = {k: None if x is None else x.astype(np.float64) for k, x in b.items()}
        g = d["g"] * (S.clip_factor(norm, largest) if norm is not None else 1.0)
        m0, v0 = d["m"], d["v"]
        if self.bits == 8:
            m0 = m0 * np.repeat(d["ms"], 64)[:m0.size].reshape(m0.shape)
            v0 = (v0 * np.repeat(d["vs"], 64)[:v0.size].reshape(v0.shape)) ** 2
        p, m, v = S.adamw(d["p"], g, m0, v0, step, rate, b1, b2, eps, decay)
        mag = b1 * np.abs(m0) + (1 - b1) * np.abs(g)
        den = np.sqrt(v / (1 - b2 ** step)) + eps
        upd = rate / (1 - b1 ** step) / den
        tol = 2.0 ** -22 * np.abs(d["p"]) + 2.0 ** -20 * upd * np.abs(m) + 2.0 ** -21 * upd * mag
        assert (np.abs(now["p"] - p) <= tol + 1e-40).all(), f"{what}: param against 64 bits"
        if self.bits == 32:
            assert (np.abs(now["m"] - m) <= 2.0 ** -21 * mag + 1e-44).all(), f"{what}: m against 64 bits"
            assert (np.abs(now["v"] - v) <= 2.0 ** -21 * v + 1e-44).all(), f"{what}: v against 64 bits"
            return
        for code, sc, want, least, size in ((now["m"], now["ms"], m, 2.0 ** -10, mag), (now["v"], now["vs"], np.sqrt(v), 2.0 ** -9, np.sqrt(v))):
            assert (np.abs(sc - S.held(want)) <= 2.0 ** -20 * _blocks(size).max(1) / 448).all(), f"{what}: scales"
            unit = np.repeat(sc.astype(np.float64), 64)[:want.size].reshape(want.shape)
            assert (np.abs(code * unit - want) <= 2.0 ** -4 * np.abs(want) + least * unit + 2.0 ** -19 * size).all(), f"{what}: codes"

    def _check_packs(self, on):
        """The packed forms are those that the library's own packing gives."""
        torch = _torch()
        P = self.P
        for t in self.tensors:
            if t.kind == "plain" or t.pack is None or not on[t.group]:
                continue
            w = t.copy
            r, side = (w.shape[1], w.shape[0]) if t.kind == "A" else w.shape
            other = torch.zeros((r, 128) if t.kind == "A" else (128, r), dtype=torch.bfloat16, device="cuda")
            A, B = (w, other) if t.kind == "A" else (other, w)
            At, Bt = P.pack_adapter(A, B)
            bw = P.pack_adapters_bwd(P.Adapters([A], [B], torch.ones(1, device="cuda")))
            fwd, bwd = (At, bw.Ar[0]) if t.kind == "A" else (Bt, bw.Bop[0])
            assert torch.equal(t.pack.flatten(), fwd.flatten()), (t.kind, tuple(w.shape), "pack")
            assert torch.equal(t.pack_bwd.flatten(), bwd.flatten()), (t.kind, tuple(w.shape), "pack_bwd")


SHAPES = {
    "one value": [("plain", 1, 1, 0)],
    "short vectors": [("plain", 1, n, n % 2) for n in (1, 2, 3, 5, 63, 64, 65, 127, 4095, 4096, 4097, 8191)],
    "vectors of whole quads": [("plain", 1, n, n % 3) for n in (4, 8, 60, 100, 196, 396, 1000, 4100, 8188)],
    "rank 1": [("A", 4160, 1, 0), ("B", 1, 4160, 0), ("A", 64, 1, 0), ("B", 1, 64, 1)],
    "rank 2 and 3": [("A", 2112, 2, 0), ("B", 2, 2112, 0), ("A", 1344, 3, 1), ("B", 3, 1408, 1)],
    "rank 8": [("A", 4096, 8, 0), ("B", 8, 6144, 0)],
    "rank 16": [("A", 512, 16, 0), ("B", 16, 320, 0)],
    "rank 33": [("A", 128, 33, 0), ("B", 33, 192, 0)],
    "rank 64": [("A", 256, 64, 0), ("B", 64, 384, 0)],
    "all ranks": [x for r in range(1, 65) for x in (("A", 192, r, r % 5), ("B", r, 128, r % 5))],
    "tenants": [x for g, r in enumerate((5, 64, 8, 17, 32)) for x in (("A", 640, r, g), ("B", r, 1344, g), ("A", 1344, r, g), ("B", r, 640, g))]
    + [("plain", 3, 333, 2)],
}


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("clip", [False, True])
@pytest.mark.parametrize("name", SHAPES)
def test_steps(name, bits, clip):
    print("[case] adamw", name, bits, clip, flush=True)
    groups = 1 + max(s[3] for s in SHAPES[name])
    c = Case(SHAPES[name], groups, bits, len(name))
    rng = np.random.default_rng(3)
    for k in range(3):
        active = None if k == 0 else [int(v) for v in rng.integers(0, 2, groups)]
        before = c.values()
        norms = c.norms(before, active)
        got = c.step(active, clip)
        c.steps += 1 if active is None else np.asarray(active, np.int32)
        assert np.array_equal(c.opt.steps.cpu().numpy(), c.steps)
        if clip:
            assert (np.abs(got.double().cpu().numpy() - norms) <= 2.0 ** -23 * norms).all()
        else:
            assert got is None
        c.check(before, norms, active, clip)
        for t in c.tensors:  # the next step's gradients
            t.grad.mul_(-0.7).add_(0.003)


def test_states_are_made_as_zeros():
    torch = _torch()
    import precision_gemm_amd as P
    rng = np.random.default_rng(1)
    for bits in (32, 8):
        t = P.AdamWTensor(torch.ones(100, device="cuda"), torch.from_numpy(rng.standard_normal(100).astype(F)).cuda())
        opt = P.AdamW([t], 1, state_bits=bits)
        h = torch.tensor([[0.1, 0.9, 0.99, 0.0, 0.0, 0.0]], dtype=torch.float64, device="cuda")
        P.adamw_step(opt, h)
        assert torch.allclose(t.param, 1 - 0.1 * t.grad.sign(), atol=1e-5) and int(opt.steps[0]) == 1


def test_adapters_of_a_projection():
    """The handle made from an adapter set: its bf16 adapters, packed forms and backward forms are
    stepped, and the layer's pointer tables keep pointing at them."""
    torch = _torch()
    import precision_gemm_amd as P
    print("[case] adapters", flush=True)
    g = torch.Generator(device="cuda").manual_seed(0)
    ranks, K, N = (5, 16, 64), 256, 384
    ad = P.Adapters([torch.randn(K, r, generator=g, device="cuda").bfloat16() for r in ranks],
                    [torch.randn(r, N, generator=g, device="cuda").bfloat16() for r in ranks], torch.ones(3, device="cuda"))
    bw = P.pack_adapters_bwd(ad)
    grads = P.alloc_grads(ad, K, N)
    for m in grads.dA + grads.dB:
        m.normal_(generator=g)
    ts = P.adamw_adapters(ad, grads, bw, group0=1)
    assert [t.group for t in ts] == [1, 1, 2, 2, 3, 3] and torch.equal(ts[0].param, ad.A[0].float())
    opt = P.AdamW(ts, 4)
    before = [a.clone() for a in ad.A + ad.B]
    h = torch.tensor([[0.1, 0.9, 0.99, 1e-8, 0.0, 0.0]] * 4, dtype=torch.float64, device="cuda")
    P.adamw_step(opt, h)
    fresh = P.Adapters([a.clone() for a in ad.A], [b.clone() for b in ad.B], torch.ones(3, device="cuda"))
    fbw = P.pack_adapters_bwd(fresh)
    for a in range(3):
        assert torch.equal(ad.At[a], fresh.At[a]) and torch.equal(ad.Bt[a], fresh.Bt[a])
        assert torch.equal(bw.Ar[a], fbw.Ar[a]) and torch.equal(bw.Bop[a], fbw.Bop[a])
        assert int(ad.A_ptrs[a]) == ad.At[a].data_ptr() and int(bw.Bop_ptrs[a]) == bw.Bop[a].data_ptr()
    for b, a, d in zip(before, ad.A + ad.B, grads.dA + grads.dB):
        assert torch.allclose(a.float(), b.float() - 0.1 * d.sign(), atol=0.02)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_group_whose_gradient_is_not_finite(bits, bad):
    torch = _torch()
    print("[case] not finite", bits, bad, flush=True)
    c = Case([("A", 128, 8, 0), ("B", 8, 128, 0), ("A", 128, 8, 1), ("plain", 1, 100, 2)], 3, bits, 4)
    c.tensors[1].grad[3, 77] = bad
    before, status = c.values(), torch.zeros(1, dtype=torch.int32, device="cuda")
    norms = c.norms([dict(v, g=np.nan_to_num(v["g"], nan=0, posinf=0, neginf=0)) for v in before], None)
    packs = [t.pack.clone() for t in c.tensors[:2]]
    norm = c.step(clip=True, status=status)
    assert int(status) == c.P.LORA_ADAMW_NOT_FINITE and not torch.isfinite(norm[0]) and torch.isfinite(norm[1:]).all()
    for t, b, now in zip(c.tensors[:2], before[:2], c.values()[:2]):
        for k in ("p", "m", "v", "ms", "vs"):
            assert b[k] is None or np.array_equal(b[k], now[k])
    assert all(torch.equal(t.pack, p) for t, p in zip(c.tensors[:2], packs))
    c.steps += np.array([0, 1, 1], np.int32)
    assert np.array_equal(c.opt.steps.cpu().numpy(), c.steps)
    keep = c.tensors
    c.tensors, norms = keep[2:], norms
    c.check(before[2:], norms, [0, 1, 1], True)
    # without clipping it is taken as it is: the value itself becomes no number, no other does
    c.tensors = keep
    c.step(clip=False)
    p = keep[1].param
    assert not torch.isfinite(p[3, 77]) and int((~torch.isfinite(p)).sum()) == 1 and torch.isfinite(keep[2].param).all()


def test_gradients_of_zero_and_tiny_ones():
    """Blocks of zeros, and of values whose inverse would overflow, are held as zero in 8 bits; a root
    far below its block's largest keeps a code that is not 0."""
    torch = _torch()
    import precision_gemm_amd as P
    print("[case] tiny", flush=True)
    g = torch.zeros(256, device="cuda")
    g[64:128] = 1e-35
    g[128], g[129:192] = 1.0, 1e-12
    g[192:] = 1e-30
    t = P.AdamWTensor(torch.ones(256, device="cuda"), g)
    opt = P.AdamW([t], 1, state_bits=8)
    h = torch.tensor([[0.1, 0.9, 0.99, 1e-8, 0.0, 0.0]], dtype=torch.float64, device="cuda")
    P.adamw_step(opt, h)
    assert torch.isfinite(t.param).all() and torch.equal(t.param[:64], torch.ones(64, device="cuda"))
    m, v = t.m.float(), t.v.float()
    assert not m[:128].any() and not v[:128].any() and not t.m_scale[:2].any() and not t.v_scale[:2].any()
    assert float(m[128]) == 448 and float(v[128]) == 448 and (v[129:192] == 2.0 ** -9).all() and not m[129:192].any()
    for _ in range(3):
        g.zero_()
        P.adamw_step(opt, h)
    assert torch.isfinite(t.param).all() and (t.param - 1).abs().max() < 0.5


def test_refusals():
    torch = _torch()
    import precision_gemm_amd as P
    w, g = torch.zeros((128, 8), device="cuda"), torch.zeros((128, 8), device="cuda")
    T = P.AdamWTensor
    for kw, match in ((dict(grad=g.half()), "grad must have dtype"), (dict(grad=g[:64]), "grad must have 1024 values"),
                      (dict(grad=g.view(8, 128)), "shape of param"), (dict(grad=g.cpu()), "grad must be a device tensor"),
                      (dict(kind="C"), "kind"), (dict(copy=w), "copy must have dtype"),
                      (dict(pack=w.bfloat16()), "pack must have 2048 values"), (dict(m=w.half()), "m must have dtype"),
                      (dict(m_scale=w), "8 bits"), (dict(param=w.t(), grad=g.t()), "contiguous"),
                      (dict(kind="plain", pack=w.bfloat16()), "for A and B")):
        with pytest.raises(ValueError, match=match):
            P.AdamW([T(**{**dict(param=w, grad=g, kind="A"), **kw})], 1)
    with pytest.raises(RuntimeError, match="status 1"):
        P.AdamW([T(w, g, 1, "A")], 1)
    with pytest.raises(RuntimeError, match="status 1"):  # the same tensor twice
        P.AdamW([T(w, g, 0, "A"), T(w, g, 0, "A")], 1)
    with pytest.raises(RuntimeError, match="status 2"):
        P.AdamW([T(torch.zeros((100, 8), device="cuda"), torch.zeros((100, 8), device="cuda"), 0, "A")], 1)
    with pytest.raises(ValueError, match="steps must have dtype"):
        P.AdamW([T(w, g, 0, "A")], 1, steps=torch.zeros(1, device="cuda"))
    opt = P.AdamW([T(w, g, 0, "A")], 2)
    h = torch.zeros((2, 6), dtype=torch.float64, device="cuda")
    for kw, match in ((dict(hyper=h.float()), "hyper must have dtype"), (dict(hyper=h[:1]), "hyper must have shape"),
                      (dict(active=torch.ones(2, device="cuda")), "active must have dtype"),
                      (dict(grad_norm=torch.ones(2, device="cuda")), "step that clips"),
                      (dict(status=torch.zeros(2, dtype=torch.int32, device="cuda")), "status must have shape"),
                      (dict(clip=torch.ones(2)), "truth value")):
        with pytest.raises(ValueError, match=match):
            P.adamw_step(opt, **{"hyper": h, **kw})


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("clip", [False, True])
def test_graph_replays(bits, clip):
    """A captured step, replayed: every replay is the eager step from the same state."""
    torch = _torch()
    print("[case] adamw graph", bits, clip, flush=True)
    shapes = SHAPES["tenants"]
    a, b = (Case(shapes, 5, bits, 9) for _ in range(2))
    norm, status = torch.zeros(5, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    active = torch.ones(5, dtype=torch.int32, device="cuda")
    kw = dict(grad_norm=norm) if clip else {}
    a.P.adamw_step(a.opt, a.hyper_dev, active=active, clip=clip, status=status, **kw)
    b.step(clip=clip)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.P.adamw_step(a.opt, a.hyper_dev, active=active, clip=clip, status=status, **kw)
    for i in range(4):
        active[i] = 0
        want = b.step([int(v) for v in active.cpu()], clip)
        g.replay()
        torch.cuda.synchronize()
        for s, t in zip(a.tensors, b.tensors):
            for f in ("param", "m", "v", "m_scale", "v_scale", "copy", "pack", "pack_bwd"):
                x, y = getattr(s, f), getattr(t, f)
                assert x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8)), (i, f)
        assert torch.equal(a.opt.steps, b.opt.steps) and (not clip or torch.equal(norm, want)) and int(status) == 0
        for c in (a, b):
            for t in c.tensors:
                t.grad.mul_(0.9)
