"""GPU parity of the attention block (head norms with rotation, their gradients, the append to
a paged cache, drafted trees, attention over the cache) with the fp64 oracle.

Tolerances, from the arithmetic (u = 2^-8 is half a step of bf16's 8 significant bits, relative):
 * forward: fp32 until one bf16 rounding: u |y|, and 2^-18 of the pair's magnitudes for the fp32
   steps (a 256-term sum of squares, a reciprocal square root, four products);
 * e4m3 codes: half a step is 2^-4 relative, 2^-10 absolute below 2^-6;
 * gradients: u |dx| plus 2^-16 of the terms that are subtracted; weights' gradients 2^-16 of the
   sum of magnitudes (fp32 partial sums) and 1e-5 relative Frobenius;
 * attention: probabilities enter the product in bf16 (u each), the output is rounded once (u):
   u |out| + 2 u sum p |V|, the second u for the fp32 scores and sums (each below 2^-16 here);
   lse in fp32: 2^-20 of the largest score's terms and of the lse itself.
"""

import numpy as np
import pytest

from oracle import attention as A

pytestmark = pytest.mark.gpu

U = 2.0 ** -8


def _torch():
    import torch
    return torch


def _bf(rng, shape, std=1.0):
    """bf16 device tensor and its values in fp64."""
    torch = _torch()
    t = torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32)).to(torch.bfloat16)
    return t.cuda(), t.double().numpy()


def _f64(t):
    return t.detach().double().cpu().numpy()


def _i32(v):
    torch = _torch()
    return torch.from_numpy(np.ascontiguousarray(np.asarray(v, np.int32))).cuda()


def _within(got, ref, tol, what):
    assert np.isfinite(got).all(), f"{what}: not finite"
    over = np.abs(got - ref) - tol
    assert (over <= 0).all(), f"{what}: off by {np.abs(got - ref).flat[over.argmax()]:.3e}, allowed {np.broadcast_to(tol, over.shape).flat[over.argmax()]:.3e}"


def _rope_inputs(T, n_q, n_kv, D, rot, norm, seed, extra=0):
    torch = _torch()
    import precision_gemm_amd as P
    rng = np.random.default_rng(seed)
    width = (n_q + 2 * n_kv) * D
    qkv, x = _bf(rng, (T, width + extra), 1.5)
    x = x[:, :width].reshape(T, -1, D)
    pos = rng.integers(0, 500, T)
    cs = P.rope_table(500, rot) if rot else None
    w = [torch.from_numpy((1 + 0.2 * rng.standard_normal(D)).astype(np.float32)).cuda() if norm else None for _ in range(2)]
    return rng, qkv[:, :width] if extra else qkv, x, pos, cs, w


def _pair_size(n, rot, interleaved):
    """Magnitude of each value's rotated pair."""
    m = np.abs(n)
    if rot:
        a, b = A._pairs(rot, interleaved)
        s = m[..., a] + m[..., b]
        m = m.copy()
        m[..., a], m[..., b] = s, s
    return m


def _check_heads(got, x, pos, cs, w, inter, eps, what):
    csn, wn = (None if cs is None else _f64(cs)), (None if w is None else _f64(w))
    rot = 0 if cs is None else cs.shape[1]
    ref = A.norm_rope(x, pos, csn, wn, eps, inter)
    size = _pair_size(A.norm_rope(x, pos, None, wn, eps), rot, inter)
    _within(got, ref, U * np.abs(ref) + 2.0 ** -18 * size + 2.0 ** -133, what)
    return ref, size


ROPE = [  # T, n_q, n_kv, D, rot, interleaved, norm, extra columns of a row
    (1, 32, 8, 128, 128, False, True, 0),
    (7, 28, 4, 64, 32, True, True, 0),
    (33, 5, 1, 256, 256, False, True, 8),
    (130, 15, 3, 128, 64, False, False, 24),
    (3, 3, 3, 256, 16, True, False, 0),
    (11, 4, 2, 64, 0, False, True, 0),
    (2, 1, 1, 64, 48, True, True, 0),
    (1100, 32, 8, 128, 128, True, True, 0),
    (1031, 9, 9, 64, 64, False, True, 0),
]


@pytest.mark.parametrize("T,n_q,n_kv,D,rot,inter,norm,extra", ROPE)
def test_norm_rope(T, n_q, n_kv, D, rot, inter, norm, extra):
    torch = _torch()
    import precision_gemm_amd as P
    print("[case] norm_rope", T, n_q, n_kv, D, rot, inter, norm, extra, flush=True)
    _, qkv, x, pos, cs, (qw, kw) = _rope_inputs(T, n_q, n_kv, D, rot, norm, 1, extra)
    kw_args = dict(cos_sin=cs, q_weight=qw, k_weight=kw, eps=1e-5, interleaved=inter)
    before = qkv.clone()
    q, k = P.qk_norm_rope(qkv, _i32(pos), n_q, n_kv, D, **kw_args)
    assert torch.equal(qkv, before)
    _check_heads(_f64(q), x[:, :n_q], pos, cs, qw, inter, 1e-5, "q")
    _check_heads(_f64(k), x[:, n_q:n_q + n_kv], pos, cs, kw, inter, 1e-5, "k")
    # in place: the heads' own rows
    P.qk_norm_rope(qkv, _i32(pos), n_q, n_kv, D, q_out=qkv[:, :n_q * D], k_out=qkv[:, n_q * D:(n_q + n_kv) * D], **kw_args)
    assert torch.equal(qkv[:, :n_q * D], q.flatten(1)) and torch.equal(qkv[:, n_q * D:(n_q + n_kv) * D], k.flatten(1))
    assert torch.equal(qkv[:, (n_q + n_kv) * D:], before[:, (n_q + n_kv) * D:])


@pytest.mark.parametrize("T,n_q,n_kv,D,rot,inter,norm,extra", ROPE + [(5000, 4, 1, 64, 64, False, True, 0)])
def test_norm_rope_backward(T, n_q, n_kv, D, rot, inter, norm, extra):
    torch = _torch()
    import precision_gemm_amd as P
    print("[case] norm_rope_backward", T, n_q, n_kv, D, rot, inter, norm, extra, flush=True)
    rng, qkv, x, pos, cs, (qw, kw) = _rope_inputs(T, n_q, n_kv, D, rot, norm, 2, extra)
    dq, dqn = _bf(rng, (T, n_q, D), 0.02)
    dk, dkn = _bf(rng, (T, n_kv, D), 0.02)
    dv, dvn = _bf(rng, (T, n_kv, D), 0.02)
    args = dict(cos_sin=cs, q_weight=qw, k_weight=kw, eps=1e-5, interleaved=inter)
    dqkv, dqw, dkw = P.qk_norm_rope_backward(qkv, _i32(pos), dq, dk, dv, **args)
    got = _f64(dqkv).reshape(T, -1, D)
    csn = None if cs is None else _f64(cs)
    for name, xs, dy, w, g, dw in (("q", x[:, :n_q], dqn, qw, got[:, :n_q], dqw),
                                   ("k", x[:, n_q:n_q + n_kv], dkn, kw, got[:, n_q:n_q + n_kv], dkw)):
        wn = None if w is None else _f64(w)
        ref, dw_ref = A.norm_rope_backward(xs, dy, pos, csn, wn, 1e-5, inter)
        turned = A.rotate(dy, pos, csn, inter, sign=-1.0)
        size = _pair_size(dy, rot, inter)
        if norm:
            r = 1 / np.sqrt((xs * xs).mean(-1, keepdims=True) + 1e-5)
            xh = xs * r
            size = r * (size * np.abs(wn) + np.abs(xh) * (np.abs(turned * wn) * np.abs(xh)).mean(-1, keepdims=True))
            mag = (np.abs(turned * xh)).sum((0, 1))
            _within(_f64(dw), dw_ref, 2.0 ** -16 * mag, "d" + name + "_weight")
            assert np.linalg.norm(_f64(dw) - dw_ref) <= 1e-5 * np.linalg.norm(dw_ref)
        else:
            assert dw is None
        _within(g, ref, U * np.abs(ref) + 2.0 ** -16 * size + 2.0 ** -133, "d" + name)
    assert np.array_equal(got[:, n_q + n_kv:], dvn)
    # bitwise the same again, and with dv left to the caller, with buffers of the caller's
    if norm:
        ws = torch.full((P.qk_norm_rope_backward_workspace_bytes(T, D),), 255, dtype=torch.uint8, device="cuda")
        mine = torch.full_like(dqkv, 7.0)
        again = P.qk_norm_rope_backward(qkv, _i32(pos), dq, dk, None, dqkv=mine, workspace=ws, **args)
        cut = (n_q + n_kv) * D
        assert torch.equal(mine[:, :cut], dqkv[:, :cut]) and (mine[:, cut:] == 7.0).all()
        assert torch.equal(again[1], dqw) and torch.equal(again[2], dkw)


def test_norm_rope_backward_against_differences():
    """The gradient call against central differences of the forward call's own formula: the
    forward in 64 bits of the oracle, at the kernel's inputs, along random directions."""
    import precision_gemm_amd as P
    print("[case] norm_rope_backward differences", flush=True)
    T, n_q, n_kv, D, rot = 9, 6, 2, 64, 32
    rng, qkv, x, pos, cs, (qw, kw) = _rope_inputs(T, n_q, n_kv, D, rot, True, 3)
    dq, dqn = _bf(rng, (T, n_q, D))
    dk, dkn = _bf(rng, (T, n_kv, D))
    dqkv, dqw, dkw = P.qk_norm_rope_backward(qkv, _i32(pos), dq, dk, dq[:, :n_kv].contiguous(), cos_sin=cs, q_weight=qw,
                                             k_weight=kw, eps=1e-5)
    g = _f64(dqkv).reshape(T, -1, D)
    csn, w = _f64(cs), [_f64(qw), _f64(kw)]
    loss = lambda xs, w: ((A.norm_rope(xs[:, :n_q], pos, csn, w[0], 1e-5) * dqn).sum()  # noqa: E731
                          + (A.norm_rope(xs[:, n_q:n_q + n_kv], pos, csn, w[1], 1e-5) * dkn).sum())
    for _ in range(8):
        d = rng.standard_normal(x.shape)
        d[:, n_q + n_kv:] = 0
        h = 1e-5
        num = (loss(x + h * d, w) - loss(x - h * d, w)) / (2 * h)
        # the sum of bf16-rounded gradients along d: u of each term, in quadrature, four deviations
        assert abs((g * d).sum() - num) <= 4 * U * np.linalg.norm(g * d) + 1e-6 * abs(num)
        dw = [rng.standard_normal(D) for _ in range(2)]
        num = (loss(x, [a + h * b for a, b in zip(w, dw)]) - loss(x, [a - h * b for a, b in zip(w, dw)])) / (2 * h)
        # 1e-5 relative, as above, and the differences' own cancellation
        assert abs(_f64(dqw) @ dw[0] + _f64(dkw) @ dw[1] - num) <= 1e-5 * (
            np.linalg.norm(_f64(dqw)) * np.linalg.norm(dw[0]) + np.linalg.norm(_f64(dkw)) * np.linalg.norm(dw[1])) + 1e-6 * abs(num)


def test_rope_bad_positions_and_no_tokens():
    torch = _torch()
    import precision_gemm_amd as P
    print("[case] positions outside the table", flush=True)
    T, n_q, n_kv, D = 6, 4, 2, 64
    rng, qkv, x, pos, cs, (qw, kw) = _rope_inputs(T, n_q, n_kv, D, 64, True, 4)
    pos[1], pos[4] = -1, 500
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, k = P.qk_norm_rope(qkv, _i32(pos), n_q, n_kv, D, cos_sin=cs, q_weight=qw, k_weight=kw, status=status)
    assert status.item() == P.LORA_ATTN_BAD_POSITION
    bad = np.array([1, 4])
    ok = np.array([0, 2, 3, 5])
    assert not _f64(q)[bad].any() and not _f64(k)[bad].any()
    _check_heads(_f64(q)[ok], x[ok, :n_q], pos[ok], cs, qw, False, 1e-6, "q")
    status.zero_()
    dq, dqn = _bf(rng, (T, n_q, D))
    dk, dkn = _bf(rng, (T, n_kv, D))
    dqkv, dqw, dkw = P.qk_norm_rope_backward(qkv, _i32(pos), dq, dk, dk, cos_sin=cs, q_weight=qw, k_weight=kw, status=status)
    assert status.item() == P.LORA_ATTN_BAD_POSITION
    assert not _f64(dqkv)[bad][:, :(n_q + n_kv) * D].any()
    _, dw_ref = A.norm_rope_backward(x[ok, :n_q], dqn[ok], pos[ok], _f64(cs), _f64(qw), 1e-6)
    assert np.linalg.norm(_f64(dqw) - dw_ref) <= 1e-5 * np.linalg.norm(dw_ref)
    # no tokens: nothing but zero gradients of the weights
    e = lambda n: torch.empty((0, n, D), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    none = torch.empty((0, (n_q + 2 * n_kv) * D), dtype=torch.bfloat16, device="cuda")
    q, k = P.qk_norm_rope(none, _i32([]), n_q, n_kv, D, cos_sin=cs, q_weight=qw, k_weight=kw)
    assert q.shape == (0, n_q, D) and k.shape == (0, n_kv, D)
    _, dqw, dkw = P.qk_norm_rope_backward(none, _i32([]), e(n_q), e(n_kv), e(n_kv), cos_sin=cs, q_weight=qw, k_weight=kw)
    assert not dqw.any() and not dkw.any()


def test_norm_rope_infinities():
    """An infinite or NaN value reaches its own head (through the norm, or its rotated pair), no other."""
    torch = _torch()
    import precision_gemm_amd as P
    print("[case] infinities", flush=True)
    T, n_q, n_kv, D = 3, 4, 2, 64
    _, qkv, x, pos, cs, _ = _rope_inputs(T, n_q, n_kv, D, 32, False, 5)
    pos[:] = 3
    qkv[1, 40] = float("inf")    # head 0, past the rotated values
    qkv[1, D + 3] = float("nan")  # head 1, a rotated pair (3, 19)
    q, _ = P.qk_norm_rope(qkv, _i32(pos), n_q, n_kv, D, cos_sin=cs)
    g = _f64(q)
    assert g[1, 0, 40] == np.inf and np.isfinite(np.delete(g[1, 0], 40)).all()
    assert sorted(np.flatnonzero(~np.isfinite(g[1, 1]))) == [3, 19]
    assert np.isfinite(g[1, 2:]).all() and np.isfinite(g[[0, 2]]).all()


# ---- the append ----

def _fp8_table():
    torch = _torch()
    return torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,n_q,n_kv,D,rot,inter,norm,extra,page", [r + (p,) for r, p in zip(ROPE, (16, 32, 64, 16, 128, 256, 1024, 64, 32))])
def test_append(T, n_q, n_kv, D, rot, inter, norm, extra, page, fp8):
    torch = _torch()
    import precision_gemm_amd as P
    print("[case] append", T, n_q, n_kv, D, rot, inter, norm, extra, page, fp8, flush=True)
    rng, qkv, x, pos, cs, (qw, kw) = _rope_inputs(T, n_q, n_kv, D, rot, norm, 6, extra)
    n_pages = -(-T // page) + 3
    slots = rng.permutation(n_pages * page)[:T]
    if T > 4:
        slots[1], slots[3] = -1, -7  # not stored
    shape = (n_pages, n_kv, page, D)
    if fp8:
        old = [torch.from_numpy(rng.integers(0, 120, shape).astype(np.uint8)).cuda().view(torch.float8_e4m3fn) for _ in range(2)]
        scales = [rng.uniform(0.005, 0.02, n_kv).astype(np.float32) for _ in range(2)]
        sc = [torch.from_numpy(s).cuda() for s in scales]
    else:
        old = [_bf(rng, shape)[0] for _ in range(2)]
        scales, sc = [np.ones(n_kv)] * 2, [None, None]
    kc, vc = old[0].clone(), old[1].clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = P.rope_append_kv(qkv, _i32(pos), _i32(slots), kc, vc, n_q, cos_sin=cs, q_weight=qw, k_weight=kw, eps=1e-5,
                         interleaved=inter, k_scale=sc[0], v_scale=sc[1], status=status)
    assert status.item() == 0
    _check_heads(_f64(q), x[:, :n_q], pos, cs, qw, inter, 1e-5, "q")
    csn, wn = (None if cs is None else _f64(cs)), (None if kw is None else _f64(kw))
    krows = A.norm_rope(x[:, n_q:n_q + n_kv], pos, csn, wn, 1e-5, inter)
    ksize = _pair_size(A.norm_rope(x[:, n_q:n_q + n_kv], pos, None, wn, 1e-5), rot, inter)
    vrows = x[:, n_q + n_kv:]
    for name, cache, was, rows, size, s in (("k", kc, old[0], krows, ksize, scales[0]), ("v", vc, old[1], vrows, np.abs(vrows), scales[1])):
        s = s.astype(np.float64)[None, :, None]
        ref = A.append(_f64(was), np.clip(rows / s, -448, 448) if fp8 else rows, slots)
        step = A.append(np.zeros(shape), (2.0 ** -4 * np.abs(rows / s) + 2.0 ** -10 + 2.0 ** -18 * size / s) if fp8
                        else U * np.abs(rows) + 2.0 ** -18 * size + 2.0 ** -133, slots)
        _within(_f64(cache), ref, step, name)
    # exact where no rounding is in question: the values of a bf16 cache as they came
    if not fp8:
        assert np.array_equal(_f64(vc), A.append(_f64(old[1]), vrows, slots))


def test_append_codes_and_errors():
    torch = _torch()
    import precision_gemm_amd as P
    print("[case] append: codes, saturation, bad slots", flush=True)
    D, page = 64, 16
    qkv = torch.zeros((6, 3 * D), dtype=torch.bfloat16, device="cuda")
    vals = torch.tensor([448.0, 464.0, 1e4, -1e4, float("inf"), float("-inf"), float("nan"), 0.0, 2.0 ** -9, 2.0 ** -10,
                         17.0, 18.0, 19.0, -0.0], dtype=torch.bfloat16, device="cuda")
    qkv[0, 2 * D:2 * D + 14] = vals
    qkv[:, D:2 * D] = 1.0
    kc = torch.zeros((2, 1, page, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    vc, one = kc.clone(), torch.ones(1, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cs = P.rope_table(4, 64)
    P.rope_append_kv(qkv, _i32([0, 0, 0, 4, 0, -1]), _i32([31, 32, -1, 3, 0, 5]), kc, vc, 1, cos_sin=cs, k_scale=one,
                     v_scale=one, status=status)
    assert status.item() == P.LORA_ATTN_BAD_POSITION | P.LORA_ATTN_BAD_SLOT
    want = vals.float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).tolist()
    got = vc.view(torch.uint8)[1, 0, 15, :14].tolist()
    assert got[:6] + got[7:] == want[:6] + want[7:] and got[6] & 0x7f == 0x7f
    k = kc.float()
    assert (k[1, 0, 15] == 1).all() and (k[0, 0, 0] == 1).all() and k.sum() == 2 * D


# ---- drafted trees ----

@pytest.mark.parametrize("ns", [[1], [5, 0, 64, 1], [100, 3, 130], [1] * 300])
def test_tree_mask(ns):
    torch = _torch()
    import precision_gemm_amd as P
    print("[case] tree_mask", ns[:5], flush=True)
    rng = np.random.default_rng(7)
    parents = [p for n in ns for p in [int(rng.integers(-1, j)) if j else -1 for j in range(n)]]
    indptr = np.concatenate([[0], np.cumsum(ns)])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    m = P.tree_mask(_i32(parents), _i32(indptr), max(ns), status=status).cpu().numpy().view(np.uint64)
    assert status.item() == 0
    assert [sum(int(w) << 64 * i for i, w in enumerate(r)) for r in m] == A.tree_mask(parents, indptr)


def test_tree_mask_bad_parent():
    torch = _torch()
    import precision_gemm_amd as P
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    m = P.tree_mask(_i32([-1, 1, 0, 5]), _i32([0, 4]), 4, status=status).cpu().tolist()
    assert status.item() == P.LORA_ATTN_BAD_PARENT and m == [[1], [2], [5], [8]]


@pytest.mark.parametrize("ns", [[64] * 3, [1024, 1, 513], [65, 128, 2]])
def test_tree_mask_chains(ns):
    """The deepest trees: every token the child of the one before."""
    import precision_gemm_amd as P
    print("[case] tree_mask chains", ns, flush=True)
    indptr = np.concatenate([[0], np.cumsum(ns)])
    parents = np.concatenate([np.arange(n) - 1 for n in ns])
    m = P.tree_mask(_i32(parents), _i32(indptr), max(ns)).cpu().numpy().view(np.uint64)
    for row, j in zip(m, (j for n in ns for j in range(n))):
        assert sum(int(w) << 64 * i for i, w in enumerate(row)) == (1 << (j + 1)) - 1


@pytest.mark.parametrize("indptr,rows", [([2, 4], [0, 0, 1, 3]), ([0, 3], [1, 3, 7, 0]), ([0, 2, 9], [1, 3, 0, 0]),
                                         ([-1, 2, 4], [0, 0, 1, 3]), ([0, 4], [0, 0, 0, 0])])
def test_tree_mask_bad_lengths(indptr, rows):
    """Rows that no sequence has, or whose sequence does not fit (more than max_q = 3 tokens), are 0."""
    torch = _torch()
    import precision_gemm_amd as P
    print("[case] tree_mask bad lengths", indptr, flush=True)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    parents = [-1, 0, 1, 2] if indptr[0] == 0 and len(indptr) == 2 else [-1, 0, -1, 0]
    m = P.tree_mask(_i32(parents), _i32(indptr), 3, status=status).cpu().flatten().tolist()
    assert status.item() == P.LORA_ATTN_BAD_LENGTH and m == rows


# ---- attention ----

def _put(t, where, code8, value):
    """A value into cache places, as its code in an 8-bit cache."""
    torch = _torch()
    if t.dtype == torch.bfloat16:
        t[where] = value
    else:
        t.view(torch.uint8)[where] = code8


class Batch:
    """A paged cache with B sequences, its pages dealt out of order, and their queries."""

    def __init__(self, seed, ns, kvs, n_q, n_kv, D, page, fp8, mask="none", spare=2, q_std=2.0, extra=0):
        torch = _torch()
        rng = self.rng = np.random.default_rng(seed)
        self.ns, self.kvs, self.page, self.fp8, self.D, self.n_q, self.n_kv = ns, kvs, page, fp8, D, n_q, n_kv
        pages = [-(-kv // page) for kv in kvs]
        self.n_pages = sum(pages) + spare
        order = rng.permutation(self.n_pages)
        width = max(pages + [1]) + 1
        self.table = rng.integers(0, self.n_pages, (len(ns), width))  # past a sequence's pages: any page
        at = 0
        for b, m in enumerate(pages):
            self.table[b, :m] = order[at:at + m]
            at += m
        shape = (self.n_pages, n_kv, page, D)
        if fp8:
            self.sk, self.sv = (rng.uniform(0.01, 0.02, n_kv).astype(np.float32) for _ in range(2))
            mk = lambda s, std: torch.from_numpy((rng.standard_normal(shape) * std / s[None, :, None, None]).astype(np.float32)  # noqa: E731
                                                 ).clamp(-448, 448).to(torch.float8_e4m3fn)
            self.k, self.v = mk(self.sk, 1.0).cuda(), mk(self.sv, 0.5).cuda()
        else:
            self.sk = self.sv = None
            self.k, self.v = _bf(rng, shape)[0], _bf(rng, shape, 0.5)[0]
        T = self.T = sum(ns)
        q, _ = _bf(rng, (T, n_q * D + extra), q_std)
        self.q = q[:, :n_q * D].unflatten(1, (n_q, D)) if T else q.new_empty((0, n_q, D))
        self.indptr = np.concatenate([[0], np.cumsum(ns)])
        self.masks = None
        if mask == "tree":
            self.masks = A.tree_mask([int(rng.integers(-1, j)) if j else -1 for n in ns for j in range(n)], self.indptr)
        elif mask == "any":  # any set of the drafted tokens, none and all among them
            self.masks = [int.from_bytes(rng.bytes(-(-n // 8)), "little") & ((1 << n) - 1) for n in ns for _ in range(n)]
            self.masks[::5] = [0] * len(self.masks[::5])
        self.scale = 1.0 / np.sqrt(D)

    def mask_tensor(self, junk=True):
        if self.masks is None:
            return None
        torch = _torch()
        words = max(1, -(-max(self.ns) // 64))
        rows = []
        for n, m in zip(np.repeat(self.ns, self.ns), self.masks):
            m = m | ((-1 << int(n)) if junk else 0)  # bits past the sequence's tokens say nothing
            rows.append([(m >> 64 * w) & (2 ** 64 - 1) for w in range(words)])
        return torch.from_numpy(np.array(rows, np.uint64).reshape(self.T, words).view(np.int64)).cuda()

    def run(self, **kw):
        torch = _torch()
        import precision_gemm_amd as P
        sc = [None if s is None else torch.from_numpy(s).cuda() for s in (self.sk, self.sv)]
        args = dict(tree_mask=self.mask_tensor(), scale=self.scale, k_scale=sc[0], v_scale=sc[1])
        args.update(kw)
        return P.tree_attention(self.q, self.k, self.v, _i32(self.table), _i32(self.kvs), _i32(self.indptr),
                                max(self.ns + [1]), **args)

    def oracle(self):
        k, v = _f64(self.k), _f64(self.v)
        if self.fp8:
            k, v = k * self.sk.astype(np.float64)[None, :, None, None], v * self.sv.astype(np.float64)[None, :, None, None]
        return A.tree_attention(_f64(self.q), k, v, self.table, self.kvs, self.indptr, self.masks, self.scale)

    def check(self, out, lse, rows=slice(None)):
        ref, rlse, weighted, spread = self.oracle()
        o, s = _f64(out), _f64(lse)
        _within(o[rows], ref[rows], (U * np.abs(ref) + 2 * U * weighted + 2.0 ** -133)[rows], "out")
        empty = np.isneginf(rlse)
        assert np.array_equal(np.isneginf(s)[rows], empty[rows])
        assert not o[rows][empty[rows]].any()
        tol = 2.0 ** -20 * (spread + np.abs(np.where(empty, 0, rlse)) + 1)
        _within(np.where(empty, 0, s)[rows], np.where(empty, 0, rlse)[rows], tol[rows], "lse")


ATTN = [  # ns, kvs, n_q, n_kv, D, page, mask
    ([1], [1], 4, 4, 64, 16, "none"),
    ([1, 1, 1], [1, 16, 17], 32, 8, 128, 16, "none"),
    ([1, 1], [700, 129], 8, 1, 128, 32, "none"),
    ([1] * 5, [5000, 33, 128, 127, 2048], 32, 8, 128, 64, "none"),
    ([1, 0, 1, 0], [300, 200, 31, 0], 5, 1, 64, 16, "none"),
    ([7, 3, 5], [1000, 3, 40], 28, 4, 64, 32, "none"),
    ([16, 9], [777, 16], 32, 8, 128, 16, "tree"),
    ([64, 1, 33], [100, 600, 257], 8, 2, 128, 16, "tree"),
    ([100, 70], [140, 300], 6, 2, 64, 64, "tree"),
    ([13, 20], [13, 20], 6, 6, 128, 16, "any"),
    ([130, 64], [130, 500], 3, 1, 64, 128, "any"),
    ([300], [430], 4, 2, 128, 16, "none"),
    ([4, 2], [900, 65], 8, 2, 256, 32, "tree"),
    ([40, 1], [45, 300], 15, 3, 256, 16, "any"),
    ([1], [40000], 16, 2, 128, 1024, "none"),
    ([2, 1], [90000, 70], 8, 1, 64, 16, "none"),
    ([1] * 300, [1 + (37 * b) % 90 for b in range(300)], 2, 1, 64, 16, "none"),
    # more units than workgroups, of 80 to 132 rows each: a workgroup goes from tree to tree
    ([20 + b % 14 for b in range(48)], [60 + 29 * b % 190 for b in range(48)], 32, 8, 128, 16, "tree"),
    ([9 + b % 6 for b in range(50)], [15 + 53 * b % 400 for b in range(50)], 32, 8, 64, 32, "any"),
    ([33, 32], [33, 300], 128, 64, 64, 16, "none"),
    # prompts and chunks of many row blocks, which see more and more keys
    ([700, 130], [700, 900], 8, 2, 64, 64, "none"),
    ([400, 0, 129, 1], [400, 30, 731, 300], 14, 2, 128, 16, "none"),
    ([517], [1200], 1, 1, 256, 32, "none"),
    ([150, 260], [150, 300], 24, 1, 128, 128, "none"),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ns,kvs,n_q,n_kv,D,page,mask", ATTN)
def test_tree_attention(ns, kvs, n_q, n_kv, D, page, mask, fp8):
    print("[case] tree_attention", ns[:5], kvs[:5], n_q, n_kv, D, page, mask, fp8, flush=True)
    b = Batch(8, ns, kvs, n_q, n_kv, D, page, fp8, mask, extra=8 if len(ns) == 2 else 0)
    b.check(*b.run())


@pytest.mark.parametrize("fp8", [False, True])
def test_attention_ignores_what_is_not_seen(fp8):
    """NaN and infinities in the cache past a sequence's end, in other pages and in drafted keys
    that a row does not see; rows that do see one get it."""
    torch = _torch()
    print("[case] NaN in keys that are not seen", fp8, flush=True)
    for D, n_q, n_kv in ((128, 4, 2), (64, 20, 2), (256, 3, 1), (128, 1024, 256), (64, 1024, 256)):
        b = Batch(9, [6, 9], [133, 40], n_q, n_kv, D, 16, fp8, "any")
        clean = b.run()
        b.check(*clean)
        every, nan = slice(None), float("nan")
        used = {(b.table[s, k // 16], k % 16) for s in (0, 1) for k in range(b.kvs[s])}
        for p in range(b.n_pages):
            for o in range(16):
                if (p, o) not in used:
                    _put(b.k, (p, every, o), 0x7f, nan)
                    _put(b.v, (p, every, o), 0xff, nan if o % 2 else float("inf"))
        out = b.run()
        assert torch.equal(out[0], clean[0]) and torch.equal(out[1], clean[1])
        # drafted key 4 of sequence 1 (cache place 35): not a number in some of its values
        page, off = b.table[1, 35 // 16], 35 % 16
        _put(b.v, (page, every, off, slice(5, 9)), 0x7f, nan)
        sees = np.array([bool(m >> 4 & 1) for m in b.masks[6:]])
        assert sees.any() and not sees.all()
        got = _f64(b.run()[0])[6:]
        is_nan = np.isnan(got)
        assert is_nan[sees][..., 5:9].all() and not is_nan[..., :5].any() and not is_nan[..., 9:].any()
        assert not is_nan[~sees].any()
        far = np.abs(got - _f64(clean[0])[6:])[~is_nan]
        assert far.max() <= 4 * U * np.abs(_f64(clean[0])).max()
        # and in its key: rows that see it are NaN throughout, the others as they were
        _put(b.v, (page, every, off), 0x28, 0.25)
        _put(b.k, (page, every, off, 7), 0x7f, nan)
        got = np.isnan(_f64(b.run()[0])[6:])
        assert got[sees].all() and not got[~sees].any()


def test_attention_empty_rows_and_large_scores():
    torch = _torch()
    print("[case] empty rows, large scores", flush=True)
    b = Batch(10, [5, 3], [5, 300], 4, 2, 64, 16, False, "any", q_std=60.0)
    b.masks[0] = b.masks[3] = 0
    out, lse = b.run()
    b.check(out, lse)
    assert not out[0].any() and (lse[0] == float("-inf")).all() and torch.isfinite(lse[5:]).all()
    # a query of infinity: its own row only
    keep = b.run()
    b.q[6, 1, 3] = float("inf")
    out, lse = b.run()
    rows = [r for r in range(8) if r != 6]
    assert torch.equal(out[rows], keep[0][rows]) and not torch.isfinite(lse[6, 1]) and torch.equal(out[6, [0, 2, 3]], keep[0][6, [0, 2, 3]])


def test_attention_rows_of_nan():
    """A row that sees only keys that are not numbers is NaN, not empty."""
    torch = _torch()
    print("[case] rows of NaN", flush=True)
    b = Batch(16, [2], [2], 2, 1, 64, 16, False, "any")
    b.masks = [1, 2]
    b.k[b.table[0, 0], :, 1] = float("nan")
    out, lse = b.run()
    assert torch.isfinite(out[0]).all() and torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()


def test_attention_data_errors():
    torch = _torch()
    import precision_gemm_amd as P
    print("[case] pages, lengths and offsets that do not fit", flush=True)
    b = Batch(11, [1, 2, 1, 1], [100, 50, 20, 64], 4, 2, 128, 16, False)
    clean = b.run()
    b.check(*clean)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    b.run(status=status)
    assert status.item() == 0
    # a page that does not exist: its 16 keys count as not seen
    was = b.table[0, 2]
    for wrong in (-5, b.n_pages, 2 ** 31 - 1):
        status.zero_()
        b.table[0, 2] = wrong
        out, lse = b.run(status=status)
        assert status.item() == P.LORA_ATTN_BAD_PAGE
        k, v = _f64(b.k), _f64(b.v)
        pages = [p for i, p in enumerate(b.table[0, :7]) if i != 2]
        ref, rl, w, sp = A.tree_attention(_f64(b.q)[:1], k, v, [pages], [84], [0, 1], None, b.scale)
        _within(_f64(out)[:1], ref, U * np.abs(ref) + 2 * U * w, "out without the page")
        assert torch.equal(out[1:], clean[0][1:]) and torch.equal(lse[1:], clean[1][1:])
    b.table[0, 2] = was
    # lengths below the drafted tokens or past the pages: taken as empty
    for wrong in (1, -3, 16 * b.table.shape[1] + 1):
        kvs = list(b.kvs)
        b.kvs[1] = wrong
        status.zero_()
        out, lse = b.run(status=status)
        assert status.item() == P.LORA_ATTN_BAD_LENGTH
        assert not out[1:3].any() and (lse[1:3] == float("-inf")).all()
        assert torch.equal(out[[0, 3, 4]], clean[0][[0, 3, 4]])
        b.kvs = kvs
    # offsets that leave the call, or more tokens than max_q: left out, the rest as before
    for indptr in ([0, 1, 3, 4, 9], [0, 1, 0, 4, 5], [-2, 1, 3, 4, 5]):
        keep, b.indptr = b.indptr, np.array(indptr)
        status.zero_()
        mark = torch.full_like(clean[0], 3.0)
        out, _ = b.run(status=status, out=mark)
        assert status.item() == P.LORA_ATTN_BAD_LENGTH
        b.indptr = keep
        for s, (lo, hi) in enumerate(zip(keep[:-1], keep[1:])):
            if indptr[s] == lo and indptr[s + 1] == hi:
                assert torch.equal(out[lo:hi], clean[0][lo:hi])


def test_attention_length_errors_between_prompts():
    """Sequences whose lengths do not fit, between prompts of many row blocks."""
    torch = _torch()
    import precision_gemm_amd as P
    print("[case] lengths that do not fit between prompts", flush=True)
    b = Batch(15, [150, 200, 90], [150, 333, 90], 8, 2, 64, 16, False)
    for wrong in (10, 0, -7):
        was, b.kvs = b.kvs, [150, wrong, 90]
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = b.run(status=status)
        b.kvs = was
        assert status.item() == P.LORA_ATTN_BAD_LENGTH
        assert not out[150:350].any() and (lse[150:350] == float("-inf")).all()
        for rows in (slice(0, 150), slice(350, 440)):
            b.check(out, lse, rows)


def test_attention_same_bits_whatever_the_workspace():
    """Bitwise the same again, whatever the workspace holds, on another stream, and with any mask
    bits past a sequence's tokens."""
    torch = _torch()
    import precision_gemm_amd as P
    print("[case] workspace, stream", flush=True)
    b = Batch(12, [3, 1, 5], [3000, 900, 100], 8, 2, 128, 32, False, "tree")
    want = b.run()
    b.check(*want)
    for fill in (0, 255):
        ws = torch.full((P.tree_attention_workspace_bytes(8, 2, 128, 5),), fill, dtype=torch.uint8, device="cuda")
        out, lse = torch.full_like(want[0], float("nan")), torch.full_like(want[1], float("nan"))
        got = b.run(workspace=ws, out=out, lse=lse)
        assert got[0] is out and torch.equal(out, want[0]) and torch.equal(lse, want[1])
    # one workspace for calls of different heads, lengths and numbers of rows
    big = torch.full((96 << 20,), 255, dtype=torch.uint8, device="cuda")
    others = [Batch(20 + i, ns, kvs, n_q, n_kv, D, 16, False) for i, (ns, kvs, n_q, n_kv, D) in enumerate([
        ([1], [30000], 4, 1, 64), ([40, 1], [700, 5000], 8, 1, 128), ([3], [9000], 2, 1, 256), ([1] * 9, [2000] * 9, 8, 8, 128)])]
    alone = [o.run() for o in others]
    for _ in range(2):
        for o, (a, l) in zip(others, alone):
            got = o.run(workspace=big)
            assert torch.equal(got[0], a) and torch.equal(got[1], l)
    others[0].check(*alone[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = b.run()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    masked = b.run(tree_mask=b.mask_tensor(junk=False))
    assert torch.equal(masked[0], want[0])


def test_large_cache_offsets():
    """A cache of more than 4 GiB: keys at byte and element offsets past 32 bits."""
    torch = _torch()
    import precision_gemm_amd as P
    print("[case] offsets past 32 bits", flush=True)
    n_kv, page, D, n_pages = 8, 64, 128, 70000  # 65,536 elements a page: 4.6e9 elements, 9.2e9 bytes
    rng = np.random.default_rng(13)
    k = torch.zeros((n_pages, n_kv, page, D), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros((n_pages, n_kv, page, D), dtype=torch.bfloat16, device="cuda")
    ids = [69999, 3, 69000, 40000]
    kv, n_q = 200, 16
    qkv, x = _bf(rng, (kv, (n_q + 2 * n_kv) * D))
    slots = np.array([ids[i // page] * page + i % page for i in range(kv)])
    cs = P.rope_table(256, 128)
    q = P.rope_append_kv(qkv, _i32(np.arange(kv)), _i32(slots), k, v, n_q, cos_sin=cs)
    rows = A.norm_rope(x.reshape(kv, -1, D)[:, n_q:n_q + n_kv], np.arange(kv), _f64(cs), None, 0.0)
    got = np.stack([_f64(k[s // page, :, s % page]) for s in slots])
    _within(got, rows, U * np.abs(rows) + 2.0 ** -17 * (np.abs(rows).max()), "k")
    out, lse = P.tree_attention(q[-2:], k, v, _i32([ids]), _i32([kv]), _i32([0, 2]), 2)
    sub = np.array(ids)
    ref, rl, w, sp = A.tree_attention(_f64(q[-2:]), _f64(k[sub]), _f64(v[sub]), [[0, 1, 2, 3]], [kv], [0, 2], None, 1 / np.sqrt(D))
    _within(_f64(out), ref, U * np.abs(ref) + 2 * U * w, "out")
    _within(_f64(lse), rl, 2.0 ** -20 * (sp + np.abs(rl) + 1), "lse")


def test_block_in_one_graph():
    """Append, masks and attention captured in one graph and replayed with eager work in
    between; every replay equals the eager calls bit for bit."""
    torch = _torch()
    import precision_gemm_amd as P
    print("[case] graph replay", flush=True)
    rng = np.random.default_rng(14)
    n_q, n_kv, D, page, ns, kvs = 32, 8, 128, 16, [4, 1, 7], [500, 33, 1000]
    T, width = sum(ns), (n_q + 2 * n_kv) * D
    b = Batch(15, ns, kvs, n_q, n_kv, D, page, False, "tree")
    qkv, _ = _bf(rng, (T, width))
    slots, positions = [], []
    for s, (n, kv) in enumerate(zip(ns, kvs)):
        for j in range(n):
            i = kv - n + j
            slots.append(b.table[s, i // page] * page + i % page)
            positions.append(i)
    parents = _i32([-1 if j == 0 else j - 1 for n in ns for j in range(n)])
    dev = dict(pos=_i32(positions), slots=_i32(slots), table=_i32(b.table), kvs=_i32(kvs), indptr=_i32(b.indptr))
    cs = P.rope_table(1024, 128)
    w = torch.ones(D, device="cuda")
    q_out = torch.empty((T, n_q, D), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty_like(q_out), torch.empty((T, n_q), device="cuda")
    ws = torch.empty(P.tree_attention_workspace_bytes(n_q, n_kv, D, 7), dtype=torch.uint8, device="cuda")
    dq, dk = torch.randn_like(q_out), torch.randn((T, n_kv, D), device="cuda").bfloat16()
    grads = [torch.empty((T, width), dtype=torch.bfloat16, device="cuda"), torch.empty(D, device="cuda"), torch.empty(D, device="cuda")]
    bws = torch.empty(P.qk_norm_rope_backward_workspace_bytes(T, D), dtype=torch.uint8, device="cuda")

    def chain():
        P.rope_append_kv(qkv, dev["pos"], dev["slots"], b.k, b.v, n_q, cos_sin=cs, q_weight=w, k_weight=w, q_out=q_out)
        m = P.tree_mask(parents, dev["indptr"], 7)
        P.tree_attention(q_out, b.k, b.v, dev["table"], dev["kvs"], dev["indptr"], 7, tree_mask=m, out=out, lse=lse, workspace=ws)
        P.qk_norm_rope_backward(qkv, dev["pos"], dq, dk, dk, cos_sin=cs, q_weight=w, k_weight=w, dqkv=grads[0],
                                dq_weight=grads[1], dk_weight=grads[2], workspace=bws)

    chain()
    torch.cuda.synchronize()
    want = [t.clone() for t in (q_out, out, lse, b.k, b.v, *grads)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        chain()
    for rep in range(3):
        for t in (q_out, out, lse, *grads):
            t.fill_(-7)
        ws.fill_(rep * 100)
        bws.fill_(255)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, t in zip(want, (q_out, out, lse, b.k, b.v, *grads)):
            assert torch.equal(a, t), f"replay {rep}"
