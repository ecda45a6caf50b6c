"""GPU parity of the head norms and rotation with positions of several axes (forward, backward, append)
with the fp64 oracle.  Tolerances are those of the calls with one position a token, derived beside them
(tests/test_gpu_attention.py): the arithmetic is the same, only the table's rows differ by pair."""

import numpy as np
import pytest

from oracle import attention as A
from test_gpu_attention import U, _bf, _f64, _i32, _pair_size, _torch, _within

pytestmark = pytest.mark.gpu

MAX_POS = 400

CASES = [  # T, n_q, n_kv, D, rot, interleaved rotation, norm, sections, axes in turn
    (1, 32, 8, 128, 128, False, True, (16, 24, 24), False),
    (7, 28, 4, 64, 32, True, True, (4, 8, 4), False),
    (33, 5, 1, 256, 256, False, True, (64, 32, 32), False),
    (130, 15, 3, 128, 64, False, False, (11, 11, 10), True),
    (3, 3, 3, 256, 16, True, False, (1, 3, 2, 2), False),
    (11, 4, 2, 64, 64, False, True, (32,), False),
    (2, 1, 1, 64, 48, True, True, (7, 17), True),
    (1100, 32, 8, 128, 128, True, True, (24, 20, 20), False),
    (1031, 9, 9, 64, 64, False, True, (8, 0, 24), False),
    (65, 6, 6, 256, 256, True, True, (50, 39, 39), True),
    (40, 8, 1, 128, 128, False, True, (0, 1, 63), False),
]


def _inputs(T, n_q, n_kv, D, rot, norm, sections, mixed, seed, extra=8):
    torch = _torch()
    import precision_gemm_amd as P
    rng = np.random.default_rng(seed)
    width = (n_q + 2 * n_kv) * D
    qkv, x = _bf(rng, (T, width + extra), 1.5)
    pos = rng.integers(0, MAX_POS, (len(sections), T))
    w = [torch.from_numpy((1 + 0.2 * rng.standard_normal(D)).astype(np.float32)).cuda() if norm else None for _ in range(2)]
    axes = P.rope_pair_axes(sections, mixed)
    assert len(axes) == rot // 2
    return rng, qkv[:, :width], x[:, :width].reshape(T, -1, D), pos, P.rope_table(MAX_POS, rot), w, axes


def _check(got, x, pos, cs, w, inter, axes, what):
    csn, wn = _f64(cs), None if w is None else _f64(w)
    ref = A.norm_rope(x, pos, csn, wn, 1e-5, inter, axes=axes)
    size = _pair_size(A.norm_rope(x, pos, None, wn, 1e-5), csn.shape[1], inter)
    _within(got, ref, U * np.abs(ref) + 2.0 ** -18 * size + 2.0 ** -133, what)
    return ref, size


@pytest.mark.parametrize("T,n_q,n_kv,D,rot,inter,norm,sections,mixed", CASES)
def test_forward(T, n_q, n_kv, D, rot, inter, norm, sections, mixed):
    torch = _torch()
    import precision_gemm_amd as P
    print("[case] axes forward", T, n_q, n_kv, D, rot, inter, norm, sections, mixed, flush=True)
    _, qkv, x, pos, cs, (qw, kw), axes = _inputs(T, n_q, n_kv, D, rot, norm, sections, mixed, 1)
    args = dict(cos_sin=cs, q_weight=qw, k_weight=kw, eps=1e-5, interleaved=inter)
    q, k = P.qk_norm_rope(qkv, _i32(pos), n_q, n_kv, D, pair_axes=axes, **args)
    _check(_f64(q), x[:, :n_q], pos, cs, qw, inter, axes, "q")
    _check(_f64(k), x[:, n_q:n_q + n_kv], pos, cs, kw, inter, axes, "k")
    # positions that go together on all axes are one position a token, to the bit
    same = _i32(np.stack([pos[0]] * len(sections)))
    a, b = P.qk_norm_rope(qkv, same, n_q, n_kv, D, pair_axes=axes, **args), P.qk_norm_rope(qkv, same[0], n_q, n_kv, D, **args)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("T,n_q,n_kv,D,rot,inter,norm,sections,mixed", CASES)
def test_backward(T, n_q, n_kv, D, rot, inter, norm, sections, mixed):
    torch = _torch()
    import precision_gemm_amd as P
    print("[case] axes backward", T, n_q, n_kv, D, rot, inter, norm, sections, mixed, flush=True)
    rng, qkv, x, pos, cs, (qw, kw), axes = _inputs(T, n_q, n_kv, D, rot, norm, sections, mixed, 2)
    (dq, dqn), (dk, dkn), (dv, dvn) = (_bf(rng, (T, n, D), 0.02) for n in (n_q, n_kv, n_kv))
    args = dict(cos_sin=cs, q_weight=qw, k_weight=kw, eps=1e-5, interleaved=inter, pair_axes=axes)
    dqkv, dqw, dkw = P.qk_norm_rope_backward(qkv, _i32(pos), dq, dk, dv, **args)
    got, csn = _f64(dqkv).reshape(T, -1, D), _f64(cs)
    assert torch.equal(dqkv.view(T, -1, D)[:, n_q + n_kv:], dv)
    for name, xs, dy, w, g, dw in (("q", x[:, :n_q], dqn, qw, got[:, :n_q], dqw),
                                   ("k", x[:, n_q:n_q + n_kv], dkn, kw, got[:, n_q:n_q + n_kv], dkw)):
        wn = None if w is None else _f64(w)
        ref, dwr = A.norm_rope_backward(xs, dy, pos, csn, wn, 1e-5, inter, axes=axes)
        turned = A.rotate(dy, pos, csn, inter, sign=-1.0, axes=axes)
        size = _pair_size(dy, rot, inter)
        if norm:
            r = 1 / np.sqrt((xs * xs).mean(-1, keepdims=True) + 1e-5)
            xh = xs * r
            size = r * (size * np.abs(wn) + np.abs(xh) * (np.abs(turned * wn) * np.abs(xh)).mean(-1, keepdims=True))
            _within(_f64(dw), dwr, 2.0 ** -16 * np.abs(turned * xh).sum((0, 1)), "d" + name + "_weight")
        else:
            assert dw is None
        _within(g, ref, U * np.abs(ref) + 2.0 ** -16 * size + 2.0 ** -133, "d" + name)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,n_q,n_kv,D,rot,inter,norm,sections,mixed", CASES)
def test_append(T, n_q, n_kv, D, rot, inter, norm, sections, mixed, fp8):
    torch = _torch()
    import precision_gemm_amd as P
    print("[case] axes append", T, n_q, n_kv, D, rot, inter, norm, sections, mixed, fp8, flush=True)
    rng, qkv, x, pos, cs, (qw, kw), axes = _inputs(T, n_q, n_kv, D, rot, norm, sections, mixed, 3)
    page = 16
    pages = -(-T // page) + 2
    slots = rng.permutation(pages * page)[:T]
    slots[T // 2] = -1
    shape = (pages, n_kv, page, D)
    scales = [torch.from_numpy(rng.uniform(0.01, 0.02, n_kv).astype(np.float32)).cuda() if fp8 else None for _ in range(2)]
    new = lambda: torch.zeros(shape, device="cuda").to(torch.float8_e4m3fn if fp8 else torch.bfloat16)  # noqa: E731
    args = dict(cos_sin=cs, q_weight=qw, k_weight=kw, eps=1e-5, interleaved=inter, k_scale=scales[0], v_scale=scales[1])
    kc, vc = new(), new()
    q = P.rope_append_kv(qkv, _i32(pos), _i32(slots), kc, vc, n_q, pair_axes=axes, **args)
    _check(_f64(q), x[:, :n_q], pos, cs, qw, inter, axes, "q")
    k, size = _check_keys(x[:, n_q:n_q + n_kv], pos, cs, kw, inter, axes)
    v = x[:, n_q + n_kv:]
    for name, got, ref, sc, tol in (("k", kc, k, scales[0], 2.0 ** -18 * size), ("v", vc, v, scales[1], 0.0 * v)):
        one = 1.0 if sc is None else _f64(sc)[None, :, None]
        ref, tol = ref / one, tol / one
        if fp8:
            ref = np.clip(ref, -448, 448)
            tol = tol * (1 + 2.0 ** -3) + 2.0 ** -4 * np.abs(ref) + 2.0 ** -10 + 2.0 ** -20 * np.abs(ref)
        else:
            tol = tol + U * np.abs(ref) + 2.0 ** -133
        want = A.append(np.zeros(shape), ref, slots)
        _within(_f64(got.float()), want, A.append(np.zeros(shape), np.broadcast_to(tol, ref.shape), slots), name)
    # positions that go together: the call with one position a token, to the bit
    same = _i32(np.stack([pos[0]] * len(sections)))
    c = [new() for _ in range(4)]
    qa = P.rope_append_kv(qkv, same, _i32(slots), c[0], c[1], n_q, pair_axes=axes, **args)
    qb = P.rope_append_kv(qkv, same[0], _i32(slots), c[2], c[3], n_q, **args)
    assert torch.equal(qa, qb) and all(torch.equal(c[i].view(torch.uint8), c[i + 2].view(torch.uint8)) for i in (0, 1))


def _check_keys(x, pos, cs, w, inter, axes):
    csn, wn = _f64(cs), None if w is None else _f64(w)
    return (A.norm_rope(x, pos, csn, wn, 1e-5, inter, axes=axes),
            _pair_size(A.norm_rope(x, pos, None, wn, 1e-5), csn.shape[1], inter))


@pytest.mark.parametrize("sections,mixed", [((8, 12, 12), False), ((11, 11, 10), True)])
def test_positions_outside_the_table(sections, mixed):
    """A token whose position on any axis is outside gets zeros, is not stored, and adds nothing."""
    torch = _torch()
    import precision_gemm_amd as P
    print("[case] outside", sections, flush=True)
    T, n_q, n_kv, D = 9, 4, 2, 64
    rng, qkv, x, pos, cs, (qw, kw), axes = _inputs(T, n_q, n_kv, D, 64, True, sections, mixed, 4)
    pos[0, 1], pos[1, 3], pos[2, 5], pos[2, 8] = -1, MAX_POS, 2 ** 31 - 1, -2 ** 31
    bad = np.array([1, 3, 5, 8])
    ok = np.setdiff1d(np.arange(T), bad)
    args = dict(cos_sin=cs, q_weight=qw, k_weight=kw, eps=1e-5, pair_axes=axes)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, k = P.qk_norm_rope(qkv, _i32(pos), n_q, n_kv, D, status=st, **args)
    assert int(st) == P.LORA_ATTN_BAD_POSITION and not q[bad].any() and not k[bad].any()
    _check(_f64(q)[ok], x[ok, :n_q], pos[:, ok], cs, qw, False, axes, "q")
    dq, dk, dv = (_bf(rng, (T, n, D), 0.02)[0] for n in (n_q, n_kv, n_kv))
    st.zero_()
    dqkv, dqw, dkw = P.qk_norm_rope_backward(qkv, _i32(pos), dq, dk, dv, status=st, **args)
    assert int(st) == P.LORA_ATTN_BAD_POSITION and not dqkv.view(T, -1, D)[bad, :n_q + n_kv].any()
    only = P.qk_norm_rope_backward(qkv[ok].contiguous(), _i32(pos[:, ok]), dq[ok], dk[ok], dv[ok], **args)
    assert torch.allclose(dqw, only[1], rtol=1e-5, atol=1e-7) and torch.allclose(dkw, only[2], rtol=1e-5, atol=1e-7)
    cache = [torch.full((2, n_kv, 16, D), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    st.zero_()
    P.rope_append_kv(qkv, _i32(pos), _i32(np.arange(T)), cache[0], cache[1], n_q, status=st, **args)
    assert int(st) == P.LORA_ATTN_BAD_POSITION
    assert (cache[0][0, :, bad] == 5).all() and (cache[1][0, :, bad] == 5).all() and not (cache[0][0, :, ok] == 5).all()


def test_refusals():
    torch = _torch()
    import precision_gemm_amd as P
    qkv, cs = torch.zeros((3, 4 * 64), dtype=torch.bfloat16, device="cuda"), P.rope_table(10, 64)
    pos = torch.zeros((3, 3), dtype=torch.int32, device="cuda")
    axes = P.rope_pair_axes((16, 8, 8))
    ok = dict(cos_sin=cs, pair_axes=axes)
    P.qk_norm_rope(qkv, pos, 2, 1, 64, **ok)
    for kw, match in ((dict(pair_axes=axes[:31]), "32 pairs"), (dict(pair_axes=list(axes)), "must be bytes"),
                      (dict(pair_axes=bytes([3]) + axes[1:]), "names axis 3 of 3"), (dict(cos_sin=None), "is for a rotation"),
                      (dict(positions=pos[0]), "positions must be"), (dict(positions=pos[:2]), "names axis 2 of 2"),
                      (dict(positions=torch.zeros((5, 3), dtype=torch.int32, device="cuda")), "positions must be"),
                      (dict(positions=pos[:, :2]), "positions must have shape"), (dict(positions=pos.long()), "positions must have dtype"),
                      (dict(positions=None), "positions must be a tensor"), (dict(pair_axes=None), "positions must have shape")):
        args = {**dict(positions=pos), **ok, **kw}
        with pytest.raises(ValueError, match=match):
            P.qk_norm_rope(qkv, args.pop("positions"), 2, 1, 64, **args)
    # no rotation at all needs no positions
    with pytest.raises(ValueError, match="is for a rotation"):
        P.qk_norm_rope(qkv, None, 2, 1, 64, pair_axes=b"")
