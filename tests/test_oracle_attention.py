"""Pins of the attention block's oracle: hand-worked values, complex-number rotation, central
differences for the gradients, and attention against dense arithmetic."""

import numpy as np
import pytest

from oracle import attention as A


def _table(n, rot, theta=100.0):
    a = np.arange(n)[:, None] * theta ** (-np.arange(rot // 2) * 2.0 / rot)
    return np.concatenate([np.cos(a), np.sin(a)], 1)


def test_rotation_by_hand():
    cs = np.array([[1.0, 0.0], [0.0, 1.0]])  # positions 0: no turn, 1: a quarter turn; rot 2
    x = np.array([[[3.0, 4.0, 5.0]], [[3.0, 4.0, 5.0]]])
    assert np.array_equal(A.rotate(x, [0, 1], cs), [[[3, 4, 5]], [[-4, 3, 5]]])
    assert np.array_equal(A.rotate(x, [1, 0], cs, sign=-1.0), [[[4, -3, 5]], [[3, 4, 5]]])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_as_complex_numbers(interleaved):
    rng = np.random.default_rng(0)
    x, pos, rot = rng.standard_normal((5, 3, 12)), np.array([0, 3, 9, 2, 9]), 8
    ang = pos[:, None] * 100.0 ** (-np.arange(4) / 4)
    z = np.exp(1j * ang)[:, None]
    y = A.rotate(x, pos, _table(10, rot), interleaved)
    pair = (lambda v: v[..., 0:8:2] + 1j * v[..., 1:8:2]) if interleaved else (lambda v: v[..., :4] + 1j * v[..., 4:8])
    assert np.allclose(pair(y), pair(x) * z, atol=1e-12) and np.array_equal(y[..., 8:], x[..., 8:])
    assert np.allclose(A.rotate(y, pos, _table(10, rot), interleaved, sign=-1.0), x, atol=1e-12)


def test_norm_by_hand():
    y = A.norm_rope(np.array([[[3.0, 4.0]]]), None, None, np.array([2.0, 1.0]), 0.0)
    assert np.allclose(y, np.array([[[6.0, 4.0]]]) / np.sqrt(12.5))


@pytest.mark.parametrize("interleaved,rot,norm", [(False, 8, True), (True, 4, True), (False, 8, False)])
def test_gradients_against_differences(interleaved, rot, norm):
    rng = np.random.default_rng(1)
    x, dy, pos = rng.standard_normal((3, 2, 8)), rng.standard_normal((3, 2, 8)), np.array([4, 0, 7])
    w, cs, h = (rng.standard_normal(8) if norm else None), _table(8, rot), 1e-6
    f = lambda x, w: (A.norm_rope(x, pos, cs, w, 1e-3, interleaved) * dy).sum()  # noqa: E731
    dx, dw = A.norm_rope_backward(x, dy, pos, cs, w, 1e-3, interleaved)
    for idx in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[idx] = h
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - dx[idx]) < 1e-7
    for d in range(8 if norm else 0):
        e = np.zeros(8)
        e[d] = h
        assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - dw[d]) < 1e-7


def test_append_and_mask():
    c = A.append(np.zeros((2, 1, 4, 2)), np.arange(6.0).reshape(3, 1, 2), [5, -1, 0])
    assert np.array_equal(c[1, 0, 1], [0, 1]) and np.array_equal(c[0, 0, 0], [4, 5]) and np.count_nonzero(c) == 3
    assert A.tree_mask([-1, 0, 0, 2, -1, 0], [0, 4, 4, 6]) == [1, 3, 5, 13, 1, 3]


def test_attention_against_dense():
    rng = np.random.default_rng(2)
    page, D, kv, n = 4, 8, 10, 3
    kc, vc, q = rng.standard_normal((5, 2, page, D)), rng.standard_normal((5, 2, page, D)), rng.standard_normal((n, 4, D))
    table = np.array([[3, 0, 4]])
    masks = [1, 3, 5]
    out, lse, _, _ = A.tree_attention(q, kc, vc, table, [kv], [0, n], masks, 0.3)
    k = np.concatenate([kc[3], kc[0], kc[4]], 1)[:, :kv]
    v = np.concatenate([vc[3], vc[0], vc[4]], 1)[:, :kv]
    s = np.einsum("jhd,hkd->jhk", q, np.repeat(k, 2, 0)) * 0.3
    for j in range(n):
        for i in range(n):
            if not masks[j] >> i & 1:
                s[j, :, kv - n + i] = -np.inf
    p = np.exp(s)
    assert np.allclose(lse, np.log(p.sum(-1)))
    assert np.allclose(out, np.einsum("jhk,hkd->jhd", p / p.sum(-1, keepdims=True), np.repeat(v, 2, 0)))


def test_empty_rows():
    z = np.zeros((1, 1, 4, 8))
    out, lse, _, _ = A.tree_attention(np.ones((2, 1, 8)), z + 1, z + 1, [[0]], [2], [0, 2], [1, 0], 1.0)
    assert np.array_equal(out[0, 0], np.ones(8)) and np.array_equal(out[1, 0], np.zeros(8)) and lse[1, 0] == -np.inf
