"""Pins of the oracle for norms and the AdamW step: hand-worked values and central differences; and of
the rotation by positions of several axes."""

import numpy as np
import pytest

from oracle import attention as A
from oracle import step as S


def test_norms_by_hand():
    x = np.array([[1.0, 3.0, 5.0, 7.0]])  # mean 4, variance 5, mean square 21
    assert np.allclose(S.layer_norm(x, None, None, 4.0), [[-1.0, -1 / 3, 1 / 3, 1.0]])
    w, b = np.array([2.0, 3.0, 0.0, 1.0]), np.array([0.0, 1.0, 1.0, 0.0])
    assert np.allclose(S.layer_norm(x, w, b, 4.0), [[-2.0, 0.0, 1.0, 1.0]])
    assert np.allclose(S.layer_norm(x, w, None, 4.0, rms=True), [[0.4, 1.8, 0.0, 1.4]])


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("weighted", [False, True])
def test_norm_gradients_against_differences(rms, weighted):
    rng = np.random.default_rng(0)
    x, dy, ds = (rng.standard_normal((3, 8)) for _ in range(3))
    w, b = (rng.standard_normal(8) if weighted else np.ones(8)), rng.standard_normal(8)
    f = lambda x, w, b: (S.layer_norm(x, w, b, 1e-2, rms) * dy).sum() + (x * ds).sum()  # noqa: E731
    dx, dw, db = S.layer_norm_backward(dy, x, w if weighted else None, 1e-2, rms, ds)
    h = 1e-6
    for at in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[at] = h
        assert abs((f(x + e, w, b) - f(x - e, w, b)) / (2 * h) - dx[at]) < 1e-7
    for d in range(8):
        e = np.zeros(8)
        e[d] = h
        assert abs((f(x, w + e, b) - f(x, w - e, b)) / (2 * h) - dw[d]) < 1e-7
        assert abs((f(x, w, b + e) - f(x, w, b - e)) / (2 * h) - db[d]) < 1e-7


def test_adamw_by_hand():
    # the first step: m / (1 - beta1) = g, sqrt(v / (1 - beta2)) = |g|
    p, m, v = S.adamw([1.0, -2.0], [4.0, -0.5], [0.0, 0.0], [0.0, 0.0], 1, 0.1, 0.9, 0.99, 0.0, 0.5)
    assert np.allclose(p, [1.0 - 0.05 - 0.1, -2.0 + 0.1 + 0.1]) and np.allclose(m, [0.4, -0.05]) and np.allclose(v, [0.16, 0.0025])
    # the second, with another gradient
    p, m, v = S.adamw([0.0], [2.0], [0.4], [0.16], 2, 0.1, 0.9, 0.99, 1.0, 0.0)
    mh, vh = 0.56 / 0.19, 0.1984 / 0.0199
    assert np.allclose(p, -0.1 * mh / (np.sqrt(vh) + 1)) and np.allclose(m, 0.56) and np.allclose(v, 0.1984)


def test_clipping_and_scales():
    assert S.clip_factor(2.0, 1.0) == 1.0 / (2.0 + 1e-6) and S.clip_factor(0.5, 1.0) == 1.0 and S.clip_factor(9.0, 0.0) == 1.0
    x = np.zeros(100)
    x[3], x[99] = -7.0, 448.0
    assert np.array_equal(S.held(x), [7.0 / 448, 1.0])


@pytest.mark.parametrize("interleaved", [False, True])
def test_axes_as_complex_numbers(interleaved):
    rng = np.random.default_rng(1)
    x, pos, axes = rng.standard_normal((5, 3, 12)), rng.integers(0, 10, (3, 5)), [0, 2, 1, 2]
    f = 100.0 ** (-np.arange(4) / 4)
    a = np.arange(10)[:, None] * f
    cs = np.concatenate([np.cos(a), np.sin(a)], 1)
    z = np.exp(1j * pos[axes].T * f)[:, None]
    y = A.rotate(x, pos, cs, interleaved, axes=axes)
    pair = (lambda v: v[..., 0:8:2] + 1j * v[..., 1:8:2]) if interleaved else (lambda v: v[..., :4] + 1j * v[..., 4:8])
    assert np.allclose(pair(y), pair(x) * z, atol=1e-12) and np.array_equal(y[..., 8:], x[..., 8:])
    same = np.stack([pos[0]] * 3)  # positions that go together: the rotation by one of them
    assert np.array_equal(A.rotate(x, same, cs, interleaved, axes=axes), A.rotate(x, pos[0], cs, interleaved))
