"""Norms at both ends of every width that has a form of its own, each with and without the mean, the
residual (backwards: its gradient) and the weights' gradients, for fewer rows than a workgroup takes and
for more than all workgroups take at once.  Tolerances: tests/test_gpu_norm.py."""

import numpy as np
import pytest

from oracle import step as S
from test_gpu_norm import U, _bf, _f32, _f64, _sizes, _within

pytestmark = pytest.mark.gpu

WIDTHS = [8, 504, 512, 520, 1024, 1032, 2048, 2056, 4096, 4104, 6144, 6152, 8192, 8200, 12288, 16384]


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("K", WIDTHS)
def test_forward(K, residual, rms):
    import torch
    import precision_gemm_amd as P
    T = 37
    print("[case] norm width", K, residual, rms, flush=True)
    rng = np.random.default_rng(K)
    x, res = _bf(rng, (T, K), 1.5, 0.3)[0], _bf(rng, (T, K))[0] if residual else None
    w, b = _f32(rng, K, 0.2, 1.0), _f32(rng, K, 0.2)
    y, h = P.layer_norm(x, w, b, residual=res, eps=1e-5, rms=rms)
    assert torch.equal(h, (x.float() + res.float()).bfloat16() if residual else x)
    hn, wn, bn = _f64(h), _f64(w), _f64(b)
    ref = S.layer_norm(hn, wn, bn, 1e-5, rms)
    size = _sizes(hn, wn, 1e-5, rms)[2]
    _within(_f64(y), ref, U * np.abs(ref) + 2.0 ** -18 * (size * np.abs(wn) + np.abs(ref) + np.abs(bn)) + 2.0 ** -133, "y")


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dsum", [False, True])
@pytest.mark.parametrize("T", [3, 1301])
@pytest.mark.parametrize("K", WIDTHS)
def test_backward(K, T, dsum, rms):
    import torch
    import precision_gemm_amd as P
    if T * K > 1301 * 8200:
        T = 530  # more rows than workgroups all the same
    print("[case] norm width backward", K, T, dsum, rms, flush=True)
    rng = np.random.default_rng(K + T)
    (h, hn), (dy, dyn) = _bf(rng, (T, K), 1.5, 0.3), _bf(rng, (T, K), 0.02, 0.001)
    ds, dsn = _bf(rng, (T, K), 0.02) if dsum else (None, 0.0)
    w = _f32(rng, K, 0.2, 1.0)
    wn = _f64(w)
    dx, dw, db = P.layer_norm_backward(dy, h, w, dsum=ds, eps=1e-5, rms=rms)
    ref, dwr, dbr = S.layer_norm_backward(dyn, hn, wn, 1e-5, rms, None if ds is None else dsn)
    r, xh, size = _sizes(hn, wn, 1e-5, rms)
    g = np.abs(dyn * wn)
    terms = r * (g + (0 if rms else g.mean(1, keepdims=True)) + (np.abs(xh) + size) * (g * (np.abs(xh) + 2.0 ** -2 * size)).mean(1, keepdims=True))
    _within(_f64(dx), ref, U * np.abs(ref) + 2.0 ** -16 * (terms + np.abs(dsn)) + 2.0 ** -133, "dx")
    _within(_f64(dw), dwr, 2.0 ** -16 * np.abs(dyn * xh).sum(0) + 2.0 ** -18 * (np.abs(dyn) * size).sum(0), "dweight")
    _within(_f64(db), dbr, 2.0 ** -16 * np.abs(dyn).sum(0), "dbias")
    for weight_grad, bias_grad in ((False, False), (True, False), (False, True)):
        got = P.layer_norm_backward(dy, h, w, dsum=ds, eps=1e-5, rms=rms, weight_grad=weight_grad, bias_grad=bias_grad)
        assert torch.equal(got[0], dx)
        assert torch.equal(got[1], dw) if weight_grad else got[1] is None
        assert torch.equal(got[2], db) if bias_grad else got[2] is None
