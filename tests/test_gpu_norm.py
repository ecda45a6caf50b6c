"""GPU parity of the norms of the hidden states and their gradients with the fp64 oracle.

Tolerances, from the arithmetic (u = 2^-8 is half a step of bf16, relative; v = 2^-24 of fp32):
 * forward: y is rounded once, u |y|; before that the fp32 steps: a mean of K <= 16,384 values summed
   in at most 16 + 6 + 4 levels (v each, of the mean magnitude), the deviation's subtraction (v of the
   value and of the mean), r (2^-20), three products and a sum: 2^-18 (|h| + mean|h|) r |w| and 2^-18
   |y| + |b| cover them;
 * h is the correctly rounded sum: exact;
 * dx: u |dx|, and 2^-16 of the terms that are subtracted, r (|g| + mean|g| + |xh| mean|g xh|), |dsum|;
 * dweight, dbias: 2^-16 of the sum of magnitudes (fp32 partial sums over at most 65,536 / 256 rows, and
   256 partial rows in order), with the deviation's own error 2^-18 (|h| + mean|h|) r of each term.
"""

import numpy as np
import pytest

from oracle import step as S

pytestmark = pytest.mark.gpu

U = 2.0 ** -8


def _torch():
    import torch
    return torch


def _bf(rng, shape, std=1.0, mean=0.0, extra=0):
    """bf16 device tensor (rows of ``extra`` more values in memory) and its values in fp64."""
    torch = _torch()
    a = (rng.standard_normal((shape[0], shape[1] + extra)) * std + mean).astype(np.float32)
    t = torch.from_numpy(a).to(torch.bfloat16).cuda()[:, :shape[1]]
    return t, t.double().cpu().numpy()


def _f32(rng, n, std, mean=0.0):
    return _torch().from_numpy((mean + std * rng.standard_normal(n)).astype(np.float32)).cuda()


def _f64(t):
    return t.detach().double().cpu().numpy()


def _within(got, ref, tol, what):
    assert np.isfinite(got).all(), f"{what}: not finite"
    over = np.abs(got - ref) - tol
    at = over.argmax()
    assert (over <= 0).all(), f"{what}: off by {np.abs(got - ref).flat[at]:.3e}, allowed {np.broadcast_to(tol, over.shape).flat[at]:.3e}"


def _sizes(h, w, eps, rms):
    """1 / deviation, xh, and the error scale of xh."""
    mean = np.zeros_like(h[:, :1]) if rms else h.mean(1, keepdims=True)
    r = 1 / np.sqrt(((h - mean) ** 2).mean(1, keepdims=True) + eps)
    return r, (h - mean) * r, (np.abs(h) + (0 if rms else np.abs(h).mean(1, keepdims=True))) * r


CASES = [  # T, K, rms, residual, weight, bias, extra values of a row, mean of the rows
    (1, 8, False, False, True, True, 0, 0.0),
    (1, 4096, False, True, True, True, 0, 0.0),
    (3, 64, True, False, True, False, 8, 0.0),
    (16, 4096, True, True, True, False, 0, 1.0),
    (17, 512, False, True, True, True, 24, 30.0),
    (33, 520, False, False, False, False, 0, 2.0),
    (5, 2048, True, True, False, True, 0, 0.0),
    (70, 2056, False, True, True, True, 16, -3.0),
    (9, 4104, False, False, True, False, 0, 0.0),
    (300, 5376, True, False, True, False, 0, 0.0),
    (2, 8192, False, True, True, True, 0, 0.5),
    (7, 8200, False, True, True, True, 8, 0.0),
    (3, 16384, True, True, True, True, 0, 0.0),
    (4, 16376, False, False, True, True, 0, 100.0),
    (1031, 1792, False, True, True, True, 0, 0.0),
    (5000, 256, True, True, True, False, 0, 0.0),
    (4099, 24, False, False, True, True, 0, 0.0),
]


@pytest.mark.parametrize("T,K,rms,residual,weight,bias,extra,mean", CASES)
def test_layer_norm(T, K, rms, residual, weight, bias, extra, mean):
    torch = _torch()
    import precision_gemm_amd as P
    print("[case] layer_norm", T, K, rms, residual, weight, bias, extra, flush=True)
    rng = np.random.default_rng(T * 7 + K)
    x, _ = _bf(rng, (T, K), 1.5, mean, extra)
    res, _ = _bf(rng, (T, K), 2.0, 0.0, extra) if residual else (None, None)
    w = _f32(rng, K, 0.2, 1.0) if weight else None
    b = _f32(rng, K, 0.2) if bias else None
    keep = x.clone(), None if res is None else res.clone()
    y, h = P.layer_norm(x, w, b, residual=res, eps=1e-5, rms=rms)
    assert torch.equal(x, keep[0]) and (res is None or torch.equal(res, keep[1]))
    assert y.shape == h.shape == (T, K) and y.is_contiguous()
    if residual:
        assert torch.equal(h, (x.float() + res.float()).bfloat16())
    else:
        assert h is x or h.data_ptr() == x.data_ptr()
    hn, wn, bn = _f64(h), 1.0 if w is None else _f64(w), 0.0 if b is None else _f64(b)
    ref = S.layer_norm(hn, None if w is None else wn, None if b is None else bn, 1e-5, rms)
    r, xh, size = _sizes(hn, wn, 1e-5, rms)
    _within(_f64(y), ref, U * np.abs(ref) + 2.0 ** -18 * (size * np.abs(wn) + np.abs(ref) + np.abs(bn)) + 2.0 ** -133, "y")
    # in place: y in x's rows, h in the residual's
    if residual:
        y2, h2 = P.layer_norm(x, w, b, residual=res, eps=1e-5, rms=rms, out=x, sum_out=res)
        assert y2.data_ptr() == x.data_ptr() and torch.equal(x, y) and torch.equal(res, h)
    else:
        P.layer_norm(x, w, b, eps=1e-5, rms=rms, out=x)
        assert torch.equal(x, y)


@pytest.mark.parametrize("T,K,rms,residual,weight,bias,extra,mean", CASES)
def test_layer_norm_backward(T, K, rms, residual, weight, bias, extra, mean):
    torch = _torch()
    import precision_gemm_amd as P
    print("[case] layer_norm_backward", T, K, rms, residual, weight, bias, extra, flush=True)
    rng = np.random.default_rng(T * 11 + K)
    h, hn = _bf(rng, (T, K), 1.5, mean, extra)
    dy, dyn = _bf(rng, (T, K), 0.02, 0.001, extra)
    ds, dsn = _bf(rng, (T, K), 0.02, 0.0, extra) if residual else (None, 0.0)
    w = _f32(rng, K, 0.2, 1.0) if weight else None
    wn = np.ones(K) if w is None else _f64(w)
    dx, dw, db = P.layer_norm_backward(dy, h, w, dsum=ds, eps=1e-5, rms=rms, bias_grad=bias)
    assert dw.shape == (K,) and (db is None) == (not bias)
    ref, dwr, dbr = S.layer_norm_backward(dyn, hn, wn, 1e-5, rms, None if ds is None else dsn)
    r, xh, size = _sizes(hn, wn, 1e-5, rms)
    g = np.abs(dyn * wn)
    terms = r * (g + (0 if rms else g.mean(1, keepdims=True)) + (np.abs(xh) + size) * (g * (np.abs(xh) + 2.0 ** -2 * size)).mean(1, keepdims=True))
    _within(_f64(dx), ref, U * np.abs(ref) + 2.0 ** -16 * (terms + np.abs(dsn)) + 2.0 ** -133, "dx")
    _within(_f64(dw), dwr, 2.0 ** -16 * np.abs(dyn * xh).sum(0) + 2.0 ** -18 * (np.abs(dyn) * size).sum(0), "dweight")
    if bias:
        _within(_f64(db), dbr, 2.0 ** -16 * np.abs(dyn).sum(0), "dbias")
    # the same bits again, with buffers that are the caller's; frozen weights leave dx as it is
    ws = torch.full((P.layer_norm_backward_workspace_bytes(T, K),), 0xff, dtype=torch.uint8, device="cuda")
    got = P.layer_norm_backward(dy, h, w, dsum=ds, eps=1e-5, rms=rms, bias_grad=bias, dx=torch.empty_like(dx), dweight=torch.empty_like(dw),
                                dbias=torch.empty_like(db) if bias else None, workspace=ws)
    assert torch.equal(got[0], dx) and torch.equal(got[1], dw) and (not bias or torch.equal(got[2], db))
    only = P.layer_norm_backward(dy, h, w, dsum=ds, eps=1e-5, rms=rms, weight_grad=False, bias_grad=False)
    assert torch.equal(only[0], dx) and only[1] is None and only[2] is None
    if bias:
        alone = P.layer_norm_backward(dy, h, w, dsum=ds, eps=1e-5, rms=rms, weight_grad=False)
        assert torch.equal(alone[2], db) and alone[1] is None
    # dx in the rows of dsum, or of dy
    P.layer_norm_backward(dy, h, w, dsum=ds, eps=1e-5, rms=rms, bias_grad=bias, dx=ds if residual else dy)
    assert torch.equal(ds if residual else dy, dx)


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_rows_that_are_constant_or_not_numbers(rms, eps):
    """A row of equal values has no deviation: with eps it is all bias.  A row with a NaN or an infinity
    is no number, and no other row is touched by it; the weights' gradients are."""
    torch = _torch()
    import precision_gemm_amd as P
    print("[case] special rows", rms, eps, flush=True)
    rng = np.random.default_rng(5)
    x, xn = _bf(rng, (6, 1000), 1.0)
    x[1], x[2], x[3, 17], x[4, 999] = 0.0, 3.0, float("nan"), float("inf")
    w, b = _f32(rng, 1000, 0.2, 1.0), _f32(rng, 1000, 0.2)
    y, _ = P.layer_norm(x, w, b, eps=eps, rms=rms)
    good = _f64(y[[0, 5]])
    ref = S.layer_norm(xn[[0, 5]], _f64(w), _f64(b), eps, rms)
    _within(good, ref, U * np.abs(ref) + 2.0 ** -16, "the other rows")
    assert y[3].isnan().all() and y[4].isnan().any() and not y[0].isnan().any()
    if eps:
        assert torch.equal(y[1], b.bfloat16())
        assert rms or torch.equal(y[2], b.bfloat16())
    dy, dyn = _bf(rng, (6, 1000), 0.1)
    dx, dw, db = P.layer_norm_backward(dy, x, w, eps=eps, rms=rms)
    ref = S.layer_norm_backward(dyn[[0, 5]], xn[[0, 5]], _f64(w), eps, rms)[0]
    _within(_f64(dx[[0, 5]]), ref, U * np.abs(ref) + 2.0 ** -14, "the other rows' gradients")
    assert dw.isnan().any() and not db.isnan().any()


def test_eps_zero_with_rows_to_spare():
    """With eps = 0 a workgroup's rows behind the last one are no numbers: they reach nothing."""
    import precision_gemm_amd as P
    print("[case] eps 0", flush=True)
    rng = np.random.default_rng(6)
    for T, K in ((1, 64), (3, 512), (5, 1024), (1, 4096), (257, 2048)):
        h, hn = _bf(rng, (T, K))
        dy, dyn = _bf(rng, (T, K), 0.1)
        dx, dw, db = P.layer_norm_backward(dy, h, None, eps=0.0)
        ref, dwr, dbr = S.layer_norm_backward(dyn, hn, None, 0.0)
        _within(_f64(dx), ref, U * np.abs(ref) + 2.0 ** -14, "dx")
        _within(_f64(dw), dwr, 2.0 ** -14 * np.abs(dyn).sum(0), "dweight")
        _within(_f64(db), dbr, 2.0 ** -16 * np.abs(dyn).sum(0), "dbias")


def test_no_rows():
    torch = _torch()
    import precision_gemm_amd as P
    x = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
    y, h = P.layer_norm(x, None, None, residual=x)
    assert y.shape == h.shape == (0, 64)
    dw, db = torch.full((64,), 7.0, device="cuda"), torch.full((64,), 7.0, device="cuda")
    dx, _, _ = P.layer_norm_backward(x, x, None, dweight=dw, dbias=db)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


def test_refusals():
    torch = _torch()
    import precision_gemm_amd as P
    x = torch.zeros((3, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(64, device="cuda")
    with pytest.raises(ValueError, match="weight must have shape"):
        P.layer_norm(x, w[:32])
    with pytest.raises(ValueError, match="bias must have dtype"):
        P.layer_norm(x, w, w.bfloat16())
    with pytest.raises(ValueError, match="residual must be 3 rows of 64"):
        P.layer_norm(x, w, residual=x[:2])
    with pytest.raises(ValueError, match="sum_out is for a residual"):
        P.layer_norm(x, w, sum_out=x)
    with pytest.raises(ValueError, match="dense within each row"):
        P.layer_norm(x[:, ::2])
    with pytest.raises(RuntimeError, match="status 2"):
        P.layer_norm(x[:, :60].contiguous())
    with pytest.raises(RuntimeError, match="status 1"):  # rows that are not 16-byte aligned
        P.layer_norm(x[:, 4:52])
    with pytest.raises(ValueError, match="truth value"):
        P.layer_norm(x, rms=torch.ones(2))
    with pytest.raises(ValueError, match="eps"):
        P.layer_norm(x, eps="small")
    with pytest.raises(ValueError, match="h must be 3 rows of 64"):
        P.layer_norm_backward(x, x[:, :32])
    with pytest.raises(ValueError, match="are wanted"):
        P.layer_norm_backward(x, x, w, bias_grad=False, dbias=w)
    with pytest.raises(RuntimeError, match="status 3"):
        P.layer_norm_backward(x, x, w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


def test_graph_replays():
    """Forward and backward captured in a graph: every replay has the eager results of its inputs."""
    torch = _torch()
    import precision_gemm_amd as P
    print("[case] norm graph", flush=True)
    rng = np.random.default_rng(8)
    T, K = 130, 4096
    x, res, dy = (_bf(rng, (T, K))[0].contiguous() for _ in range(3))
    w, b = _f32(rng, K, 0.2, 1.0), _f32(rng, K, 0.2)
    bufs = dict(dx=torch.empty_like(x), dweight=torch.empty(K, device="cuda"), dbias=torch.empty(K, device="cuda"),
                workspace=torch.empty(P.layer_norm_backward_workspace_bytes(T, K), dtype=torch.uint8, device="cuda"))
    y, h = torch.empty_like(x), torch.empty_like(x)

    def step():
        P.layer_norm(x, w, b, residual=res, out=y, sum_out=h)
        P.layer_norm_backward(dy, h, w, dsum=y, **bufs)

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(4):
        for t in (x, res, dy):
            t.copy_(_bf(rng, (T, K))[0])
        g.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in (y, h, bufs["dx"], bufs["dweight"], bufs["dbias"])]
        yy, hh = P.layer_norm(x, w, b, residual=res)
        want = (yy, hh, *P.layer_norm_backward(dy, hh, w, dsum=yy))
        assert all(torch.equal(a, c) for a, c in zip(got, want)), i
