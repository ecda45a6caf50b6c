"""Norms, AdamW step and rotation by several axes at their edges: offsets that pass 32 bits, other streams
than the default one, groups without tensors, many groups, buffers that may not be shared."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

F = np.float32


def test_norm_rows_past_32_bits():
    """Rows more than 2^31 values apart from the first: the last rows' results are those of a dense batch."""
    import torch
    import precision_gemm_amd as P
    T, K, ld = 65536, 1024, 40000
    print("[case] norm past 32 bits", flush=True)
    x = torch.empty((T, ld), dtype=torch.bfloat16, device="cuda")[:, :K]
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(0))
    assert T * ld > 2 ** 31
    w = torch.linspace(0.5, 1.5, K, device="cuda")
    dense = x[-300:].contiguous()
    want, _ = P.layer_norm(dense, w)
    y, h = P.layer_norm(x, w, residual=x, out=None)
    assert torch.equal(h[-300:], (2 * dense.float()).bfloat16())
    y, _ = P.layer_norm(x, w)
    assert torch.equal(y[-300:], want)
    dx, dw, _ = P.layer_norm_backward(x, x, w, dsum=x)
    want, _, _ = P.layer_norm_backward(dense, dense, w, dsum=dense)
    assert torch.equal(dx[-300:], want)
    # the same rows again, each counted once: their gradient is the dense batch's by the chunks
    parts = sum(P.layer_norm_backward(c.contiguous(), c.contiguous(), w)[1].double() for c in x.split(8192))
    assert torch.allclose(dw.double(), parts, rtol=1e-4, atol=1e-2)
    P.layer_norm(x, w, out=x)
    assert torch.equal(x[-300:], y[-300:])


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_of_a_billion_values(bits):
    """A vector whose buffers pass 4 GB: its last values step as a short vector of the same values does."""
    import torch
    import precision_gemm_amd as P
    n = 2 ** 30 + 77
    at = n - 5000 - (n - 5000) % 64  # a block's first value
    m = n - at
    print("[case] adamw past 32 bits", bits, flush=True)
    g = torch.Generator(device="cuda").manual_seed(1)
    tail, tg = torch.randn(m, generator=g, device="cuda"), torch.randn(m, generator=g, device="cuda")
    p, d = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    p[at:], d[at:] = tail, tg
    p[:64], d[:64] = 1.0, 0.5
    big = P.AdamWTensor(p, d, copy=torch.zeros(n, dtype=torch.bfloat16, device="cuda"))
    small = P.AdamWTensor(tail.clone(), tg.clone())
    h = torch.tensor([[0.01, 0.9, 0.99, 1e-8, 0.1, 1.0]], dtype=torch.float64, device="cuda")
    a, b = P.AdamW([big], 1, state_bits=bits), P.AdamW([small], 1, state_bits=bits)
    for _ in range(2):
        P.adamw_step(a, h)
        P.adamw_step(b, h)
    assert torch.equal(p[at:], small.param) and torch.equal(big.copy[at:], small.param.bfloat16())
    assert torch.equal(big.m[at:].view(torch.uint8), small.m.view(torch.uint8))
    assert torch.equal(big.v[at:].view(torch.uint8), small.v.view(torch.uint8))
    assert not p[64:at].any() and not big.copy[64:at].any() and (p[:64] < 1).all()
    norm = P.adamw_step(a, h, clip=True)
    want = (tg.double().square().sum() + 64 * 0.25).sqrt()
    assert abs(float(norm) - float(want)) <= 2.0 ** -23 * float(want)


def _small(n_groups, groups, bits=32):
    import torch
    import precision_gemm_amd as P
    g = torch.Generator(device="cuda").manual_seed(2)
    ts = [P.AdamWTensor(torch.randn(64, 8, generator=g, device="cuda"), torch.randn(64, 8, generator=g, device="cuda"), k, "A",
                        pack=torch.zeros(16 * 64, dtype=torch.bfloat16, device="cuda")) for k in groups]
    h = torch.tensor([[0.01, 0.9, 0.99, 1e-8, 0.1, 1.0]] * n_groups, dtype=torch.float64, device="cuda")
    return P.AdamW(ts, n_groups, state_bits=bits), h


@pytest.mark.parametrize("clip", [False, True])
@pytest.mark.parametrize("n_tiles", [2, 1500])
def test_groups_without_tensors(clip, n_tiles):
    """They make no steps and have no norm, in one launch and in several."""
    import torch
    import precision_gemm_amd as P
    print("[case] empty groups", clip, n_tiles, flush=True)
    opt, h = _small(9, [2, 7] * (n_tiles // 2))
    norm = P.adamw_step(opt, h, clip=clip)
    assert opt.steps.tolist() == [0, 0, 1, 0, 0, 0, 0, 1, 0]
    if clip:
        assert [bool(v) for v in norm.tolist()] == [False, False, True, False, False, False, False, True, False]
    # all idle: nothing moves
    before = [t.param.clone() for t in opt.tensors[:4]]
    norm = P.adamw_step(opt, h, active=torch.zeros(9, dtype=torch.int32, device="cuda"), clip=clip)
    assert opt.steps.tolist() == [0, 0, 1, 0, 0, 0, 0, 1, 0] and (norm is None or not norm.any())
    assert all(torch.equal(t.param, p) for t, p in zip(opt.tensors, before))


@pytest.mark.parametrize("clip", [False, True])
def test_most_groups(clip):
    """8,192 tenants, every second one with a tensor."""
    import torch
    import precision_gemm_amd as P
    print("[case] most groups", clip, flush=True)
    opt, h = _small(8192, range(1, 8192, 2))
    one, h1 = _small(8192, [1])
    P.adamw_step(opt, h, clip=clip)
    P.adamw_step(one, h, clip=clip)
    assert torch.equal(opt.steps, (torch.arange(8192, device="cuda") % 2).int())
    assert torch.equal(opt.tensors[0].param, one.tensors[0].param)


def test_one_launch_and_several_are_the_same():
    """A step of few tiles takes its coefficients in the workgroups, one of many in a launch of its own."""
    import torch
    import precision_gemm_amd as P
    print("[case] one launch and several", flush=True)
    for bits in (32, 8):
        few, h = _small(3, [0, 2], bits)
        many, _ = _small(3, [0, 2] + [1] * 1100, bits)
        for _ in range(5):
            P.adamw_step(few, h)
            P.adamw_step(many, h)
        for a, b in zip(few.tensors, many.tensors):
            for f in ("param", "m", "v", "pack"):
                assert torch.equal(getattr(a, f).view(torch.uint8), getattr(b, f).view(torch.uint8)), (bits, f)
        assert few.steps.tolist() == [5, 0, 5] and many.steps.tolist() == [5, 5, 5]


def test_another_stream():
    """Calls go to the current stream: work queued before them there is seen by them."""
    import torch
    import precision_gemm_amd as P
    print("[case] stream", flush=True)
    x = torch.zeros((2048, 4096), dtype=torch.bfloat16, device="cuda")
    src = torch.randn((2048, 4096), device="cuda").bfloat16()
    opt, h = _small(2, [0, 1])
    ref, _ = _small(2, [0, 1])
    for t in ref.tensors:
        t.grad.mul_(3.0)
    P.adamw_step(ref, h)
    want, _ = P.layer_norm(src)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        x.copy_(src)
        for t in opt.tensors:
            t.grad.mul_(3.0)
        y, _ = P.layer_norm(x)
        dx, dw, db = P.layer_norm_backward(y, x)
        P.adamw_step(opt, h)
    s.synchronize()
    assert torch.equal(y, want) and all(torch.equal(a.param, b.param) for a, b in zip(opt.tensors, ref.tensors))
    again = P.layer_norm_backward(want, src)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1]) and torch.equal(db, again[2])


def test_rows_that_may_not_be_shared():
    import torch
    import precision_gemm_amd as P
    x = torch.zeros((3, 64), dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(x)
    with pytest.raises(RuntimeError, match="status 1"):
        P.layer_norm(x, residual=x, out=out, sum_out=out)
    with pytest.raises(RuntimeError, match="status 1"):  # one row for all tokens
        P.layer_norm(x, residual=x[:1].expand(3, 64))


def test_axes_with_most_tokens():
    """65,536 tokens: positions of the last axis lie past those of the others."""
    import torch
    import precision_gemm_amd as P
    print("[case] axes most tokens", flush=True)
    T = 65536
    g = torch.Generator(device="cuda").manual_seed(3)
    qkv = torch.randn((T, 3 * 64), generator=g, device="cuda").bfloat16()
    pos = torch.randint(0, 500, (4, T), generator=g, device="cuda", dtype=torch.int32)
    args = dict(cos_sin=P.rope_table(500, 64), pair_axes=P.rope_pair_axes((8, 8, 8, 8)))
    q, k = P.qk_norm_rope(qkv, pos, 1, 1, 64, **args)
    a, b = P.qk_norm_rope(qkv[-100:].contiguous(), pos[:, -100:].contiguous(), 1, 1, 64, **args)
    assert torch.equal(q[-100:], a) and torch.equal(k[-100:], b)


@pytest.mark.parametrize("T,K,rms,extra", [(5, 64, False, 0), (16, 4096, True, 8), (1, 520, False, 0)])
def test_norm_over_its_input_has_no_h(T, K, rms, extra):
    """Without a residual h is x itself: where y takes x's place there is none, and the backward, which needs
    it, refuses what is returned in its place."""
    import torch
    import precision_gemm_amd as P
    print("[case] norm in place", T, K, rms, flush=True)
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((T, K + extra), generator=g, device="cuda").bfloat16()[:, :K]
    other = torch.empty((T, K), dtype=torch.bfloat16, device="cuda")
    want, h = P.layer_norm(x, rms=rms)
    assert h is x
    y, h = P.layer_norm(x, rms=rms, out=other)
    assert h is x and y is other and torch.equal(y, want)
    # the other half of one buffer's rows is another place
    both = torch.cat([x, x], 1)
    y, h = P.layer_norm(both[:, :K], rms=rms, out=both[:, K:])
    assert torch.equal(h, x) and torch.equal(both[:, K:], want) and torch.equal(both[:, :K], x)
    y, h = P.layer_norm(x, rms=rms, out=x)
    assert h is None and y.data_ptr() == x.data_ptr() and torch.equal(x, want)
    with pytest.raises(ValueError, match="h must be a tensor"):
        P.layer_norm_backward(y, h, rms=rms)
    # with a residual h is the sum, in a place of its own
    r = torch.randn((T, K), generator=g, device="cuda").bfloat16()
    s = (x.float() + r.float()).bfloat16()
    y, h = P.layer_norm(x, residual=r, rms=rms, out=x)
    assert torch.equal(h, s) and torch.equal(x, P.layer_norm(s, rms=rms)[0])


def test_norm_over_its_input_without_rows():
    import torch
    import precision_gemm_amd as P
    x = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
    y, h = P.layer_norm(x, out=x)
    assert y.shape == (0, 64) and (h is None or h.shape == (0, 64))
