"""A training step around the layer, as it is used: the residual's addition and the norm, the QKV layer
with each token's adapter, head norms and rotation by positions of three axes, and back through all of
them to the adapters' next step, whose packed forms the next forward reads.

Against the same chain in 64 bits on the CPU under autograd (the adapters' and the frozen weight's own
8- and 16-bit values, the GPU's bf16 intermediates free to differ): gradients within 2 % relative
Frobenius.  Every bf16 intermediate (h, y, qkv, the heads, dqkv, the layer's dY times its channel scale,
dx) carries relative errors of at most 2^-8 = 0.4 % a value, six in a row, uncorrelated for the most part:
2.4 % if they all pointed the same way, about 1 % as they come.
"""

import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

T, HIDDEN, N_Q, N_KV, D, RANKS = 200, 512, 4, 2, 64, (5, 16, 64)
N = (N_Q + 2 * N_KV) * D


class Model:
    def __init__(self, seed=0):
        import torch
        import precision_gemm_amd as P
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        w = rand(N, HIDDEN) / math.sqrt(HIDDEN)
        scale = w.abs().amax(1) / 448.0
        row = P.LowpWeight("fp8", (w / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8), scale)
        self.dense = row.q.view(torch.float8_e4m3fn).double() * scale.double()[:, None]
        self.w, self.wt = P.pack_weight(row), P.pack_weight_t(row)
        self.ad = P.Adapters([(rand(HIDDEN, r) / math.sqrt(HIDDEN)).bfloat16() for r in RANKS],
                             [(0.05 * rand(r, N)).bfloat16() for r in RANKS], torch.tensor([1.0, 0.5, 2.0], device="cuda"))
        self.bw = P.pack_adapters_bwd(self.ad)
        self.grads = P.alloc_grads(self.ad, HIDDEN, N)
        self.norm_w, self.norm_b = 1 + 0.1 * rand(HIDDEN), 0.1 * rand(HIDDEN)
        self.q_w, self.k_w = 1 + 0.1 * rand(D), 0.1 * rand(D) + 1
        self.dnorm_w, self.dnorm_b = torch.zeros_like(self.norm_w), torch.zeros_like(self.norm_b)
        self.heads = dict(cos_sin=P.rope_table(64, D), q_weight=self.q_w, k_weight=self.k_w, pair_axes=P.rope_pair_axes((8, 12, 12)))
        self.x, self.res = rand(T, HIDDEN).bfloat16(), rand(T, HIDDEN).bfloat16()
        self.pos = torch.randint(0, 64, (3, T), generator=g, device="cuda", dtype=torch.int32)
        # tenant 1 has no tokens in this batch
        self.ids = (torch.arange(T, device="cuda") * 7 % 5 < 2).int() * 2
        self.out_grad = [rand(T, n, D).bfloat16() for n in (N_Q, N_KV, N_KV)]
        self.dsum = rand(T, HIDDEN).bfloat16()
        self.seg = P.empty_segments(self.ids, 3)
        self.ws = P.alloc_workspace(T, HIDDEN, N, 3, 64)
        self.t = torch.zeros((T, 64), device="cuda")
        self.bws = torch.empty(max(16, P.ops.backward_workspace_bytes(T, HIDDEN, N, 3, 64)), dtype=torch.uint8, device="cuda")
        self.nws = torch.empty(P.layer_norm_backward_workspace_bytes(T, HIDDEN), dtype=torch.uint8, device="cuda")
        self.hws = torch.empty(P.qk_norm_rope_backward_workspace_bytes(T, D), dtype=torch.uint8, device="cuda")
        self.active = torch.zeros(3, dtype=torch.int32, device="cuda")

    def optimizer(self, bits):
        import precision_gemm_amd as P
        ts = P.adamw_adapters(self.ad, self.grads, self.bw)
        # the norm's weights go with tenant 2
        ts += [P.AdamWTensor(self.norm_w, self.dnorm_w, 2), P.AdamWTensor(self.norm_b, self.dnorm_b, 2)]
        return P.AdamW(ts, 3, state_bits=bits)

    def forward(self):
        import precision_gemm_amd as P
        P.build_segments(self.ids, 3, self.seg)
        y, h = P.layer_norm(self.x, self.norm_w, self.norm_b, residual=self.res, eps=1e-5)
        qkv = P.gemm_lowp_lora_epilogue(y, self.w, self.seg, self.ad, self.ws, t=self.t, act_bf16=True)
        q, k = P.qk_norm_rope(qkv, self.pos, N_Q, N_KV, D, **self.heads)
        return y, h, qkv, q, k

    def backward(self, y, h, qkv):
        import precision_gemm_amd as P
        dq, dk, dv = self.out_grad
        dqkv, _, _ = P.qk_norm_rope_backward(qkv, self.pos, dq, dk, dv, workspace=self.hws, **self.heads)
        dy, _, _ = P.lora_backward(y, dqkv, self.t, self.wt, self.w.scale, self.seg, self.ad, self.bw, grads=self.grads,
                                   workspace=self.bws)
        dx, _, _ = P.layer_norm_backward(dy, h, self.norm_w, dsum=self.dsum, eps=1e-5, dweight=self.dnorm_w, dbias=self.dnorm_b,
                                         workspace=self.nws)
        self.active.copy_(self.seg.seg_indptr[1:] > self.seg.seg_indptr[:-1])
        return dx


def reference(m):
    """Gradients of the chain in 64 bits: (dx, dA, dB, dnorm_w, dnorm_b)."""
    import torch
    c = lambda t: t.detach().double().cpu()  # noqa: E731
    x, res, w = c(m.x), c(m.res), c(m.dense)
    leaf = lambda t: c(t).requires_grad_()  # noqa: E731
    A, B, nw, nb = [leaf(a) for a in m.ad.A], [leaf(b) for b in m.ad.B], leaf(m.norm_w), leaf(m.norm_b)
    h = (x + res).requires_grad_()
    d = h - h.mean(1, keepdim=True)
    y = d / torch.sqrt((d * d).mean(1, keepdim=True) + 1e-5) * nw + nb
    ids, sc = m.ids.cpu(), m.ad.scales.double().cpu()
    low = torch.zeros(T, N, dtype=torch.float64)
    for a in range(3):
        rows = ids == a
        low = low + rows[:, None] * (sc[a] * (y @ A[a]) @ B[a])
    qkv = (y @ w.T + low).view(T, -1, D)
    axes, cs, pos = list(m.heads["pair_axes"]), c(m.heads["cos_sin"]), m.pos.cpu().long()
    pair = torch.arange(D // 2)
    cos, sin = cs[pos[axes].T, pair][:, None], cs[pos[axes].T, D // 2 + pair][:, None]

    def head(v, weight):
        v = v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6) * c(weight)
        a, b = v[..., :D // 2], v[..., D // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    q, k = head(qkv[:, :N_Q], m.q_w), head(qkv[:, N_Q:N_Q + N_KV], m.k_w)
    gq, gk, gv = (c(g) for g in m.out_grad)
    loss = (q * gq).sum() + (k * gk).sum() + (qkv[:, N_Q + N_KV:] * gv).sum() + (h * c(m.dsum)).sum()
    loss.backward()
    return h.grad, [a.grad for a in A], [b.grad for b in B], nw.grad, nb.grad


def _near(got, ref, what, most=0.02):
    off = float((got.double().cpu() - ref).norm() / ref.norm())
    assert off <= most, f"{what}: {off:.4f} off"


def test_gradients_of_the_chain():
    print("[case] chain gradients", flush=True)
    m = Model()
    y, h, qkv, _, _ = m.forward()
    dx = m.backward(y, h, qkv)
    rdx, rA, rB, rnw, rnb = reference(m)
    _near(dx, rdx, "dx")
    _near(m.dnorm_w, rnw, "dweight")
    _near(m.dnorm_b, rnb, "dbias")
    for a in (0, 2):
        _near(m.grads.dA[a], rA[a], f"dA {a}")
        _near(m.grads.dB[a], rB[a], f"dB {a}")
    assert not m.grads.dA[1].any() and not m.grads.dB[1].any()
    assert m.active.tolist() == [1, 0, 1]


@pytest.mark.parametrize("bits", [32, 8])
def test_steps_of_the_chain(bits):
    """Three whole steps, eager and as replays of one captured graph: the same bits; the idle tenant is
    as it was; the forward after the steps reads what fresh packs of the stepped adapters would give."""
    import torch
    import precision_gemm_amd as P
    print("[case] chain steps", bits, flush=True)
    hyper = torch.tensor([[1e-3, 0.9, 0.99, 1e-8, 0.01, 1.0]] * 3, dtype=torch.float64, device="cuda")

    def run(captured):
        m = Model()
        opt = m.optimizer(bits)
        norm = torch.zeros(3, device="cuda")
        keep = [a.clone() for a in (m.ad.A[1], m.ad.B[1], m.ad.At[1], m.ad.Bt[1])]

        def step():
            y, h, qkv, _, _ = m.forward()
            dx = m.backward(y, h, qkv)
            P.adamw_step(opt, hyper, active=m.active, clip=True, grad_norm=norm)
            return dx

        if captured:
            state = [t.clone() for s in opt.tensors for t in (s.param, s.m, s.v, s.m_scale, s.v_scale, s.copy, s.pack, s.pack_bwd)
                     if t is not None]
            bufs = [t for s in opt.tensors for t in (s.param, s.m, s.v, s.m_scale, s.v_scale, s.copy, s.pack, s.pack_bwd) if t is not None]
            step()  # what it allocates once is there for the capture
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                dx = step()
            for b, s in zip(bufs, state):
                b.view(torch.uint8).copy_(s.view(torch.uint8))
            opt.steps.zero_()
        out = []
        for _ in range(3):
            if captured:
                graph.replay()
                torch.cuda.synchronize()
            else:
                dx = step()
            out.append((dx.clone(), norm.clone()))
        assert opt.steps.tolist() == [3, 0, 3]
        assert all(torch.equal(a, b) for a, b in zip(keep, (m.ad.A[1], m.ad.B[1], m.ad.At[1], m.ad.Bt[1])))
        fresh = P.Adapters([a.clone() for a in m.ad.A], [b.clone() for b in m.ad.B], m.ad.scales)
        y, _, qkv, _, _ = m.forward()
        again = P.gemm_lowp_lora_epilogue(y, m.w, m.seg, fresh, m.ws, act_bf16=True)
        assert torch.equal(qkv, again)
        return out, [s.param.clone() for s in opt.tensors], qkv

    a, b = run(False), run(True)
    for (dx, n), (dx2, n2) in zip(a[0], b[0]):
        assert torch.equal(dx, dx2) and torch.equal(n, n2) and float(n[1]) == 0 and float(n[0]) > 0
    assert all(torch.equal(p, q) for p, q in zip(a[1], b[1])) and torch.equal(a[2], b[2])
    assert not np.isnan(a[2].float().cpu().numpy()).any()
