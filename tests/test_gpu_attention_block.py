"""The attention block as examples/attention_block.py chains it: QKV projection, cache, drafted
trees, output projection; and its backward.

Tolerances (relative Frobenius, u = 2^-8 half a step of bf16):
 * served against the oracle's whole block in fp64: five roundings on the way (QKV, rotated
   heads, probabilities, attention's output, y), each at most u: 5 u; an FP8 cache adds half a
   step of e4m3 (2^-4) for keys and for values;
 * trees against the same tokens in order: the two runs differ by the order of sums and the few
   roundings that it moves: 5 u; with an FP8 cache a moved code is a step of 2^-3: 2^-4;
 * gradients against autograd in fp32: eight roundings (the five before, dattn, dq/dk/dv, dqkv),
   doubled for what the softmax's gradient subtracts: 16 u = 2^-4.
"""

import importlib.util
import os

import numpy as np
import pytest

from oracle import attention as A

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
RANKS = [8, 16, 32]


@pytest.fixture(scope="module")
def ex():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_block.py")
    spec = importlib.util.spec_from_file_location("attention_block_example", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _off(got, ref):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    return np.linalg.norm(got - ref) / np.linalg.norm(ref)


def _oracle_block(block, x, tenant):
    """The block in fp64 on one sequence, in order; ``x`` bf16 [n, hidden]."""
    n = len(x)

    def project(p, rows):
        a, b = p.ad.A[tenant].double().cpu().numpy(), p.ad.B[tenant].double().cpu().numpy()
        return rows @ p.dense.double().cpu().numpy().T + rows @ a @ b

    D, n_q, n_kv = block.D, block.n_q, block.n_kv
    qkv = project(block.qkv, x.double().numpy()).reshape(n, -1, D)
    cs, pos = block.heads["cos_sin"].double().cpu().numpy(), np.arange(n)
    q = A.norm_rope(qkv[:, :n_q], pos, cs, block.q_weight.double().cpu().numpy(), 1e-6)
    k = A.norm_rope(qkv[:, n_q:n_q + n_kv], pos, cs, block.k_weight.double().cpu().numpy(), 1e-6)
    v = qkv[:, n_q + n_kv:]
    one = lambda m: m.transpose(1, 0, 2)[None]  # a cache of one page  # noqa: E731
    out = A.tree_attention(q, one(k), one(v), np.zeros((1, 1), int), [n], [0, n], None, D ** -0.5)[0]
    return project(block.o, out.reshape(n, -1))


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("n_q,n_kv,D", [(8, 2, 128), (12, 4, 64), (4, 2, 256)])
def test_served_trees(ex, kv, n_q, n_kv, D):
    import torch
    print("[case] serve", kv, n_q, n_kv, D, flush=True)
    block = ex.AttentionBlock(1024, n_q, n_kv, D, RANKS, max_pos=512, train=True)
    prompts, ids = [70, 1, 33, 128], [0, 1, 2, 1]
    xs, ys, status = ex.serve(block, prompts, ids, rounds=3, tree=16, kv=kv)
    assert status == 0
    assert all(len(x) == len(y) > p + 2 for x, y, p in zip(xs, ys, prompts))
    # the same tokens in order, in one call
    lens = [len(x) for x in xs]
    step = ex.Step(block, ex.Cache(block, len(xs), max(lens), page_size=32, kv=kv), sum(lens), max(lens), tree=False)
    step.load(torch.cat(xs), torch.tensor(ids, dtype=torch.int32).repeat_interleave(torch.tensor(lens)), [0] * len(xs), lens)
    again = step.run().cpu().split(lens)
    for b, (y, z) in enumerate(zip(ys, again)):
        off = _off(y.double(), z.double())
        assert off <= (5 * U if kv == "bf16" else 2.0 ** -4), (b, off)
    for b in (1, 2):
        off = _off(ys[b].double(), _oracle_block(block, xs[b], ids[b]))
        print(f"  sequence {b}: off by {off:.2e}", flush=True)
        assert off <= 5 * U + (2.0 ** -3 if kv == "fp8" else 0.0), (b, off)


def test_step_in_one_graph(ex):
    """A captured step replayed with eager work in between equals the eager step bit for bit."""
    import torch
    print("[case] serving step in a graph", flush=True)
    block = ex.AttentionBlock(1024, 8, 2, 128, RANKS, max_pos=512)
    gen = torch.Generator().manual_seed(5)
    cache = ex.Cache(block, 3, 200, kv="bf16")
    cache.k.copy_(torch.randn(cache.k.shape, generator=gen))
    cache.v.copy_(torch.randn(cache.v.shape, generator=gen))
    step = ex.Step(block, cache, 48, 16, tree=True)
    trees = [ex.draft(16, gen) for _ in range(3)]
    step.load(torch.randn(48, 1024, generator=gen).bfloat16(), torch.tensor([0, 1, 2], dtype=torch.int32).repeat_interleave(16),
              [150, 0, 40], [16] * 3, torch.tensor([p for t in trees for p in t[0]]),
              torch.tensor([d for t in trees for d in t[1]]))
    eager = step.run().clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.run()
    for _ in range(3):
        step.b_o["y"].zero_()
        step.ws.fill_(0x5A)
        (torch.ones(1 << 20, device="cuda") * 2).sum()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(step.b_o["y"].view(torch.int16), eager.view(torch.int16))
    assert int(step.status.item()) == 0


def test_training_step(ex):
    import torch
    print("[case] training step", flush=True)
    block = ex.AttentionBlock(1024, 8, 2, 128, RANKS, max_pos=512, train=True)
    lens = [60, 1, 35]
    x, target, ids = ex.training_batch(block, lens, len(RANKS))
    loss, grads, dx = ex.train_step(block, x, target, ids, lens)

    # the block in fp32 under autograd, from the same weights
    leaf = lambda m: m.detach().float().clone().requires_grad_()  # noqa: E731
    xr, qw, kw = leaf(x), leaf(block.q_weight), leaf(block.k_weight)
    ad = {n: [leaf(m) for m in getattr(p.ad, n[-1])] for n, p in
          (("qkv_A", block.qkv), ("qkv_B", block.qkv), ("o_A", block.o), ("o_B", block.o))}

    def project(p, name, rows):
        low = torch.zeros(len(rows), p.N, device="cuda")
        for a in range(len(RANKS)):
            here = (ids == a).float()[:, None]
            low = low + here * (rows @ ad[name + "_A"][a] @ ad[name + "_B"][a])
        return rows @ p.dense.T + low

    def heads(h, w):
        n = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + 1e-6) * w
        pos = torch.cat([torch.arange(m) for m in lens]).cuda()
        c, s = block.heads["cos_sin"][pos][:, None, :].chunk(2, -1)
        a, b = n.chunk(2, -1)
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    h = project(block.qkv, "qkv", xr).view(len(x), -1, 128)
    out = ex.causal_attention(heads(h[:, :8], qw), heads(h[:, 8:10], kw), h[:, 10:], lens)
    y = project(block.o, "o", out.flatten(1))
    ref = ((y - target) ** 2).mean()
    ref.backward()
    ref = float(ref.detach())
    assert abs(loss - ref) <= 2 * 5 * U * ref
    for name, got, want in [("dx", dx, xr.grad), ("q_weight", grads["q_weight"], qw.grad),
                            ("k_weight", grads["k_weight"], kw.grad)] + [
                                (f"{n}[{a}]", grads[n][a], ad[n][a].grad) for n in ad for a in range(len(RANKS))]:
        off = _off(got.double().cpu(), want.double().cpu())
        print(f"  {name}: off by {off:.2e}", flush=True)
        assert off <= 16 * U, (name, off)
    losses = ex.train(block, x, target, ids, lens, steps=3)
    assert losses[0] > losses[1] > losses[2]
