"""A decoder layer's attention block for many tenants, from the hidden states before the QKV
projection to those after the output projection, with random weights:

    x -> QKV projection with each token's adapter -> head norms and rotation, keys and values into a
    paged cache -> attention over the cache -> output projection with each token's adapter -> y

``serve`` fills the cache with prompts, then verifies drafted trees: every round is one replay of a
captured graph, after which one path of each tree is kept.  ``train`` runs the block's forward and
backward over whole sequences and moves the adapters and norm weights.

    python examples/attention_block.py [--kv bf16|fp8] [--rounds N]
"""

from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import precision_gemm_amd as P  # noqa: E402


class Projection:
    """A linear layer with FP8 base weight and one adapter a tenant."""

    def __init__(self, K, N, ranks, gen, train=False):
        w = torch.randn(N, K, generator=gen, device="cuda") / math.sqrt(K)
        scale = w.abs().amax(1) / 448.0
        rowmajor = P.LowpWeight("fp8", (w / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8), scale)
        self.K, self.N, self.w = K, N, P.pack_weight(rowmajor)
        self.dense = rowmajor.q.view(torch.float8_e4m3fn).float() * scale[:, None] if train else None
        self.wt = P.pack_weight_t(rowmajor) if train else None
        self.A = [torch.randn(K, r, generator=gen, device="cuda") / math.sqrt(K) for r in ranks]
        self.B = [0.05 * torch.randn(r, N, generator=gen, device="cuda") for r in ranks]
        self.pack()

    def pack(self):
        """The adapters in the forms the library reads, after they changed."""
        self.ad = P.Adapters([a.bfloat16() for a in self.A], [b.bfloat16() for b in self.B],
                             torch.ones(len(self.A), device="cuda"))
        self.bw = P.pack_adapters_bwd(self.ad) if self.wt is not None else None

    def buffers(self, T):
        return dict(ws=P.alloc_workspace(T, self.K, self.N, self.ad.n, self.ad.r_max),
                    t=torch.empty(T, self.ad.r_max, device="cuda"),
                    y=torch.empty(T, self.N, dtype=torch.bfloat16, device="cuda"))

    def forward(self, x, seg, buf, build_segments=False):
        return P.gemm_lowp_lora_epilogue(x, self.w, seg, self.ad, buf["ws"], t=buf["t"], y=buf["y"],
                                         build_segments=build_segments, act_bf16=True)

    def backward(self, x, dy, seg, buf):
        return P.lora_backward(x, dy, buf["t"], self.wt, self.w.scale, seg, self.ad, self.bw)


class AttentionBlock:
    """Weights of the block; ``hidden`` is the width of x and y."""

    def __init__(self, hidden, n_q, n_kv, head_dim, ranks, max_pos, seed=0, train=False):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.hidden, self.n_q, self.n_kv, self.D = hidden, n_q, n_kv, head_dim
        self.qkv = Projection(hidden, (n_q + 2 * n_kv) * head_dim, ranks, gen, train)
        self.o = Projection(n_q * head_dim, hidden, ranks, gen, train)
        self.q_weight = 1.0 + 0.1 * torch.randn(head_dim, generator=gen, device="cuda")
        self.k_weight = 1.0 + 0.1 * torch.randn(head_dim, generator=gen, device="cuda")
        self.heads = dict(cos_sin=P.rope_table(max_pos, head_dim), eps=1e-6)


class Step:
    """One shape of a serving step: ``max_q`` tokens at most a sequence, T in all.  Inputs and
    outputs keep their places, so that a captured step can be replayed."""

    def __init__(self, block, cache, T, max_q, tree):
        self.block, self.cache, self.max_q = block, cache, max_q
        dev = dict(device="cuda")
        i32 = dict(dtype=torch.int32, **dev)
        self.x = torch.zeros(T, block.hidden, dtype=torch.bfloat16, **dev)
        self.seg = P.empty_segments(torch.zeros(T, **i32), block.qkv.ad.n)
        self.positions, self.slots = torch.zeros(T, **i32), torch.full((T,), -1, **i32)
        self.parents = torch.full((T,), -1, **i32) if tree else None
        B = cache.page_table.shape[0]
        self.kv_len, self.q_indptr = torch.zeros(B, **i32), torch.zeros(B + 1, **i32)
        self.status = torch.zeros(1, **i32)
        self.b_qkv, self.b_o = block.qkv.buffers(T), block.o.buffers(T)
        self.q = torch.empty(T, block.n_q, block.D, dtype=torch.bfloat16, **dev)
        self.out, self.lse = torch.empty_like(self.q), torch.empty(T, block.n_q, **dev)
        self.ws = torch.empty(P.tree_attention_workspace_bytes(block.n_q, block.n_kv, block.D, max_q), dtype=torch.uint8,
                              **dev)

    def run(self):
        b, c = self.block, self.cache
        qkv = b.qkv.forward(self.x, self.seg, self.b_qkv, build_segments=True)
        P.rope_append_kv(qkv, self.positions, self.slots, c.k, c.v, b.n_q, q_weight=b.q_weight, k_weight=b.k_weight,
                         k_scale=c.k_scale, v_scale=c.v_scale, q_out=self.q, status=self.status, **b.heads)
        mask = None
        if self.parents is not None:
            mask = P.tree_mask(self.parents, self.q_indptr, self.max_q, status=self.status)
        P.tree_attention(self.q, c.k, c.v, c.page_table, self.kv_len, self.q_indptr, self.max_q, tree_mask=mask,
                         k_scale=c.k_scale, v_scale=c.v_scale, out=self.out, lse=self.lse, workspace=self.ws,
                         status=self.status)
        return b.o.forward(self.out.flatten(1), self.seg, self.b_o)

    def load(self, x, ids, lengths, drafted, parents=None, depth=None):
        """The step's inputs: sequence b has ``lengths[b]`` tokens in the cache and ``drafted[b]``
        new ones; ``depth`` is each new token's distance from the cache's end (None: in order)."""
        q0, seqs, offs = [0], [], []
        for b, n in enumerate(drafted):
            q0.append(q0[-1] + n)
            seqs += [b] * n
            offs += range(n)
        seqs, offs = torch.tensor(seqs), torch.tensor(offs)
        lengths, drafted = torch.tensor(lengths), torch.tensor(drafted)
        at = lengths[seqs] + offs
        self.x.copy_(x)
        self.seg.adapter_id.copy_(ids)
        self.positions.copy_(at if depth is None else lengths[seqs] + depth)
        self.slots.copy_(self.cache.slots(seqs, at))
        self.kv_len.copy_(lengths + drafted)
        self.q_indptr.copy_(torch.tensor(q0))
        if self.parents is not None:
            self.parents.copy_(parents)


class Cache:
    """A paged cache of ``B`` sequences up to ``longest`` tokens, pages handed out in random order."""

    def __init__(self, block, B, longest, page_size=16, kv="bf16"):
        per = -(-longest // page_size)
        self.page_size = page_size
        self.page_table = torch.randperm(B * per, generator=torch.Generator().manual_seed(1)).int().view(B, per).cuda()
        dtype = torch.float8_e4m3fn if kv == "fp8" else torch.bfloat16
        shape = (B * per, block.n_kv, page_size, block.D)
        self.k, self.v = (torch.zeros(shape, device="cuda").to(dtype) for _ in range(2))
        # normed keys stay below sqrt(D) times the largest weight; 448 is the largest e4m3 value
        self.k_scale = self.v_scale = None
        if kv == "fp8":
            self.k_scale = torch.full((block.n_kv,), math.sqrt(block.D) * float(block.k_weight.abs().max()) * 1.5 / 448.0,
                                      device="cuda")
            self.v_scale = torch.full((block.n_kv,), 8.0 / 448.0, device="cuda")

    def slots(self, seqs, at):
        pages = self.page_table.cpu()[seqs, at // self.page_size]
        return pages * self.page_size + at % self.page_size

    def keep(self, seqs, at, to):
        """Tokens ``at`` of sequences ``seqs`` moved to places ``to`` (a kept path of a tree)."""
        src, dst = self.slots(seqs, at).cuda().long(), self.slots(seqs, to).cuda().long()
        p = self.page_size
        for c in (self.k.view(torch.uint8), self.v.view(torch.uint8)):
            c[dst // p, :, dst % p] = c[src // p, :, src % p]


def draft(n, gen):
    """A random tree of n drafted tokens: parents (each before its children) and depths."""
    parents = [-1] + [int(torch.randint(max(0, j - 4), j, (1,), generator=gen)) for j in range(1, n)]
    depth = []
    for p in parents:
        depth.append(0 if p < 0 else depth[p] + 1)
    return parents, depth


def serve(block, prompts, ids, rounds=3, tree=16, kv="bf16", seed=2):
    """Prompts of the given lengths (tenant ``ids[b]`` each) into a cache, then ``rounds`` rounds of
    ``tree`` drafted tokens a sequence.  Returns (hidden states of every kept token, the block's
    outputs for them, status bits), the first two as a list over the sequences."""
    gen = torch.Generator().manual_seed(seed)
    B = len(prompts)
    ids = torch.tensor(ids, dtype=torch.int32)
    cache = Cache(block, B, max(prompts) + rounds * tree + tree, kv=kv)
    rows = lambda n: torch.randn(n, block.hidden, generator=gen).bfloat16()  # noqa: E731

    x = rows(sum(prompts))
    first = Step(block, cache, sum(prompts), max(prompts), tree=False)
    first.load(x, ids.repeat_interleave(torch.tensor(prompts)), [0] * B, prompts)
    y = first.run().cpu()
    xs, ys = list(x.split(prompts)), list(y.split(prompts))

    step = Step(block, cache, B * tree, tree, tree=True)
    graph, lengths = None, list(prompts)
    for _ in range(rounds):
        trees = [draft(tree, gen) for _ in range(B)]
        x = rows(B * tree)
        step.load(x, ids.repeat_interleave(tree), lengths, [tree] * B, torch.tensor([p for t in trees for p in t[0]]),
                  torch.tensor([d for t in trees for d in t[1]]))
        if graph is None:  # the first round runs as calls, and what they allocate once is there for the capture
            step.run()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step.run()
        graph.replay()
        y = step.b_o["y"].cpu()
        seqs, at, to = [], [], []
        for b, (parents, _) in enumerate(trees):  # the path to a random leaf is what the target accepted
            path, j = [], int(torch.randint(0, tree, (1,), generator=gen))
            while j >= 0:
                path.insert(0, j)
                j = parents[j]
            seqs += [b] * len(path)
            at += [lengths[b] + j for j in path]
            to += range(lengths[b], lengths[b] + len(path))
            pick = torch.tensor(path) + b * tree
            xs[b], ys[b] = torch.cat([xs[b], x[pick]]), torch.cat([ys[b], y[pick]])
            lengths[b] += len(path)
        cache.keep(*(torch.tensor(v) for v in (seqs, at, to)))
    return xs, ys, int(first.status.item()) | int(step.status.item())


def causal_attention(q, k, v, lens):
    """Attention of whole sequences in 32 bits (their lengths ``lens``), for autograd."""
    out, G = [], q.shape[1] // k.shape[1]
    for qs, ks, vs in zip(q.split(lens), k.split(lens), v.split(lens)):
        ks, vs = (m.repeat_interleave(G, 1).transpose(0, 1).contiguous() for m in (ks, vs))
        s = qs.transpose(0, 1).contiguous() @ ks.transpose(1, 2).contiguous() / math.sqrt(q.shape[2])
        n = len(qs)
        s = s.masked_fill(torch.ones(n, n, dtype=torch.bool, device=s.device).triu(1), -math.inf)
        out.append((s.softmax(-1) @ vs).transpose(0, 1))
    return torch.cat(out)


def train_step(block, x, target, ids, lens):
    """Loss and gradients of the block on a batch of whole sequences: mean squared error to
    ``target``.  Returns (loss, dict of gradients, dx)."""
    T, n_q, n_kv, D = len(x), block.n_q, block.n_kv, block.D
    positions = torch.cat([torch.arange(n) for n in lens]).int().cuda()
    seg = P.build_segments(ids, block.qkv.ad.n)
    b_qkv, b_o = block.qkv.buffers(T), block.o.buffers(T)
    weights = dict(q_weight=block.q_weight, k_weight=block.k_weight, **block.heads)

    qkv = block.qkv.forward(x, seg, b_qkv)
    q, k = P.qk_norm_rope(qkv, positions, n_q, n_kv, D, **weights)
    v = qkv[:, (n_q + n_kv) * D:].view(T, n_kv, D)
    leaves = [m.float().requires_grad_() for m in (q, k, v)]
    attn = causal_attention(*leaves, lens)
    a = attn.detach().bfloat16().flatten(1)
    y = block.o.forward(a, seg, b_o)
    diff = y.float() - target
    loss = float((diff * diff).mean())

    dy = (2.0 / diff.numel() * diff * LOSS_SCALE).bfloat16()
    da, _, g_o = block.o.backward(a, dy, seg, b_o)
    dq, dk, dv = (g.bfloat16() for g in torch.autograd.grad(attn, leaves, da.float().view_as(attn)))
    dqkv, dqw, dkw = P.qk_norm_rope_backward(qkv, positions, dq, dk, dv, **weights)
    dx, _, g_qkv = block.qkv.backward(x, dqkv, seg, b_qkv)
    inv = 1.0 / LOSS_SCALE
    grads = dict(qkv_A=[g * inv for g in g_qkv.dA], qkv_B=[g * inv for g in g_qkv.dB], o_A=[g * inv for g in g_o.dA],
                 o_B=[g * inv for g in g_o.dB], q_weight=dqw * inv, k_weight=dkw * inv)
    return loss, grads, dx.float() * inv


LOSS_SCALE = 4096.0


def train(block, x, target, ids, lens, steps=3, rate=1.0):
    """``steps`` steps of gradient descent on the adapters and the norm weights; the losses."""
    losses = []
    for _ in range(steps):
        loss, g, _ = train_step(block, x, target, ids, lens)
        losses.append(loss)
        for p, name in ((block.qkv, "qkv"), (block.o, "o")):
            for w, d in zip(p.A + p.B, g[name + "_A"] + g[name + "_B"]):
                w -= rate * d
            p.pack()
        block.q_weight -= rate * g["q_weight"]
        block.k_weight -= rate * g["k_weight"]
    return losses


def training_batch(block, lens, tenants, seed=3):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T = sum(lens)
    x = torch.randn(T, block.hidden, generator=gen, device="cuda").bfloat16()
    target = torch.randn(T, block.hidden, generator=gen, device="cuda")
    ids = torch.tensor([b % tenants for b, n in enumerate(lens) for _ in range(n)], dtype=torch.int32, device="cuda")
    return x, target, ids


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--kv", choices=["bf16", "fp8"], default="bf16")
    ap.add_argument("--rounds", type=int, default=3)
    a = ap.parse_args()
    ranks = [8, 16, 32, 64]
    block = AttentionBlock(4096, 32, 8, 128, ranks, max_pos=2048)
    prompts = [400, 17, 130, 256, 64, 1, 333, 90]
    xs, ys, status = serve(block, prompts, [b % 4 for b in range(len(prompts))], a.rounds, kv=a.kv)
    print(f"served {len(prompts)} conversations of {[len(x) for x in xs]} tokens, {a.rounds} rounds of 16 drafted tokens, "
          f"status {status}, mean |y| {torch.cat(ys).float().abs().mean():.3f}", flush=True)
    block = AttentionBlock(1024, 8, 2, 128, ranks, max_pos=2048, train=True)
    lens = [100, 37, 1, 62]
    print("training losses", [f"{v:.5f}" for v in train(block, *training_batch(block, lens, 4), lens)], flush=True)


if __name__ == "__main__":
    main()
