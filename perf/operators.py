"""The attention block between a decoder layer's QKV and output projections, as cases to measure.

Three operators: the norm and position rotation of each query and key head (forward and
backward), the same on the way into a paged cache of keys and values, and attention for a
tree of drafted tokens over that cache.  ``run`` computes a case in its plain form (torch
operations in 32 bits), or with ``own`` set calls this library's kernels; ``exact`` is the
same from the definitions in 64 bits.
"""

import math
import random

import numpy as np
import torch

own = False

EPS = 1e-6
THETA = 10000.0
SCRATCH_BYTES = 96 << 20   # the attention's workspace, kept by the caller from call to call

_BYTES = {False: 2, True: 1}   # of a cached value: bf16, e4m3


def listed():
    """The cases.  32 query heads, 8 key and value heads of 128 are the 6,144 columns of the
    repository's QKV projection; 16 and 4,096 tokens its decode and prefill batches."""
    h = dict(n_q=32, n_kv=8, D=128)
    rot = dict(rot=128, interleaved=False)
    return [
        # a decode batch of 16 sequences, one token each: the launch is what counts
        dict(name="norm_rope_decode", op="norm_rope", T=16, **h, **rot, norm=True, backward=False),
        # a prompt, or a training micro-batch, of 4,096 tokens
        dict(name="norm_rope_prefill", op="norm_rope", T=4096, **h, **rot, norm=True, backward=False),
        # its backward, into the gradient that the QKV projection's backward reads
        dict(name="norm_rope_backward", op="norm_rope", T=4096, **h, **rot, norm=True, backward=True),
        # the backward of an odd batch: small heads, half of each rotated, in interleaved pairs
        dict(name="norm_rope_backward_odd", op="norm_rope", T=1001, n_q=28, n_kv=4, D=64, rot=32, interleaved=True,
             norm=True, backward=True),
        # a decode batch appends one token a sequence to a 16-bit cache
        dict(name="append_decode", op="append", T=16, **h, **rot, norm=False, page=16, fp8=False),
        # a prompt of 4,096 tokens goes into an 8-bit cache, with the heads' norms on the way
        dict(name="append_prefill_fp8", op="append", T=4096, **h, **rot, norm=True, page=64, fp8=True),
        # decode of 16 short conversations
        dict(name="attend_decode", op="attend", B=16, n=1, kv=1024, ragged=False, **h, page=16, fp8=False, tree=False),
        # decode of 64 conversations of very different lengths
        dict(name="attend_decode_ragged", op="attend", B=64, n=1, kv=8192, ragged=True, **h, page=16, fp8=False,
             tree=False),
        # decode of one conversation with a long context, 8-bit cache
        dict(name="attend_long_fp8", op="attend", B=1, n=1, kv=131072, ragged=False, **h, page=64, fp8=True, tree=False),
        # trees of up to 16 drafted tokens for 8 conversations
        dict(name="attend_tree16", op="attend", B=8, n=16, kv=4096, ragged=True, **h, page=16, fp8=False, tree=True),
        # trees of up to 64 drafted tokens for 16 conversations, 8-bit cache: matrix work counts
        dict(name="attend_tree64_fp8", op="attend", B=16, n=64, kv=2048, ragged=True, **h, page=64, fp8=True, tree=True),
        # chains of up to 7 tokens, an odd group of heads, small heads
        dict(name="attend_chain7_odd", op="attend", B=5, n=7, kv=1999, ragged=True, n_q=28, n_kv=4, D=64, page=32,
             fp8=False, tree=False),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm, odd ones among them."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, v))


_LARGEST = dict(bytes=9.2e8, flops=9.3e9)   # of the listed cases with most of each, about


def draw(rng):
    """One more case of these ranges: 1 to 8,192 tokens, 1 to 64 sequences of up to 131,072
    cached tokens, trees of up to 64, groups of 1 to 8 query heads, heads of 64, 128 or 256."""
    while True:
        D = rng.choice((64, 128, 128, 256))
        n_q, n_kv = rng.choice(((32, 8), (8, 1), (28, 4), (16, 8), (40, 8), (6, 6), (15, 3), (4, 2)))
        c = dict(op=rng.choice(("norm_rope", "append", "attend", "attend")))
        if c["op"] == "attend":
            c.update(B=_log(rng, 1, 64), n=rng.choice((1, 1, _log(rng, 2, 64))), kv=_log(rng, 70, 131072),
                     ragged=rng.random() < 0.5, n_q=n_q, n_kv=n_kv, D=D, page=rng.choice((16, 32, 64, 128)),
                     fp8=rng.random() < 0.5, tree=rng.random() < 0.5)
            # the plain form's 32-bit copies: all sequences at the longest one's length, and their scores
            if c["B"] * c["kv"] * (2 * n_kv * D + 2 * c["n"] * n_q) > 1.4e9:
                continue
        else:
            c.update(T=_log(rng, 1, 8192), n_q=n_q, n_kv=n_kv, D=D, rot=rng.choice((D, D, D // 2)),
                     interleaved=rng.random() < 0.3, norm=rng.random() < 0.7)
            if c["op"] == "append":
                c.update(page=rng.choice((16, 32, 64, 128)), fp8=rng.random() < 0.5)
            else:
                c.update(backward=rng.random() < 0.5)
        sizes = [v for v in c.values() if isinstance(v, int)] + [n_q * D, n_kv * D, (n_q + 2 * n_kv) * D]
        if 3072 not in sizes and all(work(c)[k] <= v for k, v in _LARGEST.items()):
            return c


# ---- what a case's sizes are (from the case alone, so that `work` can count them) ----

def _lengths(c):
    """(cached tokens, drafted tokens among them) of each sequence of an attention case."""
    rng = random.Random("%d/%d/%d" % (c["B"], c["n"], c["kv"]))
    out = []
    for _ in range(c["B"]):
        if c["ragged"]:
            n = rng.randint(max(1, c["n"] // 2), c["n"])
            out.append((max(n, int(c["kv"] * math.exp(rng.uniform(math.log(0.125), 0.0)))), n))
        else:
            out.append((c["kv"], c["n"]))
    return out


def _parents(c):
    """The parent of each drafted token within its sequence's tree (-1: the cached prefix)."""
    rng = random.Random("tree %d/%d/%d" % (c["B"], c["n"], c["kv"]))
    return [[-1 if j == 0 else (rng.randint(max(0, j - 6), j - 1) if c["tree"] else j - 1) for j in range(n)]
            for _, n in _lengths(c)]


def _ancestors(parents):
    """The bits of each token's mask: itself and its ancestors."""
    rows = []
    for j, p in enumerate(parents):
        rows.append((rows[p] if p >= 0 else 0) | 1 << j)
    return rows


def work(c):
    D, n_q, n_kv = c["D"], c["n_q"], c["n_kv"]
    if c["op"] == "attend":
        lens, pairs = _lengths(c), 0
        for (kv, n), par in zip(lens, _parents(c)):
            pairs += n * (kv - n) + sum(bin(m).count("1") for m in _ancestors(par))
        T, tokens = sum(n for _, n in lens), sum(kv for kv, _ in lens)
        pages = sum(-(-kv // c["page"]) for kv, _ in lens)
        return {"bytes": 2.0 * tokens * n_kv * D * _BYTES[c["fp8"]] + 2.0 * 2 * T * n_q * D + 4 * T * n_q + 4 * pages
                + 8 * T * (1 if c["tree"] else 0), "flops": 4.0 * pairs * n_q * D}
    T, H = c["T"], n_q + n_kv
    table = 4.0 * T * c["rot"]
    per = (8 if c["norm"] else 0) + 3
    if c["op"] == "append":
        return {"bytes": 2.0 * T * (H + n_kv) * D + 2.0 * T * n_q * D + 2.0 * T * n_kv * D * _BYTES[c["fp8"]] + table + 8 * T,
                "flops": float(per * T * H * D)}
    if c["backward"]:
        return {"bytes": 2.0 * T * H * D * 2 + 2.0 * T * n_kv * D * 2 + 2.0 * T * H * D + table + 4 * T,
                "flops": float(2 * per * T * H * D)}
    return {"bytes": 2.0 * 2 * T * H * D + table + 4 * T, "flops": float(per * T * H * D)}


# ---- inputs ----

def _table(positions, rot, device):
    """cos and sin of the rotation angles, [positions][rot]: rot / 2 cosines, then the sines."""
    f = THETA ** (-np.arange(rot // 2) * 2.0 / rot)
    a = np.arange(positions)[:, None] * f[None, :]
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)).to(device)


def prepare(case, seed):
    c, dev = dict(case), "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    host = np.random.default_rng(seed)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16) * std

    def ints(v, dtype=np.int32):
        return torch.from_numpy(np.ascontiguousarray(np.asarray(v, dtype))).to(dev)

    D, n_q, n_kv = c["D"], c["n_q"], c["n_kv"]
    s = dict(case=c, n_q=n_q, n_kv=n_kv, D=D)

    def cache(n_pages, page, fp8, fill):
        """Keys, values [pages][kv heads][page][D] and, in 8 bits, a scale for each kv head."""
        shape = (n_pages, n_kv, page, D)
        if not fp8:
            mk = (lambda std: normal(*shape, std=std)) if fill else (lambda std: torch.zeros(shape, dtype=torch.bfloat16, device=dev))
            return dict(k=mk(1.0), v=mk(0.5), k_scale=None, v_scale=None)
        ks = torch.from_numpy(host.uniform(0.01, 0.02, n_kv).astype(np.float32)).to(dev)
        vs = torch.from_numpy(host.uniform(0.005, 0.01, n_kv).astype(np.float32)).to(dev)
        if not fill:
            z = lambda: torch.zeros(shape, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)  # noqa: E731
            return dict(k=z(), v=z(), k_scale=ks, v_scale=vs)
        codes = lambda std, sc: (normal(*shape, std=std) / sc[None, :, None, None].to(torch.bfloat16)).clamp_(  # noqa: E731
            -448, 448).to(torch.float8_e4m3fn)
        return dict(k=codes(1.0, ks), v=codes(0.5, vs), k_scale=ks, v_scale=vs)

    if c["op"] == "attend":
        lens, page = _lengths(c), c["page"]
        pages = [-(-kv // page) for kv, _ in lens]
        order = host.permutation(sum(pages))
        table = np.zeros((c["B"], max(pages)), np.int32)
        at = 0
        for b, m in enumerate(pages):
            table[b, :m] = order[at:at + m]
            at += m
        T = sum(n for _, n in lens)
        s.update(cache(sum(pages), page, c["fp8"], True))
        s.update(q=normal(T, n_q, D, std=2.0), page_table=ints(table), kv_len=ints([kv for kv, _ in lens]),
                 q_indptr=ints(np.concatenate([[0], np.cumsum([n for _, n in lens])])), max_q=max(n for _, n in lens),
                 scale=1.0 / math.sqrt(D), scratch=torch.zeros(SCRATCH_BYTES, dtype=torch.uint8, device=dev), mask=None)
        if c["tree"]:
            rows = np.array([r for p in _parents(c) for r in _ancestors(p)], np.uint64).view(np.int64)
            s["mask"] = ints(rows[:, None], np.int64)
        return s
    T, width = c["T"], (n_q + 2 * n_kv) * D
    s["qkv"] = normal(T, width, std=1.5)
    s["cos_sin"] = _table(max(2 * T, 64), c["rot"], dev)
    s["q_weight"] = 1.0 + 0.1 * torch.randn(D, generator=g, device=dev) if c["norm"] else None
    s["k_weight"] = 1.0 + 0.1 * torch.randn(D, generator=g, device=dev) if c["norm"] else None
    if c["op"] == "norm_rope":
        s["positions"] = ints(int(host.integers(0, T)) + np.arange(T))
        if c["backward"]:
            s.update(dq=normal(T, n_q, D, std=0.01), dk=normal(T, n_kv, D, std=0.01), dv=normal(T, n_kv, D, std=0.01),
                     scratch=torch.zeros(8 << 20, dtype=torch.uint8, device=dev))
        return s
    page = c["page"]
    if T <= 256:   # a decode batch: each token at its own place of its own sequence
        n_pages = 2 * T
        s["positions"] = ints(host.integers(0, 2 * T, T))
        s["slots"] = ints(host.permutation(n_pages)[:T] * page + host.integers(0, page, T))
    else:          # a prompt: whole pages, in an order of the allocator's
        n_pages = -(-T // page) + 1
        s["positions"] = ints(np.arange(T))
        order = host.permutation(n_pages)
        s["slots"] = ints(order[np.arange(T) // page] * page + np.arange(T) % page)
    s.update(cache(n_pages, page, c["fp8"], False))
    return s


# ---- the plain forms, in 32 bits ----

def _pairs(x, rot, interleaved):
    """The two members of each rotated pair of the last axis."""
    r = x[..., :rot]
    if interleaved:
        return r[..., 0::2], r[..., 1::2]
    return r[..., :rot // 2], r[..., rot // 2:]


def _unpaired(a, b, rest, interleaved):
    r = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([r, rest], -1)


def _rotated(x, cos_sin, positions, interleaved, back=False):
    rot = cos_sin.shape[1]
    cs = cos_sin[positions.long()][:, None, :]
    c, n = cs[..., :rot // 2], cs[..., rot // 2:]
    if back:
        n = -n
    a, b = _pairs(x, rot, interleaved)
    return _unpaired(a * c - b * n, b * c + a * n, x[..., rot:], interleaved)


def _normed(x, w):
    return x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w


def _heads(s):
    """Queries, keys and values of the packed rows, in 32 bits."""
    x = s["qkv"].float().view(s["qkv"].shape[0], -1, s["D"])
    return x[:, :s["n_q"]], x[:, s["n_q"]:s["n_q"] + s["n_kv"]], x[:, s["n_q"] + s["n_kv"]:]


def _plain_norm_rope(s):
    q, k, _ = _heads(s)
    inter = s["case"]["interleaved"]
    return dict(q=_rotated(_normed(q, s["q_weight"]), s["cos_sin"], s["positions"], inter).bfloat16(),
                k=_rotated(_normed(k, s["k_weight"]), s["cos_sin"], s["positions"], inter).bfloat16())


def _plain_backward(s):
    q, k, _ = _heads(s)

    def one(x, dy, w):
        g = _rotated(dy.float(), s["cos_sin"], s["positions"], s["case"]["interleaved"], back=True)
        if w is None:
            return g, None
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        xh = x * r
        dw = (g * xh).sum((0, 1))
        g = g * w
        return r * (g - xh * (g * xh).mean(-1, keepdim=True)), dw

    dq, dqw = one(q, s["dq"], s["q_weight"])
    dk, dkw = one(k, s["dk"], s["k_weight"])
    dqkv = torch.cat([dq, dk, s["dv"].float()], 1).flatten(1).bfloat16()
    return dict(dqkv=dqkv, dq_weight=dqw, dk_weight=dkw)


def _codes(x, scale):
    return (x / scale[None, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_append(s):
    q, k, v = _heads(s)
    inter, page = s["case"]["interleaved"], s["case"]["page"]
    q = _rotated(_normed(q, s["q_weight"]), s["cos_sin"], s["positions"], inter).bfloat16()
    k = _rotated(_normed(k, s["k_weight"]), s["cos_sin"], s["positions"], inter)
    at, off = s["slots"].long() // page, s["slots"].long() % page
    if s["k_scale"] is None:
        s["k"][at, :, off] = k.bfloat16()
        s["v"][at, :, off] = v.bfloat16()
    else:
        s["k"].view(torch.uint8)[at, :, off] = _codes(k, s["k_scale"])
        s["v"].view(torch.uint8)[at, :, off] = _codes(v, s["v_scale"])
    return dict(q=q, k=s["k"], v=s["v"])


def _gathered(s, name, at, off):
    """Cached rows [B][keys][kv heads][D] in 32 bits."""
    x, sc = s[name], s[name + "_scale"]
    if sc is None:
        return x[at, :, off].float()
    return x.view(torch.uint8)[at, :, off].view(torch.float8_e4m3fn).float() * sc[None, None, :, None]


def _plain_attend(s):
    c, q, dev = s["case"], s["q"], s["q"].device
    page, n_q, n_kv, D, n = c["page"], s["n_q"], s["n_kv"], s["D"], s["max_q"]
    B, G = c["B"], s["n_q"] // s["n_kv"]
    keys = torch.arange(s["page_table"].shape[1] * page, device=dev)
    at = s["page_table"].long()[:, keys // page]
    off = (keys % page).expand(B, -1)
    k, v = _gathered(s, "k", at, off), _gathered(s, "v", at, off)
    first, count = s["q_indptr"][:-1].long(), (s["q_indptr"][1:] - s["q_indptr"][:-1]).long()
    j = torch.arange(n, device=dev)
    real = j[None] < count[:, None]                                   # [B][n]
    row = torch.where(real, first[:, None] + j[None], 0)
    qp = q[row].float().view(B, n, n_kv, G, D).permute(0, 2, 3, 1, 4).reshape(B, n_kv, G * n, D)
    kt = k.permute(0, 2, 3, 1).contiguous()
    sc = torch.matmul(qp, kt).view(B, n_kv, G, n, -1) * s["scale"]
    draft = keys[None] - (s["kv_len"].long() - count)[:, None]        # [B][keys]: index among the drafted, or < 0
    if s["mask"] is None:
        seen = draft[:, None] <= j[None, :, None]
    else:
        seen = (draft[:, None] < 0) | ((s["mask"][row, 0][..., None] >> draft.clamp(0, 63)[:, None]) & 1 > 0)
    seen = seen & (keys[None] < s["kv_len"].long()[:, None])[:, None]
    sc = sc.masked_fill(~seen[:, None, None], float("-inf"))
    m = sc.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), 0.0, m)
    p = torch.exp(sc - m)
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, n_kv, G * n, -1), v.permute(0, 2, 1, 3).contiguous()).view(B, n_kv, G, n, D)
    o = torch.where(l > 0, o / l, 0.0).permute(0, 3, 1, 2, 4).reshape(B, n, n_q, D)
    lse = (m + torch.log(l)).squeeze(-1).permute(0, 3, 1, 2).reshape(B, n, n_q)
    return dict(out=o[real].bfloat16(), lse=lse[real])


_P = None


def run(s):
    c = s["case"]
    if not own:
        if c["op"] == "attend":
            return _plain_attend(s)
        if c["op"] == "append":
            return _plain_append(s)
        return _plain_backward(s) if c["backward"] else _plain_norm_rope(s)
    global _P
    if _P is None:
        import precision_gemm_amd
        _P = precision_gemm_amd
    if c["op"] == "attend":
        out, lse = _P.tree_attention(s["q"], s["k"], s["v"], s["page_table"], s["kv_len"], s["q_indptr"], s["max_q"],
                                     tree_mask=s["mask"], scale=s["scale"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                                     workspace=s["scratch"])
        return dict(out=out, lse=lse)
    rope = dict(cos_sin=s["cos_sin"], interleaved=c["interleaved"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS)
    if c["op"] == "append":
        q = _P.rope_append_kv(s["qkv"], s["positions"], s["slots"], s["k"], s["v"], s["n_q"], k_scale=s["k_scale"],
                              v_scale=s["v_scale"], **rope)
        return dict(q=q, k=s["k"], v=s["v"])
    if c["backward"]:
        dqkv, dqw, dkw = _P.qk_norm_rope_backward(s["qkv"], s["positions"], s["dq"], s["dk"], s["dv"],
                                                  workspace=s["scratch"], **rope)
        return dict(dqkv=dqkv, dq_weight=dqw, dk_weight=dkw)
    q, k = _P.qk_norm_rope(s["qkv"], s["positions"], s["n_q"], s["n_kv"], s["D"], **rope)
    return dict(q=q, k=k)


# ---- the definitions, in 64 bits ----

def _exact_angles(s):
    """The rotation of each token as complex numbers (the table's own 32-bit values)."""
    t = s["cos_sin"].double()[s["positions"].long()]
    half = t.shape[1] // 2
    return torch.complex(t[:, :half], t[:, half:])


def _exact_head(x, w, z, interleaved):
    """One head [T][D]: its norm, and its pairs as complex numbers times z."""
    if w is not None:
        x = x / torch.sqrt(x.square().mean(1, keepdim=True) + EPS) * w.double()
    return _exact_turn(x, z, interleaved)


def _exact_turn(x, z, interleaved):
    half = z.shape[1]
    first, second = (torch.arange(half) * 2, torch.arange(half) * 2 + 1) if interleaved else (torch.arange(half), torch.arange(half) + half)
    y = x.clone()
    t = torch.complex(x[:, first], x[:, second]) * z
    y[:, first], y[:, second] = t.real, t.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    c, D, n_q, n_kv = s["case"], s["D"], s["n_q"], s["n_kv"]
    if c["op"] == "attend":
        return _exact_attend(s)
    x, z, inter = s["qkv"].double(), _exact_angles(s), c["interleaved"]
    head = lambda h: x[:, h * D:(h + 1) * D]  # noqa: E731
    if c["op"] == "norm_rope" and c["backward"]:
        cols, dws = [], []
        for heads, dy, w in ((range(n_q), s["dq"], s["q_weight"]), (range(n_q, n_q + n_kv), s["dk"], s["k_weight"])):
            dw = torch.zeros(D, dtype=torch.float64, device=x.device)
            for i, h in enumerate(heads):
                g = _exact_turn(dy[:, i].double(), z.conj(), inter)
                if w is not None:
                    norm = torch.sqrt(head(h).square().mean(1, keepdim=True) + EPS)
                    dw += (g * head(h) / norm).sum(0)
                    gw = g * w.double()
                    g = gw / norm - head(h) * (gw * head(h)).sum(1, keepdim=True) / (D * norm ** 3)
                cols.append(g)
            dws.append(None if w is None else dw)
        cols.append(s["dv"].double().flatten(1))
        return dict(dqkv=torch.cat(cols, 1), dq_weight=dws[0], dk_weight=dws[1])
    q = torch.stack([_exact_head(head(h), s["q_weight"], z, inter) for h in range(n_q)], 1)
    k = torch.stack([_exact_head(head(n_q + h), s["k_weight"], z, inter) for h in range(n_kv)], 1)
    if c["op"] == "norm_rope":
        return dict(q=q, k=k)
    kc, vc = s["k"].double(), s["v"].double()
    v = x[:, (n_q + n_kv) * D:].reshape(-1, n_kv, D)
    if c["fp8"]:   # the codes' values before their rounding to 8 bits
        k = (k / s["k_scale"].double()[None, :, None]).clamp(-448, 448)
        v = (v / s["v_scale"].double()[None, :, None]).clamp(-448, 448)
    slot = s["slots"].cpu().numpy()
    at, off = (torch.from_numpy(a.astype(np.int64)).to(x.device) for a in divmod(slot, c["page"]))
    for h in range(n_kv):
        kc[at, h, off], vc[at, h, off] = k[:, h], v[:, h]
    return dict(q=q, k=kc, v=vc)


def _exact_attend(s):
    c, page, n_kv, G = s["case"], s["case"]["page"], s["n_kv"], s["n_q"] // s["n_kv"]
    outs, lses, at = [], [], 0
    for b, ((kv, n), par) in enumerate(zip(_lengths(c), _parents(c))):
        ids = s["page_table"][b, :-(-kv // page)].long()
        out = torch.zeros(n, s["n_q"], s["D"], dtype=torch.float64, device=ids.device)
        lse = torch.zeros(n, s["n_q"], dtype=torch.float64, device=ids.device)
        seen = torch.ones(n, kv, dtype=torch.bool)
        seen[:, kv - n:] = torch.tensor([[bool(m >> i & 1) for i in range(n)] for m in _ancestors(par)])
        seen = seen.to(ids.device)
        for h in range(n_kv):
            k, v = s["k"][ids, h].double().flatten(0, 1)[:kv], s["v"][ids, h].double().flatten(0, 1)[:kv]
            if c["fp8"]:
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            for i in range(h * G, (h + 1) * G):
                sc = (s["q"][at:at + n, i].double() * s["scale"]) @ k.T
                sc = torch.where(seen, sc, -math.inf)
                lse[:, i] = torch.logsumexp(sc, 1)
                out[:, i] = torch.exp(sc - lse[:, i:i + 1]) @ v
        outs.append(out)
        lses.append(lse)
        at += n
    return dict(out=torch.cat(outs), lse=torch.cat(lses))
