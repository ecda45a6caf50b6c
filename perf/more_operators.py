"""What stands around the low-precision layer in a step of serving or training, as cases to measure.

Three operators: the norm of the hidden states in front of a projection (layer norm or RMS norm,
with the residual's addition; forward and backward), an AdamW step over all tenants' adapters at
once (states in 32 or 8 bits, each tenant with its own rates, step count and gradient norm) that
writes the adapters in the forms the layer reads, and the head norm and rotation with positions of
several axes (forward, backward, and into a paged cache).  ``run`` computes a case in its plain
form (torch operations in 32 bits), or with ``own`` set calls this library's kernels; ``exact`` is
the same from the definitions in 64 bits.
"""

import math
import random

import numpy as np
import torch

own = False

EPS = 1e-6
THETA = 10000.0
BLOCK = 64                       # values that share a scale of the 8-bit states
E4M3_MAX, E4M3_LEAST = 448.0, 2.0 ** -9
NO_SCALE = 2.0 ** -100           # blocks whose largest value is below this are held as zero


def listed():
    """The cases.  4,096 channels, 32 + 8 + 8 heads of 128 and the projections 4096 x 6144,
    4096 x 4096, 4096 x 28672 and 14336 x 4096 are the repository's decoder layer; 16 and 4,096
    tokens its decode and prefill batches."""
    layer = "4096x6144,4096x4096,4096x28672,14336x4096"
    heads = dict(n_q=32, n_kv=8, D=128, rot=128)
    return [
        # a decode batch, the attention's output added to the residual stream: the launch is what counts
        dict(name="norm_decode", op="norm", T=16, K=4096, rms=False, residual=True, backward=False),
        # a prompt, or a training micro-batch, of 4,096 tokens
        dict(name="norm_prefill", op="norm", T=4096, K=4096, rms=True, residual=True, backward=False),
        # its backward, with the gradient that comes along the residual stream and both weights' gradients
        dict(name="norm_backward", op="norm", T=4096, K=4096, rms=False, residual=True, backward=True),
        # the backward of an odd batch of a wider model, no residual
        dict(name="norm_backward_odd", op="norm", T=1001, K=5376, rms=True, residual=False, backward=True),
        # a decode batch of conversations with images: one token each into a 16-bit cache
        dict(name="axes_append_decode", op="axes", T=16, **heads, sections="16,24,24", mixed=False, interleaved=False,
             norm=False, call="append", page=16, fp8=False),
        # a prompt of text and images into an 8-bit cache, with the heads' norms on the way
        dict(name="axes_append_prefill_fp8", op="axes", T=4096, **heads, sections="16,24,24", mixed=False,
             interleaved=False, norm=True, call="append", page=64, fp8=True),
        # the backward of such a batch in training
        dict(name="axes_backward", op="axes", T=4096, **heads, sections="16,24,24", mixed=False, interleaved=False,
             norm=True, call="backward"),
        # an odd batch: small heads, the axes taken in turn over the frequencies
        dict(name="axes_forward_odd", op="axes", T=1001, n_q=28, n_kv=4, D=64, rot=64, sections="11,11,10", mixed=True,
             interleaved=True, norm=True, call="forward"),
        # one tenant's adapter of one projection: the smallest step
        dict(name="adamw_one_adapter", op="adamw", ranks="8", projections="4096x4096", plain="", idle="", bits=32, clip=False),
        # 32 tenants' adapters of a decoder layer, clipped tenant by tenant
        dict(name="adamw_layer", op="adamw", ranks=",".join(["16"] * 32), projections=layer, plain="", idle="", bits=32,
             clip=True),
        # the same with states in 8 bits
        dict(name="adamw_layer_8bit", op="adamw", ranks=",".join(["16"] * 32), projections=layer, plain="", idle="", bits=8,
             clip=True),
        # tenants of all ranks, some without tokens in this batch, and two norms' weights
        dict(name="adamw_odd_8bit", op="adamw", ranks="64,5,33,8,1,16,24", projections="4096x6144,1792x5376",
             plain="4096,1001", idle="3,5", bits=8, clip=False),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm, odd ones among them."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, v))


def draw(rng):
    """One more case of these ranges: 1 to 8,192 tokens of 64 to 16,384 channels, heads of 64, 128
    or 256, two to four axes, 1 to 32 tenants of ranks 1 to 64 with 1 to 4 projections."""
    while True:
        op = rng.choice(("norm", "axes", "adamw"))
        if op == "norm":
            c = dict(op=op, T=_log(rng, 1, 8192), K=8 * _log(rng, 8, 2048), rms=rng.random() < 0.5,
                     residual=rng.random() < 0.6, backward=rng.random() < 0.6)
        elif op == "axes":
            D = rng.choice((64, 128, 128, 256))
            n_q, n_kv = rng.choice(((32, 8), (8, 1), (28, 4), (16, 8), (40, 8), (6, 6), (15, 3), (4, 2)))
            rot = rng.choice((D, D, D // 2))
            n, half, sections = rng.choice((2, 3, 3, 4)), rot // 2, []
            unit = rng.choice((8, 4, 1)) if rot >= 64 else rng.choice((4, 1))
            cuts = sorted(rng.sample(range(1, half // unit), n - 1))
            sections = [unit * (b - a) for a, b in zip([0] + cuts, cuts + [half // unit])]
            c = dict(op=op, T=_log(rng, 1, 8192), n_q=n_q, n_kv=n_kv, D=D, rot=rot, sections=",".join(map(str, sections)),
                     mixed=rng.random() < 0.3, interleaved=rng.random() < 0.3, norm=rng.random() < 0.7,
                     call=rng.choice(("forward", "append", "backward")))
            if c["call"] == "append":
                c.update(page=rng.choice((16, 32, 64, 128)), fp8=rng.random() < 0.5)
        else:
            tenants = _log(rng, 1, 32)
            ranks = [rng.choice((8, 16, 32, 64, _log(rng, 1, 64))) for _ in range(tenants)]
            projections = ["%dx%d" % (128 * _log(rng, 2, 128), 64 * _log(rng, 4, 448)) for _ in range(rng.randint(1, 4))]
            plain = [str(_log(rng, 1, 8192)) for _ in range(rng.choice((0, 0, 1, 4)))]
            idle = [str(t) for t in range(tenants) if tenants > 2 and rng.random() < 0.15]
            c = dict(op=op, ranks=",".join(map(str, ranks)), projections=",".join(projections), plain=",".join(plain),
                     idle=",".join(idle), bits=rng.choice((8, 32)), clip=rng.random() < 0.5)
            if len(idle) == tenants or sum(n for _, n, _ in _spans(c)) > 3.6e7:
                continue
        return c


# ---- what a case's sizes are ----

def _numbers(text):
    return [int(v) for v in text.split(",") if v]


def _axes(c):
    """The axis of each pair of a head: the sections one after another, or taken in turn."""
    sections = _numbers(c["sections"])
    if not c["mixed"]:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, out = list(sections), []
    while sum(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return out


def _up(v, m):
    return -(-v // m) * m


def _tensors(c):
    """(kind, rows, columns, tenant) of every tensor that a step takes: A [K, r] and B [r, N] of each
    projection and tenant, then the plain ones (tenant 0's)."""
    out = []
    for p in c["projections"].split(","):
        K, N = (int(v) for v in p.split("x"))
        for tenant, r in enumerate(_numbers(c["ranks"])):
            out += [("A", K, r, tenant), ("B", r, N, tenant)]
    return out + [("plain", 1, n, 0) for n in _numbers(c["plain"])]


def _spans(c):
    """(first, values, tenant) of every tensor in the buffers that hold all of them."""
    out, at = [], 0
    for _, rows, cols, tenant in _tensors(c):
        out.append((at, rows * cols, tenant))
        at += _up(rows * cols, BLOCK)
    return out


def _packed(kind, rows, cols):
    """Values of a tensor's two packed forms, for the forward and for the backward pass."""
    if kind == "plain":
        return 0, 0
    if kind == "A":
        return _up(cols, 16) * rows, rows * _up(cols, 8)
    return cols * _up(rows, 8), _up(rows, 16) * cols


def work(c):
    if c["op"] == "norm":
        T, K = c["T"], c["K"]
        if c["backward"]:
            return {"bytes": 2.0 * T * K * (4 if c["residual"] else 3) + 4.0 * K * (2 if c["rms"] else 3), "flops": 16.0 * T * K}
        return {"bytes": 2.0 * T * K * (4 if c["residual"] else 2) + 4.0 * K * (1 if c["rms"] else 2), "flops": 8.0 * T * K}
    if c["op"] == "axes":
        T, D, n_q, n_kv = c["T"], c["D"], c["n_q"], c["n_kv"]
        H, per = n_q + n_kv, (8 if c["norm"] else 0) + 3
        table = 4.0 * T * c["rot"] + 4.0 * T * len(_numbers(c["sections"]))
        if c["call"] == "append":
            return {"bytes": 2.0 * T * (H + n_kv) * D + 2.0 * T * n_q * D + 2.0 * T * n_kv * D * (1 if c["fp8"] else 2) + table
                    + 4 * T, "flops": float(per * T * H * D)}
        if c["call"] == "backward":
            return {"bytes": 2.0 * T * H * D * (3 if c["norm"] else 2) + 2.0 * T * n_kv * D * 2 + table,
                    "flops": float(2 * per * T * H * D)}
        return {"bytes": 2.0 * 2 * T * H * D + table, "flops": float(per * T * H * D)}
    idle, state = set(_numbers(c["idle"])), 16.0 if c["bits"] == 32 else 4.0 + 16.0 / BLOCK
    b = f = 0.0
    for kind, rows, cols, tenant in _tensors(c):
        if tenant not in idle:
            n = rows * cols
            b += n * (4 + 8 + state) + (2 * n if kind != "plain" else 0) + 2 * sum(_packed(kind, rows, cols))
            f += 20.0 * n
    return {"bytes": b, "flops": f}


# ---- inputs ----

def _table(positions, rot, device):
    """cos and sin of the rotation angles, [positions][rot]: rot / 2 cosines, then the sines."""
    f = THETA ** (-np.arange(rot // 2) * 2.0 / rot)
    a = np.arange(positions)[:, None] * f[None, :]
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)).to(device)


def _prepare_norm(c, normal, g, dev):
    T, K = c["T"], c["K"]
    scale = torch.where(torch.rand(K, generator=g, device=dev) < 0.003, 20.0, 1.0)  # a few channels stand out
    x = (torch.randn(T, K, generator=g, device=dev) * scale + 0.3 * torch.randn(T, 1, generator=g, device=dev)).bfloat16()
    s = dict(case=c, x=x, weight=1.0 + 0.1 * torch.randn(K, generator=g, device=dev),
             bias=None if c["rms"] else 0.1 * torch.randn(K, generator=g, device=dev), residual=None, dsum=None)
    if c["backward"]:
        s.update(dy=normal(T, K, std=0.01), scratch=torch.zeros(64 << 20, dtype=torch.uint8, device=dev))
        if c["residual"]:
            s["dsum"] = normal(T, K, std=0.01)
    elif c["residual"]:
        s["residual"] = normal(T, K, std=1.5)
    return s


def _prepare_axes(c, normal, g, dev, host):
    T, n_q, n_kv, D, rot = c["T"], c["n_q"], c["n_kv"], c["D"], c["rot"]
    axes = _axes(c)
    n = max(axes) + 1
    # text, whose axes go together, and images of up to 24 x 40 patches, which share one time
    pos, at, where = np.zeros((n, T), np.int64), int(host.integers(0, 100)), 0
    while where < T:
        m = min(int(host.integers(1, 200)), T - where)
        pos[:, where:where + m] = at + np.arange(m)
        at, where = at + m, where + m
        h, w = int(host.integers(2, 25)), int(host.integers(2, 41))
        m = min(h * w, T - where)
        patch = np.arange(m)
        pos[:, where:where + m] = at
        pos[1, where:where + m] += patch // w
        pos[n - 1, where:where + m] += patch % w
        at, where = at + max(h, w), where + m
    s = dict(case=c, qkv=normal(T, (n_q + 2 * n_kv) * D, std=1.5), cos_sin=_table(int(pos.max()) + 64, rot, dev),
             positions=torch.from_numpy(pos.astype(np.int32)).to(dev), pair_axes=bytes(axes),
             axis=torch.tensor(axes, device=dev), q_weight=None, k_weight=None)
    if c["norm"]:
        s["q_weight"] = 1.0 + 0.1 * torch.randn(D, generator=g, device=dev)
        s["k_weight"] = 1.0 + 0.1 * torch.randn(D, generator=g, device=dev)
    if c["call"] == "backward":
        s.update(dq=normal(T, n_q, D, std=0.01), dk=normal(T, n_kv, D, std=0.01), dv=normal(T, n_kv, D, std=0.01),
                 scratch=torch.zeros(8 << 20, dtype=torch.uint8, device=dev))
    elif c["call"] == "append":
        page = c["page"]
        if T <= 256:   # a decode batch: each token at its own place of its own sequence
            pages = 2 * T
            slots = host.permutation(pages)[:T] * page + host.integers(0, page, T)
        else:          # a prompt: whole pages, in an order of the allocator's
            pages = -(-T // page) + 1
            slots = host.permutation(pages)[np.arange(T) // page] * page + np.arange(T) % page
        s["slots"] = torch.from_numpy(slots.astype(np.int32)).to(dev)
        shape = (pages, n_kv, page, D)
        kind = torch.uint8 if c["fp8"] else torch.bfloat16
        s["k"], s["v"] = (torch.zeros(shape, dtype=kind, device=dev) for _ in range(2))
        s["k_scale"] = s["v_scale"] = None
        if c["fp8"]:
            s["k"], s["v"] = s["k"].view(torch.float8_e4m3fn), s["v"].view(torch.float8_e4m3fn)
            s["k_scale"] = torch.from_numpy(host.uniform(0.01, 0.02, n_kv).astype(np.float32)).to(dev)
            s["v_scale"] = torch.from_numpy(host.uniform(0.005, 0.01, n_kv).astype(np.float32)).to(dev)
    return s


def _operand_index(red, r, at_rank, at_red, device):
    """Source of each value of a matrix in MFMA operand order (tiles of 16 ranks, steps of 64 along
    the reduction): -1 where it is padding."""
    e = torch.arange(_up(r, 16) * red, device=device)
    k = e // 1024 % (red // 64) * 64 + e // 128 % 4 * 16 + e // 512 % 2 * 8 + e % 8
    j = e // (16 * red) * 16 + e // 8 % 16
    return torch.where(j < r, j * at_rank + k * at_red, -1)


def _rows_index(n, r, at_rank, at_row, device):
    """Source of each value of rows of r ranks, padded to a multiple of 8 (-1: padding)."""
    e = torch.arange(n * _up(r, 8), device=device)
    j, i = e % _up(r, 8), e // _up(r, 8)
    return torch.where(j < r, j * at_rank + i * at_row, -1)


def _held(x, floor, dev):
    """8-bit codes and scales of blocks [n, 64]; with `floor`, what is not 0 keeps a code that is not."""
    most = x.abs().amax(1, keepdim=True)
    most = torch.where(most >= NO_SCALE, most, 0.0)
    q = x * torch.where(most > 0, E4M3_MAX / most, 0.0)
    if floor:
        q = torch.where((x > 0) & (most > 0), q.clamp(min=E4M3_LEAST), q)
    return q.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), most / E4M3_MAX


def _prepare_adamw(c, g, dev, host):
    tensors, spans = _tensors(c), _spans(c)
    ranks = _numbers(c["ranks"])
    total = spans[-1][0] + _up(spans[-1][1], BLOCK)
    adapters = sum(n for (_, n, _), t in zip(spans, tensors) if t[0] != "plain")
    std = 10.0 ** host.uniform(-4.0, -2.5, len(ranks))   # of each tenant's gradients
    tenant = torch.cat([torch.full((_up(n, BLOCK) // BLOCK,), t, dtype=torch.int32) for _, n, t in spans]).to(dev)
    gstd = torch.from_numpy(std.astype(np.float32)).to(dev)[tenant.long()][:, None]
    rand = lambda: torch.randn(total // BLOCK, BLOCK, generator=g, device=dev)  # noqa: E731
    param, grad, m = rand() * 0.016, rand() * gstd, rand() * gstd * 0.3
    v = gstd * gstd * (rand().abs() * 0.3 + 0.5)
    for (at, n, _), t in zip(spans, tensors):   # what lies between two tensors is zero
        for b in (param, grad, m, v):
            b.view(-1)[at + n:at + _up(n, BLOCK)] = 0.0
    s = dict(case=c, param=param.view(-1), grad=grad.view(-1), tenant=tenant, adapters=adapters)
    if c["bits"] == 32:
        s.update(m=m.view(-1), v=v.view(-1), m_scale=None, v_scale=None)
    else:
        (m, ms), (v, vs) = _held(m, False, dev), _held(v.sqrt(), True, dev)
        s.update(m=m.view(-1), v=v.view(-1), m_scale=ms.view(-1), v_scale=vs.view(-1))
    # the adapters in 16 bits, [K, r] and [r, N] as they are and in the forms that the layer and its backward read
    index = [[], []]
    for (at, _, _), (kind, rows, cols, _) in zip(spans, tensors):
        if kind == "plain":
            continue
        pair = (_operand_index(rows, cols, 1, cols, dev), _rows_index(rows, cols, 1, cols, dev)) if kind == "A" else \
            (_rows_index(cols, rows, cols, 1, dev), _operand_index(cols, rows, cols, 1, dev))
        for ix, p in zip(index, pair):
            ix.append(torch.where(p < 0, adapters, p + at).int())
    s["copy"] = torch.cat([s["param"][:adapters].bfloat16(), torch.zeros(BLOCK, dtype=torch.bfloat16, device=dev)])
    s["index"] = [torch.cat(ix) for ix in index]
    s["pack"], s["pack_bwd"] = (s["copy"].index_select(0, ix) for ix in s["index"])
    G = len(ranks)
    hyper = np.zeros((G, 6))   # rate, beta1, beta2, epsilon, weight decay, largest gradient norm
    hyper[:, 0], hyper[:, 1], hyper[:, 2] = host.uniform(1e-5, 5e-5, G), 0.9, host.choice((0.95, 0.99, 0.999), G)
    hyper[:, 3], hyper[:, 4], hyper[:, 5] = 1e-8, host.uniform(0.0, 0.1, G), 1.0
    s["hyper"] = torch.from_numpy(hyper).to(dev)
    s["steps"] = torch.from_numpy(host.integers(0, 1000, G).astype(np.int32)).to(dev)
    active = np.ones(G, np.int32)
    active[_numbers(c["idle"])] = 0
    s["active"] = torch.from_numpy(active).to(dev)
    if own:
        s["optimizer"] = _optimizer(s, tensors, spans)
    return s


def _optimizer(s, tensors, spans):
    """The library's handle on these buffers."""
    import precision_gemm_amd as P
    c, out, at_pack = s["case"], [], [0, 0]
    for (at, n, _), (kind, rows, cols, tenant) in zip(spans, tensors):
        part = lambda b: None if b is None else b[at:at + n].view(rows, cols)  # noqa: E731
        scale = lambda b: None if b is None else b[at // BLOCK:(at + _up(n, BLOCK)) // BLOCK]  # noqa: E731
        packs = []
        for k, size in enumerate(_packed(kind, rows, cols)):
            packs.append(s[("pack", "pack_bwd")[k]][at_pack[k]:at_pack[k] + size] if size else None)
            at_pack[k] += size
        out.append(P.AdamWTensor(param=part(s["param"]), grad=part(s["grad"]), group=tenant, kind=kind, m=part(s["m"]),
                                 v=part(s["v"]), m_scale=scale(s["m_scale"]), v_scale=scale(s["v_scale"]),
                                 copy=part(s["copy"]) if kind != "plain" else None, pack=packs[0], pack_bwd=packs[1]))
    return P.AdamW(out, len(s["steps"]), state_bits=c["bits"], steps=s["steps"])


def prepare(case, seed):
    c, dev = dict(case), "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    host = np.random.default_rng(seed)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16) * std

    if c["op"] == "norm":
        return _prepare_norm(c, normal, g, dev)
    if c["op"] == "axes":
        return _prepare_axes(c, normal, g, dev, host)
    return _prepare_adamw(c, g, dev, host)


# ---- the plain forms, in 32 bits ----

def _plain_norm(s):
    x = s["x"].float()
    if s["residual"] is not None:
        x = (x + s["residual"].float()).bfloat16().float()
    d = x if s["case"]["rms"] else x - x.mean(1, keepdim=True)
    y = d * torch.rsqrt((d * d).mean(1, keepdim=True) + EPS) * s["weight"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return dict(y=y.bfloat16(), h=x.bfloat16())


def _plain_norm_backward(s):
    x, dy, rms = s["x"].float(), s["dy"].float(), s["case"]["rms"]
    d = x if rms else x - x.mean(1, keepdim=True)
    r = torch.rsqrt((d * d).mean(1, keepdim=True) + EPS)
    xh = d * r
    g = dy * s["weight"]
    dx = g - xh * (g * xh).mean(1, keepdim=True)
    if not rms:
        dx = dx - g.mean(1, keepdim=True)
    dx = dx * r
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    return dict(dx=dx.bfloat16(), dweight=(dy * xh).sum(0), dbias=None if rms else dy.sum(0))


def _rotated(x, s, back=False):
    rot, inter = s["case"]["rot"], s["case"]["interleaved"]
    half = rot // 2
    pos = s["positions"].long()[s["axis"]].T                       # [T][pairs]
    pair = torch.arange(half, device=pos.device)
    cos, sin = s["cos_sin"][pos, pair][:, None], s["cos_sin"][pos, half + pair][:, None]
    if back:
        sin = -sin
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if inter else (r[..., :half], r[..., half:])
    a, b = a * cos - b * sin, b * cos + a * sin
    return torch.cat([torch.stack([a, b], -1).flatten(-2) if inter else torch.cat([a, b], -1), x[..., rot:]], -1)


def _heads(s):
    """Queries, keys and values of the packed rows, in 32 bits."""
    c = s["case"]
    x = s["qkv"].float().view(c["T"], -1, c["D"])
    return x[:, :c["n_q"]], x[:, c["n_q"]:c["n_q"] + c["n_kv"]], x[:, c["n_q"] + c["n_kv"]:]


def _normed(x, w):
    return x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w


def _codes(x, scale):
    return (x / scale[None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_axes(s):
    c = s["case"]
    q, k, v = _heads(s)
    q, k = _rotated(_normed(q, s["q_weight"]), s).bfloat16(), _rotated(_normed(k, s["k_weight"]), s)
    if c["call"] == "forward":
        return dict(q=q, k=k.bfloat16())
    at, off = s["slots"].long() // c["page"], s["slots"].long() % c["page"]
    if c["fp8"]:
        s["k"].view(torch.uint8)[at, :, off] = _codes(k, s["k_scale"])
        s["v"].view(torch.uint8)[at, :, off] = _codes(v, s["v_scale"])
    else:
        s["k"][at, :, off] = k.bfloat16()
        s["v"][at, :, off] = v.bfloat16()
    return dict(q=q, k=s["k"], v=s["v"])


def _plain_axes_backward(s):
    def one(x, dy, w):
        g = _rotated(dy.float(), s, back=True)
        if w is None:
            return g, None
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        xh = x * r
        dw = (g * xh).sum((0, 1))
        g = g * w
        return r * (g - xh * (g * xh).mean(-1, keepdim=True)), dw

    q, k, _ = _heads(s)
    (dq, dqw), (dk, dkw) = one(q, s["dq"], s["q_weight"]), one(k, s["dk"], s["k_weight"])
    return dict(dqkv=torch.cat([dq, dk, s["dv"].float()], 1).flatten(1).bfloat16(), dq_weight=dqw, dk_weight=dkw)


def _plain_adamw(s):
    c, tenant, G = s["case"], s["tenant"].long(), len(s["steps"])
    blocks = lambda b: b.view(-1, BLOCK)  # noqa: E731
    g, p = blocks(s["grad"]), blocks(s["param"])
    active = s["active"] > 0
    rate, b1, b2, eps, decay, most = s["hyper"].unbind(1)
    clip = norm = None
    if c["clip"]:   # long sums, in 64 bits
        sums = torch.zeros(G, dtype=torch.float64, device=g.device).index_add_(0, tenant, g.double().square().sum(1))
        norm = torch.where(active, sums.sqrt(), 0.0)
        clip = (most / (norm + 1e-6)).clamp(max=1.0)
        active = active & torch.isfinite(norm)
    s["steps"] += active.int()
    t = s["steps"].double()
    of = lambda x: x.float()[tenant][:, None]  # noqa: E731
    if clip is not None:
        g = g * of(clip)
    m, v = blocks(s["m"]), blocks(s["v"])
    if c["bits"] == 8:
        m, root = m.float() * s["m_scale"][:, None], v.float() * s["v_scale"][:, None]
        v = root * root
    m = m * of(b1) + g * of(1.0 - b1)
    v = v * of(b2) + (g * g) * of(1.0 - b2)
    root = v.sqrt()
    d = root * of(1.0 / (1.0 - b2 ** t).sqrt()) + of(eps)
    new = p * of(1.0 - rate * decay) - (m / d) * of(rate / (1.0 - b1 ** t))
    on = active[tenant][:, None]
    p.copy_(torch.where(on, new, p))
    if c["bits"] == 8:
        (mq, ms), (vq, vs) = _held(m, False, g.device), _held(root, True, g.device)
        keep = lambda a, b: torch.where(on, a.view(torch.uint8), blocks(b).view(torch.uint8)).view(-1)  # noqa: E731
        s["m"].view(torch.uint8).copy_(keep(mq, s["m"]))
        s["v"].view(torch.uint8).copy_(keep(vq, s["v"]))
        s["m_scale"].copy_(torch.where(on, ms, s["m_scale"][:, None]).view(-1))
        s["v_scale"].copy_(torch.where(on, vs, s["v_scale"][:, None]).view(-1))
    else:
        s["m"].copy_(torch.where(on, m, blocks(s["m"])).view(-1))
        s["v"].copy_(torch.where(on, v, blocks(s["v"])).view(-1))
    s["copy"][:s["adapters"]].copy_(s["param"][:s["adapters"]])
    s["pack"], s["pack_bwd"] = (s["copy"].index_select(0, ix) for ix in s["index"])
    return _adamw_outputs(s, norm)


def _adamw_outputs(s, norm):
    return dict(param=s["param"], m=s["m"], v=s["v"], m_scale=s["m_scale"], v_scale=s["v_scale"], copy=s["copy"],
                pack=s["pack"], pack_bwd=s["pack_bwd"], steps=s["steps"], norm=None if norm is None else norm.float())


_P = None


def _own(s):
    global _P
    if _P is None:
        import precision_gemm_amd
        _P = precision_gemm_amd
    c = s["case"]
    if c["op"] == "adamw":
        return _adamw_outputs(s, _P.adamw_step(s["optimizer"], s["hyper"], active=s["active"], clip=c["clip"]))
    if c["op"] == "norm":
        if c["backward"]:
            dx, dw, db = _P.layer_norm_backward(s["dy"], s["x"], s["weight"], dsum=s["dsum"], eps=EPS, rms=c["rms"],
                                                bias_grad=not c["rms"], workspace=s["scratch"])
            return dict(dx=dx, dweight=dw, dbias=db)
        y, h = _P.layer_norm(s["x"], s["weight"], s["bias"], residual=s["residual"], eps=EPS, rms=c["rms"])
        return dict(y=y, h=h)
    rope = dict(cos_sin=s["cos_sin"], pair_axes=s["pair_axes"], interleaved=c["interleaved"], q_weight=s["q_weight"],
                k_weight=s["k_weight"], eps=EPS)
    if c["call"] == "append":
        q = _P.rope_append_kv(s["qkv"], s["positions"], s["slots"], s["k"], s["v"], c["n_q"], k_scale=s["k_scale"],
                              v_scale=s["v_scale"], **rope)
        return dict(q=q, k=s["k"], v=s["v"])
    if c["call"] == "backward":
        dqkv, dqw, dkw = _P.qk_norm_rope_backward(s["qkv"], s["positions"], s["dq"], s["dk"], s["dv"],
                                                  workspace=s["scratch"], **rope)
        return dict(dqkv=dqkv, dq_weight=dqw, dk_weight=dkw)
    q, k = _P.qk_norm_rope(s["qkv"], s["positions"], c["n_q"], c["n_kv"], c["D"], **rope)
    return dict(q=q, k=k)


def run(s):
    c = s["case"]
    if own:
        return _own(s)
    if c["op"] == "norm":
        return _plain_norm_backward(s) if c["backward"] else _plain_norm(s)
    if c["op"] == "axes":
        return _plain_axes_backward(s) if c["call"] == "backward" else _plain_axes(s)
    return _plain_adamw(s)


# ---- the definitions, in 64 bits ----

def _exact_norm(s):
    c = s["case"]
    h = s["x"].double()
    if s["residual"] is not None:
        h = (h + s["residual"].double()).float().bfloat16().double()   # what the layer after next adds to
    mean = torch.zeros_like(h[:, :1]) if c["rms"] else h.mean(1, keepdim=True)
    dev = torch.sqrt((h - mean).square().mean(1, keepdim=True) + EPS)
    w = s["weight"].double()
    if not c["backward"]:
        y = (h - mean) / dev * w
        return dict(y=y if s["bias"] is None else y + s["bias"].double(), h=h)
    dy, K = s["dy"].double(), c["K"]
    g = dy * w
    dx = g / dev - (h - mean) * (g * (h - mean)).sum(1, keepdim=True) / (K * dev ** 3)
    if not c["rms"]:
        dx = dx - g.sum(1, keepdim=True) / (K * dev)
    if s["dsum"] is not None:
        dx = dx + s["dsum"].double()
    return dict(dx=dx, dweight=(dy * (h - mean) / dev).sum(0), dbias=None if c["rms"] else dy.sum(0))


def _exact_axes(s):
    c = s["case"]
    D, n_q, n_kv, half = c["D"], c["n_q"], c["n_kv"], c["rot"] // 2
    x, table, pos = s["qkv"].double(), s["cos_sin"].double(), s["positions"].long()
    z = torch.empty(c["T"], half, dtype=torch.complex128, device=x.device)
    for i, a in enumerate(_axes(c)):   # the table's own 32-bit values
        z[:, i] = torch.complex(table[pos[a], i], table[pos[a], half + i])
    first, second = ([2 * i for i in range(half)], [2 * i + 1 for i in range(half)]) if c["interleaved"] else \
        (list(range(half)), list(range(half, 2 * half)))

    def turn(v, by):
        out = v.clone()
        t = torch.complex(v[:, first], v[:, second]) * by
        out[:, first], out[:, second] = t.real, t.imag
        return out

    def head(h):
        return x[:, h * D:(h + 1) * D]

    def forward(h, w):
        v = head(h)
        if w is not None:
            v = v / torch.sqrt(v.square().mean(1, keepdim=True) + EPS) * w.double()
        return turn(v, z)

    if c["call"] == "backward":
        cols, dws = [], []
        for heads, dy, w in ((range(n_q), s["dq"], s["q_weight"]), (range(n_q, n_q + n_kv), s["dk"], s["k_weight"])):
            dw = torch.zeros(D, dtype=torch.float64, device=x.device)
            for i, h in enumerate(heads):
                g = turn(dy[:, i].double(), z.conj())
                if w is not None:
                    norm = torch.sqrt(head(h).square().mean(1, keepdim=True) + EPS)
                    dw += (g * head(h) / norm).sum(0)
                    gw = g * w.double()
                    g = gw / norm - head(h) * (gw * head(h)).sum(1, keepdim=True) / (D * norm ** 3)
                cols.append(g)
            dws.append(None if w is None else dw)
        cols.append(s["dv"].double().flatten(1))
        return dict(dqkv=torch.cat(cols, 1), dq_weight=dws[0], dk_weight=dws[1])
    q = torch.stack([forward(h, s["q_weight"]) for h in range(n_q)], 1)
    k = torch.stack([forward(n_q + h, s["k_weight"]) for h in range(n_kv)], 1)
    if c["call"] == "forward":
        return dict(q=q, k=k)
    v = x[:, (n_q + n_kv) * D:].reshape(-1, n_kv, D)
    if c["fp8"]:   # the codes' values before their rounding to 8 bits
        k = (k / s["k_scale"].double()[None, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
        v = (v / s["v_scale"].double()[None, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    kc, vc = s["k"].double(), s["v"].double()
    at, off = (s["slots"] // c["page"]).long(), (s["slots"] % c["page"]).long()
    for h in range(n_kv):
        kc[at, h, off], vc[at, h, off] = k[:, h], v[:, h]
    return dict(q=q, k=kc, v=vc)


def _exact_adamw(s):
    c, bits = s["case"], s["case"]["bits"]
    tensors, spans = _tensors(c), _spans(c)
    hyper, active = s["hyper"].tolist(), s["active"].tolist()
    steps = [n + (1 if on else 0) for n, on in zip(s["steps"].tolist(), active)]
    G, scales = len(steps), None
    norms = [0.0] * G
    if c["clip"]:
        for at, n, t in spans:
            norms[t] += float(s["grad"][at:at + n].double().square().sum())
        norms = [math.sqrt(v) if on else 0.0 for v, on in zip(norms, active)]
    out = {k: s[k].double() for k in ("param", "m", "v", "copy", "pack", "pack_bwd")}
    if bits == 8:
        scales = {k: s[k].double() for k in ("m_scale", "v_scale")}
    at_pack = [0, 0]
    for (at, n, t), (kind, rows, cols, _) in zip(spans, tensors):
        sizes = _packed(kind, rows, cols)
        where, at_pack = at_pack, [a + b for a, b in zip(at_pack, sizes)]
        if not active[t]:
            continue
        rate, b1, b2, eps, decay, most = hyper[t]
        end, blocks = at + _up(n, BLOCK), slice(at // BLOCK, (at + _up(n, BLOCK)) // BLOCK)
        g = s["grad"][at:end].double() * (min(1.0, most / (norms[t] + 1e-6)) if c["clip"] else 1.0)
        m, v = out["m"][at:end], out["v"][at:end]
        if bits == 8:
            m = m * scales["m_scale"][blocks].repeat_interleave(BLOCK)
            v = (v * scales["v_scale"][blocks].repeat_interleave(BLOCK)).square()
        m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
        p = out["param"][at:end]
        p -= rate * decay * p + rate * (m / (1 - b1 ** steps[t])) / (torch.sqrt(v / (1 - b2 ** steps[t])) + eps)
        if bits == 8:   # the codes' values before their rounding to 8 bits
            for key, x in (("m", m), ("v", torch.sqrt(v))):
                by = x.view(-1, BLOCK).abs().amax(1) / E4M3_MAX
                scales[key + "_scale"][blocks] = by
                out[key][at:end] = torch.where(by[:, None] > 0, x.view(-1, BLOCK) / by[:, None], 0.0).view(-1)
        else:
            out["m"][at:end], out["v"][at:end] = m, v
        if kind == "plain":
            continue
        w = p[:n].view(rows, cols)
        out["copy"][at:at + n] = p[:n]
        ranks_first = w.T if kind == "A" else w            # [ranks][the other side]
        r, red = ranks_first.shape
        padded = torch.zeros(_up(r, 16), red, dtype=torch.float64, device=w.device)
        padded[:r] = ranks_first
        operand = padded.view(-1, 16, red // 64, 4, 2, 8).permute(0, 2, 4, 3, 1, 5).reshape(-1)
        rows_of = padded[:_up(r, 8)].T.reshape(-1)
        for key, a, b in zip(("pack", "pack_bwd"), where, (operand, rows_of) if kind == "A" else (rows_of, operand)):
            out[key][a:a + b.numel()] = b
    return dict(param=out["param"], m=out["m"], v=out["v"], m_scale=scales and scales["m_scale"],
                v_scale=scales and scales["v_scale"], copy=out["copy"], pack=out["pack"], pack_bwd=out["pack_bwd"],
                steps=torch.tensor(steps), norm=torch.tensor(norms, dtype=torch.float64) if c["clip"] else None)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    return _exact_axes(s) if case["op"] == "axes" else _exact_adamw(s)
