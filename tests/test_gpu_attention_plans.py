"""The attention's ways of cutting work that the smaller cases do not reach: whole prompts with two
workgroups a CU, row blocks in order that are cut without counting what they see, more sequences
than a workgroup has threads; and scales that are not positive.

Tolerances are those of test_gpu_attention.py.  Prompts are compared with the definition in 64 bits
on the device (products of two matrices a head), the rest with the fp64 oracle."""

import numpy as np
import pytest

from test_gpu_attention import U, Batch, _f64

pytestmark = pytest.mark.gpu


def _check_prompts(b, out, lse):
    """Every row against the definition: sequence by sequence, head by head, in 64 bits."""
    import torch
    G, dev = b.n_q // b.n_kv, out.device
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    for s, (n, kv) in enumerate(zip(b.ns, b.kvs)):
        if n == 0:
            continue
        r0 = int(b.indptr[s])
        ids = torch.from_numpy(b.table[s, :-(-kv // b.page)]).to(dev)
        seen = torch.arange(kv, device=dev)[None] <= torch.arange(kv - n, kv, device=dev)[:, None]
        for h in range(b.n_kv):
            k, v = (c[ids, h].double().flatten(0, 1)[:kv].contiguous() for c in (b.k, b.v))
            if b.fp8:
                k, v = k * float(b.sk[h]), v * float(b.sv[h])
            for i in range(h * G, (h + 1) * G):
                q = b.q[r0:r0 + n, i].double().contiguous()
                sc = (q @ k.t().contiguous() * b.scale).masked_fill(~seen, float("-inf"))
                rl = torch.logsumexp(sc, 1)
                p = torch.exp(sc - rl[:, None])
                ref = p @ v
                tol = U * ref.abs() + 2 * U * (p @ v.abs()) + 2.0 ** -133
                off = (out[r0:r0 + n, i].double() - ref).abs() - tol
                assert (off <= 0).all(), (s, i, int(off.flatten().argmax()), float(off.max()))
                spread = ((q.abs() @ k.abs().t().contiguous()) * seen).amax(1) * abs(b.scale)
                off = (lse[r0:r0 + n, i].double() - rl).abs() - 2.0 ** -20 * (spread + rl.abs() + 1)
                assert (off <= 0).all(), ("lse", s, i, float(off.max()))


PROMPTS = [  # ns, kvs, n_q, n_kv, D, page
    # two workgroups a CU, blocks count what they see
    ([4096], [4096], 32, 8, 128, 16),
    ([1024, 700, 0, 1, 333], [1024, 2000, 50, 1500, 333], 32, 8, 128, 64),
    ([1024, 300], [5000, 300], 28, 4, 64, 32),
    ([129] * 40, [129 + 31 * b for b in range(40)], 16, 8, 64, 16),
    # one a CU, heads of 256
    ([600, 77], [600, 1000], 16, 4, 256, 32),
    # all alike: almost every workgroup has a unit of its own (units by the longest sequence)
    ([256] * 8, [256] * 8, 32, 8, 128, 16),
    ([256, 100, 250, 180], [256, 500, 250, 181], 32, 8, 128, 16),
    ([256, 3, 17, 0], [1000, 3, 300, 9], 32, 8, 128, 64),
    ([256] * 8, [256 + 100 * b for b in range(8)], 32, 8, 64, 32),
    ([128, 90, 128, 128], [128, 777, 129, 600], 64, 8, 256, 16),
    ([1000, 900, 31], [1000, 950, 40], 10, 10, 64, 16),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ns,kvs,n_q,n_kv,D,page", PROMPTS)
def test_prompts(ns, kvs, n_q, n_kv, D, page, fp8):
    import torch
    import precision_gemm_amd as P
    print("[case] prompts", ns[:5], kvs[:5], n_q, n_kv, D, page, fp8, flush=True)
    b = Batch(40, ns, kvs, n_q, n_kv, D, page, fp8, "none")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = b.run(status=status)
    assert status.item() == 0
    _check_prompts(b, out, lse)
    again = b.run(workspace=torch.full((96 << 20,), 255, dtype=torch.uint8, device="cuda"))
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,most,n_q,n_kv,D,mask", [
    (700, 5, 16, 2, 64, "none"), (1500, 5, 8, 1, 128, "tree"), (4096, 1, 2, 1, 64, "none"), (600, 40, 4, 1, 64, "none"),
    (520, 20, 2, 1, 256, "any")])
def test_many_sequences(B, most, n_q, n_kv, D, mask, fp8):
    """More sequences than a workgroup has threads, in both kernels; some without tokens."""
    print("[case] many sequences", B, most, n_q, n_kv, D, mask, fp8, flush=True)
    ns = [(7 * b) % (most + 1) if most > 1 else 1 for b in range(B)]
    kvs = [n + (37 * b) % 60 for b, n in enumerate(ns)]
    b = Batch(41, ns, kvs, n_q, n_kv, D, 16, fp8, mask)
    b.check(*b.run())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("most,n_q,D", [(1, 2, 256), (3, 16, 256), (3, 16, 128)])
def test_most_sequences_of_a_call(most, n_q, D, fp8):
    """4,096 sequences, whose prefix sums are kept beside the largest buffers in LDS."""
    print("[case] most sequences", most, n_q, D, fp8, flush=True)
    ns = [1 + b % most for b in range(4096)]
    b = Batch(43, ns, [n + b % 9 for b, n in enumerate(ns)], n_q, 1, D, 16, fp8, "none")
    b.check(*b.run())


SCALED = [  # ns, kvs, n_q, n_kv, D, mask: few rows a kv head, 17 to 32, more; one and two workgroups a CU
    ([1, 1, 1], [1, 300, 129], 8, 2, 128, "none"),
    ([4, 3], [4, 500], 8, 2, 64, "any"),
    ([2, 7], [200, 7], 4, 2, 256, "any"),
    ([5, 8], [333, 8], 16, 4, 128, "any"),
    ([5, 8], [333, 8], 16, 4, 64, "any"),
    ([13, 20], [400, 20], 6, 1, 128, "any"),
    ([40, 1], [45, 300], 15, 3, 256, "any"),
    ([9 + b % 6 for b in range(50)], [15 + 53 * b % 400 for b in range(50)], 16, 8, 64, "any"),
    ([150, 200], [150, 444], 8, 2, 128, "none"),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("scale", [0.0, -0.0, -0.11, -1e-30])
@pytest.mark.parametrize("ns,kvs,n_q,n_kv,D,mask", SCALED)
def test_scales_that_are_not_positive(ns, kvs, n_q, n_kv, D, mask, scale, fp8):
    """A negative scale turns the scores round; a scale of 0 averages the values seen, and a row that
    sees nothing is empty all the same."""
    print("[case] scale", scale, ns[:5], n_q, n_kv, D, mask, fp8, flush=True)
    b = Batch(42, ns, kvs, n_q, n_kv, D, 16, fp8, mask)
    b.scale = scale
    out, lse = b.run()
    b.check(out, lse)
    if mask == "any" and any(n == kv for n, kv in zip(ns, kvs)):  # nothing before the drafted tokens
        assert np.isneginf(_f64(lse)).any()
