"""The attention block at its edges: rows that no sequence has, offsets that are not in order, and the
plans and scales that the ordinary cases do not reach.  Tolerances are those of test_gpu_attention.py
(its ``Batch`` builds the inputs and holds the outputs to the fp64 oracle)."""

import numpy as np
import pytest

from test_gpu_attention import Batch, _i32

pytestmark = pytest.mark.gpu


def _marked(b):
    """Buffers for a batch's outputs whose every value shows whether it was written."""
    import torch
    return torch.full((b.T, b.n_q, b.D), 3.0, dtype=torch.bfloat16, device="cuda"), torch.full((b.T, b.n_q), 5.0, device="cuda")


def _pad(b, before, after):
    """A batch's rows with others before and behind that no sequence has."""
    import torch
    extra = lambda n: torch.full((n, b.n_q, b.D), 1.5, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    b.q = torch.cat([extra(before), b.q, extra(after)])
    b.T += before + after
    b.indptr = b.indptr + before
    b.masks = None  # of the rows before the padding; the caller pads its tensor
    return b


# few rows a kv head, and many (the kernel whose waves share the keys), one and two workgroups a CU
EDGES = [  # ns, kvs, n_q, n_kv, D, page, mask
    ([1, 1, 1], [100, 16, 17], 8, 2, 128, 16, "none"),
    ([3, 0, 2], [900, 5, 40], 4, 4, 64, 32, "tree"),
    ([2, 1], [70, 300], 8, 2, 256, 16, "none"),
    ([16, 9], [777, 16], 32, 8, 128, 16, "tree"),
    ([40, 3], [45, 300], 15, 3, 256, 16, "any"),
    ([200, 30], [250, 300], 8, 2, 64, 64, "none"),
    ([12] * 64, [50 + 7 * b % 100 for b in range(64)], 16, 8, 64, 16, "none"),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("before,after", [(0, 5), (3, 0), (700, 1100)])
@pytest.mark.parametrize("ns,kvs,n_q,n_kv,D,page,mask", EDGES)
def test_rows_of_no_sequence(ns, kvs, n_q, n_kv, D, page, mask, before, after, fp8):
    """A batch padded before its first sequence and behind its last: the padding is 0 and -inf and
    reported, the rest as without it."""
    import torch
    import precision_gemm_amd as P
    print("[case] rows of no sequence", ns[:5], n_q, n_kv, D, before, after, fp8, flush=True)
    b = Batch(30, ns, kvs, n_q, n_kv, D, page, fp8, mask)
    clean, T, tm = b.run(), b.T, b.mask_tensor()
    b = _pad(b, before, after)
    if tm is not None:  # masks of the padding name keys; nobody reads them
        tm = torch.cat([tm.new_full((before, tm.shape[1]), -1), tm, tm.new_full((after, tm.shape[1]), -1)])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = _marked(b)
    b.run(out=out, lse=lse, status=status, tree_mask=tm)
    assert status.item() == P.LORA_ATTN_BAD_LENGTH
    assert torch.equal(out[before:before + T], clean[0]) and torch.equal(lse[before:before + T], clean[1])
    for rows in (slice(0, before), slice(before + T, None)):
        assert not out[rows].any() and (lse[rows] == float("-inf")).all()


@pytest.mark.parametrize("ns,kvs,n_q,n_kv,D,mask,indptrs", [
    ([1, 2, 1, 1], [100, 50, 20, 64], 4, 2, 128, "none",
     ([0, 1, 3, 4, 9], [0, 1, 0, 4, 5], [-2, 1, 3, 4, 5], [0, 1, 4, 4, 5], [3, 1, 3, 4, 5], [0, 1, 3, 4, 2], [9, 9, 9, 9, 9],
      [5, 4, 3, 2, 1], [0, 0, 0, 0, 0])),
    ([30, 41, 30], [150, 60, 800], 16, 2, 64, "tree",
     ([0, 30, 71, 120], [0, 30, 0, 101], [-1, 30, 71, 101], [0, 72, 71, 101], [71, 30, 71, 101], [0, 30, 101, 101])),
    ([30, 41, 30], [150, 60, 800], 6, 1, 256, "any", ([0, 30, 71, 120], [0, 30, 0, 101], [101, 71, 30, 0])),
])
def test_rows_of_sequences_left_out(ns, kvs, n_q, n_kv, D, mask, indptrs):
    """Offsets that leave the call, descend, or hold more tokens than max_q: every row that no
    sequence in order has is 0 and -inf, those whose sequence is as it was are too."""
    import torch
    import precision_gemm_amd as P
    b = Batch(31, ns, kvs, n_q, n_kv, D, 16, False, mask)
    clean, keep = b.run(), b.indptr
    for indptr in indptrs:
        print("[case] sequences left out", ns, n_q, D, indptr, flush=True)
        b.indptr = np.array(indptr)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = _marked(b)
        b.run(out=out, lse=lse, status=status)
        assert status.item() == P.LORA_ATTN_BAD_LENGTH
        owners = [[] for _ in range(b.T)]
        for s, (lo, hi) in enumerate(zip(indptr[:-1], indptr[1:])):
            if 0 <= lo <= hi <= b.T and hi - lo <= max(ns):
                for t in range(lo, hi):
                    owners[t].append((s, lo, hi))
        for t, own in enumerate(owners):
            if not own:
                assert not out[t].any() and (lse[t] == float("-inf")).all(), t
            elif len(own) == 1 and own[0][1:] == tuple(keep[own[0][0]:own[0][0] + 2]):
                assert torch.equal(out[t], clean[0][t]) and torch.equal(lse[t], clean[1][t]), t
        b.indptr = keep


def test_no_sequences_and_no_tokens_allowed():
    """No sequences, or none with tokens, for rows there are: all rows are 0 and -inf."""
    import torch
    import precision_gemm_amd as P
    print("[case] no sequences", flush=True)
    b = Batch(32, [2, 1], [40, 9], 4, 2, 64, 16, False)
    for table, kvs, indptr, max_q in ((np.zeros((0, 3)), [], [0], 4), (b.table, b.kvs, b.indptr, 0), (b.table, b.kvs, [0, 0, 0], 0)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = _marked(b)
        got = P.tree_attention(b.q, b.k, b.v, _i32(table), _i32(kvs), _i32(indptr), max_q, out=out, lse=lse, status=status)
        assert got[0] is out and not out.any() and (lse == float("-inf")).all()
        assert status.item() == P.LORA_ATTN_BAD_LENGTH


@pytest.mark.parametrize("fp8", [False, True])
def test_prompt_chunk_beside_decoding_sequences(fp8):
    """A chunk of a prompt among 255 decoding sequences, with page tables for 131,072 tokens and room
    for chunks of 8,192."""
    import torch
    import precision_gemm_amd as P
    print("[case] chunk beside decoding sequences", fp8, flush=True)
    ns, kvs = [1] * 256, [1 + 13 * b % 300 for b in range(256)]
    ns[100], kvs[100] = 300, 700
    b = Batch(33, ns, kvs, 32, 8, 64, 16, fp8, "none")
    table = np.zeros((256, 8192), np.int64)
    table[:, :b.table.shape[1]] = b.table
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    sc = [None if s is None else torch.from_numpy(s).cuda() for s in (b.sk, b.sv)]
    out, lse = P.tree_attention(b.q, b.k, b.v, _i32(table), _i32(kvs), _i32(b.indptr), 8192, scale=b.scale, k_scale=sc[0],
                                v_scale=sc[1], status=status)
    assert status.item() == 0
    b.check(out, lse)


@pytest.mark.parametrize("n_q,D,mask", [(4, 64, "none"), (4, 256, "none"), (64, 128, "none"), (32, 64, "tree")])
def test_offsets_that_overlap(n_q, D, mask):
    """Offsets that give the call's rows to several sequences, more rows than it has in all: every
    sequence is left out."""
    import torch
    import precision_gemm_amd as P
    print("[case] offsets that overlap", n_q, D, mask, flush=True)
    ns, kvs = [1] * 40, [30] * 40
    b = Batch(34, ns, kvs, n_q, 2, D, 16, False)
    tm = torch.ones((40, 1), dtype=torch.int64, device="cuda") if mask == "tree" else None
    for indptr in ([0, 40] * 20 + [0], [0, 21, 0, 20] + [40] * 37):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = _marked(b)
        P.tree_attention(b.q, b.k, b.v, _i32(b.table), _i32([100] * 40), _i32(indptr), 40, tree_mask=tm, out=out, lse=lse, status=status)
        assert status.item() == P.LORA_ATTN_BAD_LENGTH
        assert not out.any() and (lse == float("-inf")).all()


@pytest.mark.parametrize("indptr", [[4, 2, 6], [0, 6, 3], [0, 3, 0, 6], [5, 5, 2, 4, 1], [-3, 2, -1, 4], [600, 300, 900, 100]])
def test_masks_of_offsets_that_descend(indptr):
    """Rows of a sequence that fits keep their masks when another's offsets run over them; rows that
    no sequence has are 0."""
    import torch
    import precision_gemm_amd as P
    from oracle import attention as A
    print("[case] masks, offsets that descend", indptr, flush=True)
    T = 1000 if max(indptr) > 6 else 6
    max_q = 4 if T == 6 else 600
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want, several = [0] * T, [0] * T
    for lo, hi in zip(indptr[:-1], indptr[1:]):
        if 0 <= lo <= hi <= T and hi - lo <= max_q:
            want[lo:hi] = A.tree_mask(list(range(-1, hi - lo - 1)), [0, hi - lo])
            for t in range(lo, hi):
                several[t] += 1
    assert max(several) <= 1
    # every token the child of the one before in its own sequence (of the ones that fit)
    parents = [max(0, w.bit_length() - 1) - 1 for w in want]
    m = P.tree_mask(_i32(parents), _i32(indptr), max_q, status=status).cpu().numpy().view(np.uint64)
    assert status.item() == P.LORA_ATTN_BAD_LENGTH
    assert [sum(int(w) << 64 * i for i, w in enumerate(row)) for row in m] == want
