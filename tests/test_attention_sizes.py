"""Sizes that the attention over a paged cache accepts: its limit on a call's steps goes by the rows
that the call has, not by as many for every sequence as the longest may have (checks only; with no
workspace an accepted call ends in LORA_ERR_WORKSPACE before anything touches a device)."""

import ctypes

import pytest

from precision_gemm_amd import _lib

UNSUPPORTED, WORKSPACE = 2, 3
FAKE = ctypes.c_void_p(0x1000)


def call(B, T, max_q, capacity, n_q=32, n_kv=8, D=128, page=16, fmt=0):
    return _lib.lib().lora_tree_attention(FAKE, n_q * D, fmt, FAKE, FAKE, FAKE, FAKE, 1000, page, FAKE, capacity // page, FAKE, FAKE,
                                          B, T, max_q, n_q, n_kv, D, None, 0, 0.1, FAKE, FAKE, None, None, 0, None)


@pytest.mark.parametrize("kw", [
    dict(B=256, T=8447, max_q=8192, capacity=131072),               # a prompt's chunk beside 255 decoding sequences
    dict(B=512, T=65536, max_q=4096, capacity=131072),              # prompts and decoding sequences
    dict(B=4096, T=65536, max_q=65536, capacity=131072, fmt=1),     # a call's most sequences and tokens
    dict(B=4096, T=4096, max_q=1, capacity=1 << 20),                # decode, tables for a million tokens
    dict(B=1024, T=16384, max_q=8192, capacity=1 << 17, n_q=64, n_kv=64, D=64),
    dict(B=1, T=1, max_q=1, capacity=1 << 30),
    dict(B=2, T=65536, max_q=65536, capacity=1 << 20, page=1024),
])
def test_accepted(kw):
    assert call(**kw) == WORKSPACE


@pytest.mark.parametrize("kw", [
    dict(B=4096, T=65536, max_q=8192, capacity=1 << 23),            # as many steps as do not fit 32 bits
    dict(B=4096, T=4096, max_q=1, capacity=1 << 20, n_q=64, n_kv=64),
    dict(B=4096, T=65536, max_q=16, capacity=1 << 24, D=256),
])
def test_refused(kw):
    assert call(**kw) == UNSUPPORTED
    assert call(**dict(kw, capacity=1 << 12)) == WORKSPACE


def test_both_sides_of_the_limit():
    """n_kv N (capacity / 128 + 1) against 5e8, N = min(B ceil(R / 128), T G / 128 + min(B, T))."""
    B, T, max_q = 1000, 30000, 20000
    N = min(B * -(-max_q * 4 // 128), T * 4 / 128 + B)
    most = int((5e8 / (8 * N) - 1) * 128) // 16 * 16
    assert call(B, T, max_q, most) == WORKSPACE and call(B, T, max_q, most + 32) == UNSUPPORTED
