"""Refusals of the attention block: statuses of the C ABI (every call fails its checks before
anything touches a device) and the Python binding's argument errors."""

import ctypes

import pytest
import torch

import precision_gemm_amd as P
from precision_gemm_amd import _lib

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
NULL, FAKE, ODD = None, ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008)


@pytest.fixture(scope="module")
def L():
    return _lib.lib()


def call(f, names, base, **kw):
    a = dict(base)
    assert set(kw) <= set(a), set(kw) - set(a)
    a.update(kw)
    return f(*[a[n] for n in names.split()])


ROPE = dict(qkv=FAKE, ld=768, pos=FAKE, T=3, n_q=8, n_kv=2, D=64, cs=FAKE, mp=10, rot=64, inter=0, qw=FAKE, kw=FAKE, eps=1e-6,
            q=FAKE, ldq=512, k=FAKE, ldk=128, st=NULL, stream=NULL)
ROPE_NAMES = "qkv ld pos T n_q n_kv D cs mp rot inter qw kw eps q ldq k ldk st stream"
COMMON = [  # wrong argument, status: what the rotation's calls share
    (dict(T=-1), INVALID), (dict(T=70000), UNSUPPORTED), (dict(n_q=0), INVALID), (dict(n_kv=2000), UNSUPPORTED),
    (dict(D=96), UNSUPPORTED), (dict(D=0), INVALID), (dict(rot=-16), INVALID), (dict(rot=80), INVALID),
    (dict(rot=24), UNSUPPORTED), (dict(inter=2), INVALID), (dict(pos=NULL), INVALID), (dict(cs=NULL), INVALID),
    (dict(cs=ODD), INVALID), (dict(mp=0), INVALID), (dict(qw=NULL), INVALID), (dict(kw=ODD), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(qkv=NULL), INVALID), (dict(qkv=ODD), INVALID),
    (dict(ld=760), INVALID), (dict(ld=772), INVALID),
]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(q=NULL), INVALID), (dict(k=ODD), INVALID), (dict(ldq=504), INVALID), (dict(ldk=132), INVALID), (dict(T=0, qkv=NULL), OK)])
def test_norm_rope(L, kw, status):
    assert call(L.lora_qk_norm_rope, ROPE_NAMES, ROPE, **kw) == status


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(slots=NULL), INVALID), (dict(fmt=2), INVALID), (dict(kc=NULL), INVALID), (dict(vc=ODD), INVALID),
    (dict(fmt=1, ks=NULL), INVALID), (dict(fmt=1, vs=NULL), INVALID), (dict(n_pages=0), INVALID), (dict(page=8), UNSUPPORTED),
    (dict(page=48), UNSUPPORTED), (dict(page=2048), UNSUPPORTED), (dict(n_pages=2 ** 30), UNSUPPORTED), (dict(q=NULL), INVALID),
    (dict(T=0, slots=NULL), OK)])
def test_append(L, kw, status):
    base = dict(ROPE, slots=FAKE, fmt=0, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, n_pages=4, page=16)
    names = "qkv ld pos slots T n_q n_kv D cs mp rot inter qw kw eps q ldq fmt kc vc ks vs n_pages page st stream"
    assert call(L.lora_rope_append_kv, names, base, **kw) == status


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(dq=NULL), INVALID), (dict(dk=ODD), INVALID), (dict(dv=ODD), INVALID), (dict(out=NULL), INVALID), (dict(ldd=100), INVALID),
    (dict(dqw=NULL), INVALID), (dict(dkw=ODD), INVALID), (dict(), WORKSPACE), (dict(ws=FAKE, wsb=1000), WORKSPACE),
    (dict(ws=ODD, wsb=1 << 20), WORKSPACE)])
def test_backward(L, kw, status):
    base = dict(ROPE, dq=FAKE, dk=FAKE, dv=FAKE, out=FAKE, ldd=768, dqw=FAKE, dkw=FAKE, ws=NULL, wsb=0)
    names = "qkv ld pos dq dk dv T n_q n_kv D cs mp rot inter qw kw eps out ldd dqw dkw st ws wsb stream"
    assert call(L.lora_qk_norm_rope_backward, names, base, **kw) == status


def test_backward_workspace_bytes(L):
    f = L.lora_qk_norm_rope_backward_workspace_bytes
    assert f(1, 64) == 768 * 256 and f(65536, 256) == 768 * 1024 and f(0, 64) == 0 and f(5, 96) == 0 and f(70000, 64) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(), WORKSPACE), (dict(ws=FAKE, wsb=1000), WORKSPACE), (dict(ws=ODD, wsb=1 << 30), WORKSPACE),
    (dict(T=-1), INVALID), (dict(T=70000), UNSUPPORTED), (dict(D=192), UNSUPPORTED), (dict(n_q=7), INVALID), (dict(fmt=3), INVALID),
    (dict(fmt=1, ks=NULL), INVALID), (dict(n_pages=0), INVALID), (dict(page=24), UNSUPPORTED), (dict(B=-1), INVALID),
    (dict(B=5000), UNSUPPORTED), (dict(max_q=-1), INVALID), (dict(max_q=65), UNSUPPORTED), (dict(words=17), UNSUPPORTED),
    (dict(words=0), INVALID), (dict(mask=NULL, words=0, max_q=65), WORKSPACE), (dict(scale=float("inf")), INVALID),
    (dict(q=NULL), INVALID), (dict(q=ODD), INVALID), (dict(ldq=500), INVALID), (dict(table=NULL), INVALID), (dict(mp=0), INVALID),
    (dict(mp=-1), INVALID), (dict(mp=2 ** 29), UNSUPPORTED), (dict(kv=NULL), INVALID), (dict(ip=NULL), INVALID),
    (dict(out=NULL), INVALID), (dict(out=ODD), INVALID), (dict(lse=NULL), WORKSPACE), (dict(kc=NULL), INVALID), (dict(vc=ODD), INVALID),
    (dict(B=4096, mp=2 ** 26, n_q=1024, n_kv=1024, ldq=65536), UNSUPPORTED), (dict(T=0, q=NULL), OK), (dict(B=0), OK), (dict(max_q=0), OK)])
def test_attention(L, kw, status):
    base = dict(q=FAKE, ldq=512, fmt=0, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, n_pages=4, page=16, table=FAKE, mp=3, kv=FAKE, ip=FAKE,
                B=2, T=5, max_q=4, n_q=8, n_kv=2, D=64, mask=FAKE, words=1, scale=0.1, out=FAKE, lse=FAKE, st=NULL, ws=NULL,
                wsb=0, stream=NULL)
    names = "q ldq fmt kc vc ks vs n_pages page table mp kv ip B T max_q n_q n_kv D mask words scale out lse st ws wsb stream"
    assert call(L.lora_tree_attention, names, base, **kw) == status


def test_attention_workspace_bytes(L):
    f = L.lora_tree_attention_workspace_bytes
    assert 0 < f(32, 8, 128, 1) < 96 << 20 and 0 < f(8, 8, 256, 65536) < 96 << 20
    assert f(7, 2, 64, 1) == 0 and f(8, 2, 80, 1) == 0 and f(8, 2, 64, 0) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(parents=NULL), INVALID), (dict(ip=NULL), INVALID), (dict(mask=NULL), INVALID), (dict(words=0), INVALID),
    (dict(words=17), UNSUPPORTED), (dict(max_q=65), UNSUPPORTED), (dict(B=0), INVALID), (dict(B=5000), UNSUPPORTED), (dict(T=0), OK),
    (dict(T=-1), INVALID)])
def test_mask(L, kw, status):
    base = dict(parents=FAKE, ip=FAKE, B=2, T=5, max_q=4, words=1, mask=FAKE, st=NULL, stream=NULL)
    assert call(L.lora_tree_mask, "parents ip B T max_q words mask st stream", base, **kw) == status


def test_python_refusals():
    """Tensors on the host, of another type or shape are refused by name."""
    x = torch.zeros((3, 768), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="qkv must be a device tensor"):
        P.qk_norm_rope(x, None, 8, 2, 64)
    with pytest.raises(ValueError, match="qkv must have dtype"):
        P.qk_norm_rope(x.float(), None, 8, 2, 64)
    with pytest.raises(ValueError, match="k_cache"):
        P.rope_append_kv(x, None, None, x, x, 8)
    with pytest.raises(ValueError, match="dq must be a device tensor"):
        P.qk_norm_rope_backward(x, None, x.view(3, 12, 64)[:, :8], x.view(3, 12, 64)[:, :2], None)
    with pytest.raises(ValueError, match="parents must be a device tensor"):
        P.tree_mask(torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 3)
    c = torch.zeros((2, 2, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="8-bit cache"):
        P.tree_attention(x.view(3, 12, 64), c, c, None, None, None, 1, k_scale=x)
    with pytest.raises(ValueError, match="v_cache must have dtype"):
        P.tree_attention(x.view(3, 12, 64), c, c.float(), None, None, None, 1)
    with pytest.raises(ValueError, match="heads of 128"):
        P.tree_attention(torch.zeros((3, 6, 128), dtype=torch.bfloat16), c, c, None, None, None, 1)


def test_rope_table():
    t = P.rope_table(5, 8, 100.0, device="cpu").double()
    a = torch.arange(5, dtype=torch.float64)[:, None] * 100.0 ** (-torch.arange(4, dtype=torch.float64) / 4)
    assert t.shape == (5, 8) and (t - torch.cat([a.cos(), a.sin()], 1)).abs().max() <= 2.0 ** -24
