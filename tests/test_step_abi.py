"""Refusals of the norms, the AdamW step and the rotation by several axes: statuses of the C ABI
(every call fails its checks before anything touches a device), the plan of a step (a host function),
and the Python bindings' argument errors."""

import ctypes

import numpy as np
import pytest
import torch

import precision_gemm_amd as P
from precision_gemm_amd import _lib
from precision_gemm_amd._lib import AdamWTensorStruct

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


SIZES = [(dict(T=-1), INVALID), (dict(T=70000), UNSUPPORTED), (dict(K=0), INVALID), (dict(K=12), UNSUPPORTED),
         (dict(K=16392), UNSUPPORTED), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(rms=2), INVALID)]


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(x=NULL), INVALID), (dict(x=ODD), INVALID), (dict(ldx=56), INVALID), (dict(ldx=68), INVALID), (dict(res=ODD), INVALID),
    (dict(res=NULL), INVALID), (dict(sum=NULL), INVALID), (dict(ldr=56), INVALID), (dict(lds=60), INVALID), (dict(y=NULL), INVALID),
    (dict(ldy=63), INVALID), (dict(sum=ctypes.c_void_p(0x2000)), INVALID), (dict(w=ODD), INVALID), (dict(b=ODD), INVALID), (dict(T=0, x=NULL), OK)])
def test_layer_norm(L, kw, status):
    base = dict(x=FAKE, ldx=64, res=FAKE, ldr=64, T=3, K=64, w=FAKE, b=FAKE, eps=1e-6, rms=0, y=ctypes.c_void_p(0x2000), ldy=64, sum=FAKE, lds=64,
                stream=NULL)
    assert call(L.lora_layer_norm, "x ldx res ldr T K w b eps rms y ldy sum lds stream", base, **kw) == status


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(), WORKSPACE), (dict(ws=FAKE, wsb=1000), WORKSPACE), (dict(ws=ODD, wsb=1 << 20), WORKSPACE),
    (dict(db=NULL), WORKSPACE), (dict(dw=NULL), WORKSPACE), (dict(dw=ODD), INVALID), (dict(db=ODD), INVALID),
    (dict(dw=ODD, T=0), INVALID), (dict(dy=NULL), INVALID), (dict(h=ODD), INVALID), (dict(dx=NULL), INVALID), (dict(w=ODD), INVALID),
    (dict(dsum=ODD), INVALID), (dict(lddy=60), INVALID), (dict(ldh=8), INVALID), (dict(ldds=8), INVALID), (dict(lddx=70), INVALID),
    (dict(T=0, dw=NULL, db=NULL, K=12), UNSUPPORTED)])
def test_layer_norm_backward(L, kw, status):
    base = dict(dy=FAKE, lddy=64, h=FAKE, ldh=64, w=FAKE, dsum=FAKE, ldds=64, T=3, K=64, eps=1e-6, rms=0, dx=FAKE, lddx=64, dw=FAKE,
                db=FAKE, ws=NULL, wsb=0, stream=NULL)
    names = "dy lddy h ldh w dsum ldds T K eps rms dx lddx dw db ws wsb stream"
    assert call(L.lora_layer_norm_backward, names, base, **kw) == status


def test_norm_workspace_bytes(L):
    f = L.lora_layer_norm_backward_workspace_bytes
    assert f(1, 64) >= 2 * 64 * 4 and f(65536, 16384) > 0
    assert f(0, 64) == 0 and f(5, 12) == 0 and f(70000, 64) == 0 and f(5, 16392) == 0


# ---- the plan of an AdamW step ----

def tensor(rows, cols, kind, group=0, bits=32, at=None, **kw):
    """A tensor whose buffers lie one behind another from ``at`` on."""
    at = [at if at is not None else 1 << 20]

    def take(n):
        p = at[0]
        at[0] += -(-n // 16) * 16
        return p

    v = rows * cols
    s = AdamWTensorStruct(take(4 * v), take(4 * v), take(bits // 8 * v), take(bits // 8 * v), rows=rows, cols=cols, group=group, kind=kind)
    if bits == 8:
        s.m_scale, s.v_scale = take(-(-v // 64) * 4), take(-(-v // 64) * 4)
    if kind:
        s.copy, s.pack, s.pack_bwd = take(2 * v), take(0), None
        r, side = (cols, rows) if kind == 1 else (rows, cols)
        a, b = -(-r // 16) * 32 * side, -(-r // 8) * 16 * side
        s.pack = take(a if kind == 1 else b)
        s.pack_bwd = take(b if kind == 1 else a)
    for k, x in kw.items():
        setattr(s, k, x)
    s.end = at[0]
    return s


class Tile(ctypes.Structure):
    _fields_ = [("tensor", AdamWTensorStruct), ("first", ctypes.c_int32), ("reserved", ctypes.c_int32)]


def plan(L, tensors, n_groups=2, bits=32, want=True):
    a = (AdamWTensorStruct * max(1, len(tensors)))(*tensors)
    n = ctypes.c_int64(-5)
    st = L.lora_adamw_plan(a, len(tensors), n_groups, bits, ctypes.byref(n), None, None)
    if st != OK or not want:
        return st, n.value, None, None
    tiles, first = (Tile * n.value)(), np.full(n_groups + 1, -1, np.int32)
    st = L.lora_adamw_plan(a, len(tensors), n_groups, bits, ctypes.byref(n), tiles, first.ctypes.data)
    return st, n.value, tiles, first


def test_plan_covers_every_value_once(L):
    ts, at = [], 1 << 20
    for rows, cols, kind, group in ((128, 8, 1, 1), (5, 640, 2, 0), (1, 10000, 0, 1), (4096, 1, 1, 0), (64, 64, 1, 0), (1, 1, 0, 2),
                                    (64, 192, 2, 1), (33, 128, 2, 0), (640, 7, 1, 1)):
        ts.append(tensor(rows, cols, kind, group, at=at))
        at = ts[-1].end
    st, n, tiles, first = plan(L, ts, n_groups=4)
    assert st == OK and n == len(tiles) == first[4] and first[0] == 0 and first[3] == first[4]
    for g in range(4):
        for x in tiles[first[g]:first[g + 1]]:
            assert x.tensor.group == g
    for t in ts:
        mine = [x for x in tiles if x.tensor.param == t.param]
        assert all(bytes(x.tensor) == bytes(t) for x in mine)
        starts = sorted(x.first for x in mine)
        side = t.rows if t.kind == 1 else t.cols if t.kind == 2 else t.rows * t.cols
        r = t.cols if t.kind == 1 else t.rows
        span = 4096 if t.kind == 0 else 512 if r <= 4 else 256 if r <= 16 else 128 if r <= 32 else 64
        assert starts == list(range(0, side, span))


@pytest.mark.parametrize("kind,bits", [(0, 32), (1, 32), (2, 8)])
@pytest.mark.parametrize("kw,status", [
    (dict(param=None), INVALID), (dict(grad=None), INVALID), (dict(m=None), INVALID), (dict(v=0x1008), INVALID),
    (dict(grad=0x1004), INVALID), (dict(copy=0x1002), INVALID), (dict(group=2), INVALID), (dict(group=-1), INVALID), (dict(rows=0), INVALID),
    (dict(cols=-1), INVALID), (dict(kind=3), INVALID), (dict(rows=1 << 16, cols=1 << 16), UNSUPPORTED)])
def test_plan_refuses(L, kind, bits, kw, status):
    t = tensor(64, 64, kind, bits=bits)
    for k, x in kw.items():
        setattr(t, k, x)
    if kind == 0 or kw.get("kind") == 3 or status == UNSUPPORTED:
        t.pack = t.pack_bwd = None
    assert plan(L, [t], bits=bits)[0] == status


def test_plan_refuses_more(L):
    assert plan(L, [tensor(64, 65, 1)])[0] == UNSUPPORTED and plan(L, [tensor(60, 8, 1)])[0] == UNSUPPORTED
    assert plan(L, [tensor(65, 64, 2)])[0] == UNSUPPORTED and plan(L, [tensor(8, 96, 2)])[0] == UNSUPPORTED
    assert plan(L, [tensor(1, 64, 0, pack=0x9000)])[0] == INVALID
    assert plan(L, [tensor(1, 64, 0, m_scale=0x9000)])[0] == INVALID          # scales are for 8 bits
    assert plan(L, [tensor(1, 64, 0, bits=8, v_scale=None)], bits=8)[0] == INVALID
    assert plan(L, [tensor(1, 64, 0)], bits=16)[0] == INVALID and plan(L, [tensor(1, 64, 0)], n_groups=0)[0] == INVALID
    assert plan(L, [tensor(1, 64, 0)], n_groups=9000)[0] == UNSUPPORTED
    n = ctypes.c_int64(0)
    assert L.lora_adamw_plan(None, 1, 1, 32, ctypes.byref(n), None, None) == INVALID
    assert L.lora_adamw_plan(None, 0, 1, 32, ctypes.byref(n), None, None) == OK and n.value == 0
    a, tiles, first = (AdamWTensorStruct * 1)(tensor(1, 64, 0)), (Tile * 9)(), np.zeros(2, np.int32)
    n.value = 9  # not the number of tiles
    assert L.lora_adamw_plan(a, 1, 1, 32, ctypes.byref(n), tiles, first.ctypes.data) == INVALID
    n.value = 1
    assert L.lora_adamw_plan(a, 1, 1, 32, ctypes.byref(n), tiles, None) == INVALID


def test_plan_refuses_overlaps(L):
    """A buffer that a step writes is nobody else's; gradients may be shared."""
    a = tensor(64, 16, 1)
    b = tensor(64, 16, 1, group=1, at=a.end)
    assert plan(L, [a, b])[0] == OK
    assert plan(L, [a, a])[0] == INVALID
    for field in ("param", "m", "v", "copy", "pack", "pack_bwd"):
        c = tensor(64, 16, 1, group=1, at=a.end)
        setattr(c, field, getattr(a, field) + 16)
        assert plan(L, [a, c])[0] == INVALID, field
        c = tensor(64, 16, 1, group=1, at=a.end)
        setattr(c, field, a.grad)
        assert plan(L, [a, c])[0] == INVALID, field
    c = tensor(64, 16, 1, group=1, at=a.end, grad=a.grad)
    assert plan(L, [a, c])[0] == OK


@pytest.mark.parametrize("kw,status", [
    (dict(), WORKSPACE), (dict(ws=ODD, wsb=1 << 20), WORKSPACE), (dict(ws=FAKE, wsb=64), WORKSPACE), (dict(n=-1), INVALID),
    (dict(n=1 << 31), UNSUPPORTED), (dict(n=1 << 22), UNSUPPORTED), (dict(n=(1 << 22) - 1), WORKSPACE), (dict(G=0), INVALID),
    (dict(G=9000), UNSUPPORTED), (dict(bits=16), INVALID),
    (dict(tiles=NULL), INVALID), (dict(first=NULL), INVALID), (dict(hyper=NULL), INVALID), (dict(hyper=ctypes.c_void_p(0x1004)), INVALID),
    (dict(steps=NULL), INVALID), (dict(active=ctypes.c_void_p(0x1002)), INVALID), (dict(norm=ctypes.c_void_p(0x1002)), INVALID)])
def test_step(L, kw, status):
    base = dict(tiles=FAKE, n=5, first=FAKE, G=2, bits=32, hyper=FAKE, active=FAKE, steps=FAKE, norm=FAKE, st=NULL, ws=NULL,
                wsb=0, stream=NULL)
    assert call(L.lora_adamw_step, "tiles n first G bits hyper active steps norm st ws wsb stream", base, **kw) == status


def test_step_workspace_bytes(L):
    f = L.lora_adamw_workspace_bytes
    assert f(0, 1) > 0 and f(1000, 3) >= 8000 and f(-1, 1) == 0 and f(5, 0) == 0 and f(1 << 31, 1) == 0 and f(5, 9000) == 0
    assert f((1 << 22) - 1, 1) > 0 and f(1 << 22, 1) == 0


def test_plan_refuses_more_tiles_than_a_launch_has(L):
    """4,194,304 tiles of 1,024 threads are 2^32 threads: no launch has as many."""
    n = 8200
    ts = [tensor(1, 2 ** 21, 0, at=(i + 1) << 32) for i in range(n)]  # 512 tiles each
    assert plan(L, ts, want=False)[0] == UNSUPPORTED
    st, count, _, _ = plan(L, ts[:8191], want=False)
    assert st == OK and count == 8191 * 512


# ---- positions of several axes ----

AXES = ctypes.create_string_buffer(bytes([0, 1, 2, 1] * 8), 32)
ROPE = dict(qkv=FAKE, ld=768, pos=FAKE, n=3, axes=AXES, T=3, n_q=8, n_kv=2, D=64, cs=FAKE, mp=10, rot=64, inter=0, qw=FAKE, kw=FAKE,
            eps=1e-6, q=FAKE, ldq=512, st=NULL, stream=NULL)
COMMON = [(dict(n=0), INVALID), (dict(n=-1), INVALID), (dict(n=5), UNSUPPORTED), (dict(n=2), INVALID), (dict(axes=NULL), INVALID),
          (dict(pos=NULL), INVALID), (dict(rot=80), INVALID), (dict(rot=24), UNSUPPORTED), (dict(D=96), UNSUPPORTED), (dict(mp=0), INVALID),
          (dict(qkv=NULL), INVALID), (dict(ld=760), INVALID), (dict(T=-1), INVALID), (dict(T=70000), UNSUPPORTED)]


@pytest.mark.parametrize("kw,status", COMMON + [(dict(k=NULL), INVALID), (dict(T=0, qkv=NULL), OK)])
def test_norm_rope_axes(L, kw, status):
    base = dict(ROPE, k=FAKE, ldk=128)
    names = "qkv ld pos n axes T n_q n_kv D cs mp rot inter qw kw eps q ldq k ldk st stream"
    assert call(L.lora_qk_norm_rope_axes, names, base, **kw) == status


@pytest.mark.parametrize("kw,status", COMMON + [(dict(slots=NULL), INVALID), (dict(fmt=2), INVALID), (dict(page=48), UNSUPPORTED)])
def test_append_axes(L, kw, status):
    base = dict(ROPE, slots=FAKE, fmt=0, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, n_pages=4, page=16)
    names = "qkv ld pos n axes slots T n_q n_kv D cs mp rot inter qw kw eps q ldq fmt kc vc ks vs n_pages page st stream"
    assert call(L.lora_rope_axes_append_kv, names, base, **kw) == status


@pytest.mark.parametrize("kw,status", COMMON + [(dict(), WORKSPACE), (dict(dq=NULL), INVALID), (dict(dqw=NULL), INVALID)])
def test_backward_axes(L, kw, status):
    base = dict(ROPE, dq=FAKE, dk=FAKE, dv=FAKE, out=FAKE, ldd=768, dqw=FAKE, dkw=FAKE, ws=NULL, wsb=0)
    names = "qkv ld pos n axes dq dk dv T n_q n_kv D cs mp rot inter qw kw eps out ldd dqw dkw st ws wsb stream"
    assert call(L.lora_qk_norm_rope_axes_backward, names, base, **kw) == status


def test_pair_axes():
    assert P.rope_pair_axes((2, 1, 3)) == bytes([0, 0, 1, 2, 2, 2])
    assert P.rope_pair_axes((2, 1, 3), interleaved=True) == bytes([0, 1, 2, 0, 2, 2])
    assert P.rope_pair_axes((0, 2)) == bytes([1, 1])
    for bad in ((), (1, 1, 1, 1, 1), (-1, 2)):
        with pytest.raises(ValueError, match="sections"):
            P.rope_pair_axes(bad)


def test_python_refusals():
    """Tensors on the host, of another type or shape are refused by name."""
    x = torch.zeros((3, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x must be a device tensor"):
        P.layer_norm(x)
    with pytest.raises(ValueError, match="x must have dtype"):
        P.layer_norm(x.float())
    with pytest.raises(ValueError, match="channels"):
        P.layer_norm(x[0])
    with pytest.raises(ValueError, match="dy must be a device tensor"):
        P.layer_norm_backward(x, x)
    with pytest.raises(ValueError, match="h must be a tensor"):
        P.layer_norm_backward(x, None)
    w = torch.zeros(64)
    for bits in (16, None):
        with pytest.raises(ValueError, match="state_bits"):
            P.AdamW([P.AdamWTensor(w, w)], 1, state_bits=bits)
    with pytest.raises(ValueError, match="param must be a device tensor"):
        P.AdamW([P.AdamWTensor(w, w)], 1)
    with pytest.raises(ValueError, match="at least"):
        P.AdamW([], 1)
