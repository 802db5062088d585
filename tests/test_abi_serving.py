"""Argument checks of the serving-step entry points, without a GPU."""
import ctypes

import pytest
import torch

from progressive_kv_quantization_gb300 import lynx as L


@pytest.fixture
def a(lynx_lib):
    buf = ctypes.create_string_buffer(64)
    p = ctypes.c_void_p((ctypes.addressof(buf) + 15) & ~15)
    p.buf = buf
    return p


def test_assign_pages_argument_checks(lynx_lib, a):
    b = ctypes.c_void_p(a.value + 8)

    def call(ctx=a, new=a, B=1, Hkv=1, table=a, mp=1, free=a, nf=1, rows=1, cu=a, pos=a, slots=a, out=b, taken=a):
        return lynx_lib.lynx_assign_pages(ctx, new, B, Hkv, table, mp, free, nf, rows, cu, pos, slots, out, taken, None)
    for kw in (dict(B=0), dict(Hkv=0), dict(mp=0), dict(nf=-1), dict(rows=-1), dict(ctx=None), dict(new=None),
               dict(table=None), dict(free=None), dict(cu=None), dict(pos=None), dict(slots=None), dict(out=None),
               dict(taken=None), dict(out=a)):
        assert call(**kw) == -1, kw
    assert call(mp=1 << 23) == -2 and call(rows=(1 << 30) + 1) == -2 and call(nf=(1 << 30) + 1) == -2 and call(Hkv=1 << 24) == -2
    for name in ("ctx", "new", "table", "free", "cu", "pos", "out", "taken"):
        assert call(**{name: ctypes.c_void_p(a.value + 2)}) == -3, name
    assert call(slots=ctypes.c_void_p(a.value + 4)) == -3


def test_qkv_append_argument_checks(lynx_lib, a):
    def call(qkv=a, n=1, stride=384, Hq=1, Hkv=1, D=128, wq=None, wk=None, eps=1e-6, cs=a, mp=4, rot=128, il=0, pos=a,
             slots=a, q=a, k=a, v=a, pool=1):
        return lynx_lib.lynx_qkv_append(qkv, n, stride, Hq, Hkv, D, wq, wk, eps, cs, mp, rot, il, pos, slots, q, k, v,
                                        pool, None)
    for kw in (dict(n=-1), dict(Hq=0), dict(Hkv=0), dict(stride=383), dict(il=2), dict(pool=0), dict(cs=None),
               dict(mp=0), dict(qkv=None), dict(pos=None), dict(slots=None), dict(q=None), dict(k=None), dict(v=None)):
        assert call(**kw) == -1, kw
    for kw in (dict(D=64), dict(rot=8), dict(rot=144), dict(rot=-16), dict(wq=a, eps=-1.0), dict(wk=a, eps=float("nan")),
               dict(Hq=65535, stride=1 << 24)):
        assert call(**kw) == -2, kw
    for name in ("qkv", "cs", "q", "k", "v"):
        assert call(**{name: ctypes.c_void_p(a.value + 8)}) == -3, name
    assert call(stride=388) == -3
    assert call(pos=ctypes.c_void_p(a.value + 2)) == -3 and call(slots=ctypes.c_void_p(a.value + 4)) == -3
    assert call(n=0, qkv=None, pos=None, slots=None, q=None, k=None, v=None, cs=None) == 0


def test_qkv_append_refuses_norm_weights_off_16_bytes(lynx_lib, a):
    """A slice of a longer weight vector: the kernel reads four weights at once."""
    def call(wq, wk):
        return lynx_lib.lynx_qkv_append(a, 1, 384, 1, 1, 128, wq, wk, 1e-6, a, 4, 128, 0, a, a, a, a, a, 1, None)
    for off in (4, 8, 12):
        w = ctypes.c_void_p(a.value + off)
        assert call(w, None) == -3 and call(None, w) == -3


def test_chunk_attn_argument_checks(lynx_lib, a):
    size = lynx_lib.lynx_chunk_attn_workspace_size(1, 1, 4, 2, 128)

    def call(q=a, n=1, stride=512, cu=a, B=1, Hq=4, Hkv=2, D=128, k=a, v=a, pool=1, table=a, mp=1, ctx=a, scale=0.1,
             causal=1, out=a, dt=0, lse=a, ws=a, wsb=size):
        return lynx_lib.lynx_chunk_attn_bf16(q, n, stride, cu, B, Hq, Hkv, D, k, v, pool, table, mp, ctx, scale, causal,
                                             out, dt, lse, ws, wsb, None)
    for kw in (dict(n=-1), dict(B=0), dict(Hq=0), dict(Hkv=0), dict(Hq=3, Hkv=2), dict(mp=0), dict(stride=511),
               dict(dt=2), dict(causal=2), dict(scale=0.0), dict(scale=float("inf")), dict(q=None), dict(cu=None),
               dict(k=None), dict(v=None), dict(table=None), dict(ctx=None), dict(out=None), dict(pool=0)):
        assert call(**kw) == -1, kw
    for kw in (dict(D=64), dict(mp=1 << 23), dict(n=1 << 30), dict(B=65536), dict(pool=1 << 24)):
        assert call(**kw) == -2, kw
    for name in ("q", "k", "v", "out", "ws"):
        assert call(**{name: ctypes.c_void_p(a.value + 8)}) == -3, name
    for name in ("cu", "table", "ctx", "lse"):
        assert call(**{name: ctypes.c_void_p(a.value + 2)}) == -3, name
    assert call(stride=516) == -3
    assert call(ws=None) == -4 and call(wsb=size - 1) == -4
    assert call(n=0, q=None, cu=None, k=None, v=None, table=None, ctx=None, out=None, ws=None) == 0
    assert size > 0 and lynx_lib.lynx_chunk_attn_workspace_size(1, 1, 4, 3, 128) == 0


def test_verify_drafts_argument_checks(lynx_lib, a):
    def call(p=a, pb=20, pt=10, q=a, qb=10, qt=10, dt=1, B=1, T=1, V=10, d=a, nd=None, u=a, tok=a, n=a):
        return lynx_lib.lynx_verify_drafts(p, pb, pt, q, qb, qt, dt, B, T, V, d, nd, u, tok, n, None)
    for kw in (dict(B=0), dict(T=0), dict(V=0), dict(dt=2), dict(p=None), dict(d=None), dict(u=None), dict(tok=None),
               dict(n=None), dict(pt=9), dict(qt=9), dict(pb=-1), dict(qb=-1)):
        assert call(**kw) == -1, kw
    assert call(T=65) == -2 and call(V=(1 << 20) + 1, pt=1 << 21, qt=1 << 21) == -2 and call(B=(1 << 24) + 1) == -2
    for name in ("p", "q", "d", "nd", "u", "tok", "n"):
        assert call(**{name: ctypes.c_void_p(a.value + 2)}) == -3, name
    assert call(dt=0, p=ctypes.c_void_p(a.value + 1)) == -3


def test_outputs_that_share_memory_with_inputs_are_refused(lynx_lib, a):
    """Spans that meet in one element only; every call is refused before a launch."""
    def at(offset):
        return ctypes.c_void_p((1 << 40) + offset)
    far = [at((i + 1) << 32) for i in range(16)]

    def assign(**kw):
        x = dict(ctx=far[0], new=far[1], free=far[2], cu=far[3], pos=far[4], slots=far[5], out=far[6], taken=far[7])
        x.update(kw)
        return lynx_lib.lynx_assign_pages(x["ctx"], x["new"], 8, 2, far[8], 4, x["free"], 9, 5, x["cu"], x["pos"],
                                          x["slots"], x["out"], x["taken"], None)
    for name, size in (("cu", 36), ("pos", 20), ("slots", 80), ("out", 32), ("taken", 4)):
        for read, length in (("ctx", 32), ("new", 32), ("free", 36)):
            base = 1 << 20
            assert assign(**{name: at(base), read: at(base + size // 8 * 8 - 8 if size > 8 else base)}) == -1
            assert assign(**{read: at(base), name: at(base + (length - 4) // 8 * 8)}) == -1

    def append(qkv, q, n, stride):
        return lynx_lib.lynx_qkv_append(qkv, n, stride, 4, 2, 128, None, None, 0.0, None, 0, 0, 0, far[0], far[1], q,
                                        far[2], far[3], 4, None)
    last = (2 * 1032 + 1024) * 2          # bytes from the first row's start to the third one's end
    assert append(at(0), at(last - 16), 3, 1032) == -1
    assert append(at(3 * 1024 - 16), at(0), 3, 1032) == -1
    size = lynx_lib.lynx_chunk_attn_workspace_size(3, 1, 4, 2, 128)

    def chunk(q=far[0], out=far[1], lse=far[2], ws=far[3], dt=0):
        return lynx_lib.lynx_chunk_attn_bf16(q, 3, 1032, far[4], 1, 4, 2, 128, far[5], far[6], 4, far[7], 1, far[8], 0.1,
                                             1, out, dt, lse, ws, size, None)
    span = (2 * 1032 + 512) * 2
    assert chunk(q=at(0), out=at(0)) == -1 and chunk(q=at(0), out=at(span - 16)) == -1
    assert chunk(q=at(0), lse=at(span - 4)) == -1 and chunk(q=at(0), ws=at(span - 16)) == -1
    assert chunk(out=at(0), q=at(3 * 1024 - 16)) == -1 and chunk(out=at(0), dt=1, q=at(3 * 2048 - 16)) == -1
    assert chunk(ws=at(0), q=at(size // 16 * 16 - 16)) == -1

    def verify(d=far[0], nd=far[1], u=far[2], tok=far[3], n=far[4]):
        return lynx_lib.lynx_verify_drafts(far[5], 400, 100, far[6], 300, 100, 1, 2, 3, 100, d, nd, u, tok, n, None)
    assert verify(tok=at(0), d=at(28)) == -1 and verify(tok=at(0), u=at(0)) == -1 and verify(tok=at(4), nd=at(0)) == -1
    assert verify(n=at(0), d=at(4)) == -1 and verify(n=at(28), u=at(0)) == -1 and verify(n=far[1]) == -1


def test_bindings_refuse_host_tensors():
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(L.LynxError, match="CUDA"):
        L.lynx_assign_pages(i, i, torch.zeros(1, 1, 1, dtype=torch.int32), i, 1)
    x = torch.zeros(1, 384, dtype=torch.bfloat16)
    pages = torch.zeros(1, 128, 256, dtype=torch.bfloat16)
    with pytest.raises(L.LynxError, match="CUDA"):
        L.lynx_qkv_append(x, 1, 1, None, i, torch.zeros(1, 1, dtype=torch.int64), pages, pages)
    with pytest.raises(L.LynxError, match="CUDA"):
        L.lynx_verify_drafts(torch.zeros(1, 2, 4), None, torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, 2))
