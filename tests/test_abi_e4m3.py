"""Argument checks of the entry points over pages in 8 bits and of the token log probabilities, without a GPU."""
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


def off(p, n):
    return ctypes.c_void_p(p.value + n)


def test_decode_attn_argument_checks(lynx_lib, a):
    size = lynx_lib.lynx_decode_attn_e4m3_workspace_size(1, 1, 4, 2, 128)

    def call(q=a, B=1, T=1, Hq=4, Hkv=2, D=128, k=a, v=a, sc=a, pool=1, table=a, mp=1, ctx=a, scale=0.1, causal=1, out=a,
             lse=a, ws=a, wsb=size):
        return lynx_lib.lynx_decode_attn_e4m3(q, B, T, Hq, Hkv, D, k, v, sc, pool, table, mp, ctx, scale, causal, out, lse,
                                              ws, wsb, None)
    for kw in (dict(B=0), dict(T=0), dict(Hq=0), dict(Hkv=0), dict(Hq=3), dict(mp=0), dict(causal=2), dict(scale=0.0),
               dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")), dict(q=None), dict(k=None), dict(v=None),
               dict(sc=None), dict(table=None), dict(ctx=None), dict(out=None), dict(pool=0), dict(pool=-1)):
        assert call(**kw) == -1, kw
    for kw in (dict(D=64), dict(T=65), dict(T=64, Hq=10), dict(B=65536), dict(mp=1 << 23), dict(pool=1 << 23)):
        assert call(**kw) == -2, kw
    for name in ("q", "k", "v", "sc", "out", "ws"):
        assert call(**{name: off(a, 8)}) == -3, name
    for name in ("table", "ctx", "lse"):
        assert call(**{name: off(a, 2)}) == -3, name
    assert call(ws=None) == -4 and call(wsb=size - 1) == -4
    assert size > 0
    for bad in ((0, 1, 4, 2, 128), (1, 65, 4, 2, 128), (1, 1, 4, 3, 128), (1, 1, 4, 2, 64), (1, 64, 48, 8, 128)):
        assert lynx_lib.lynx_decode_attn_e4m3_workspace_size(*bad) == 0, bad


def test_chunk_attn_argument_checks(lynx_lib, a):
    size = lynx_lib.lynx_chunk_attn_workspace_size(1, 1, 4, 2, 128)

    def call(q=a, n=1, stride=512, cu=a, B=1, Hq=4, Hkv=2, D=128, k=a, v=a, sc=a, pool=1, table=a, mp=1, ctx=a, scale=0.1,
             causal=1, out=a, dt=0, lse=a, ws=a, wsb=size):
        return lynx_lib.lynx_chunk_attn_e4m3(q, n, stride, cu, B, Hq, Hkv, D, k, v, sc, pool, table, mp, ctx, scale, causal,
                                             out, dt, lse, ws, wsb, None)
    for kw in (dict(n=-1), dict(B=0), dict(Hq=0), dict(Hkv=0), dict(Hq=3), dict(mp=0), dict(stride=511), dict(dt=2),
               dict(causal=2), dict(scale=0.0), dict(scale=float("inf")), dict(q=None), dict(cu=None), dict(k=None),
               dict(v=None), dict(sc=None), dict(table=None), dict(ctx=None), dict(out=None), dict(pool=0)):
        assert call(**kw) == -1, kw
    for kw in (dict(D=64), dict(mp=1 << 23), dict(n=1 << 30), dict(B=65536), dict(pool=1 << 23), dict(scale=2.0 ** 21)):
        assert call(**kw) == -2, kw
    for name in ("q", "k", "v", "sc", "out", "ws"):
        assert call(**{name: off(a, 8)}) == -3, name
    for name in ("cu", "table", "ctx", "lse"):
        assert call(**{name: off(a, 2)}) == -3, name
    assert call(stride=516) == -3 and call(ws=None) == -4 and call(wsb=size - 1) == -4
    assert call(n=0, q=None, cu=None, k=None, v=None, sc=None, table=None, ctx=None, out=None, ws=None) == 0


def test_qkv_append_argument_checks(lynx_lib, a):
    def call(qkv=a, n=1, stride=384, Hq=1, Hkv=1, D=128, wq=None, wk=None, eps=1e-6, cs=a, mp=4, rot=128, il=0, pos=a,
             slots=a, q=a, k=a, v=a, sc=a, pool=1):
        return lynx_lib.lynx_qkv_append_e4m3(qkv, n, stride, Hq, Hkv, D, wq, wk, eps, cs, mp, rot, il, pos, slots, q, k, v,
                                             sc, pool, None)
    for kw in (dict(n=-1), dict(Hq=0), dict(Hkv=0), dict(stride=383), dict(il=2), dict(pool=0), dict(cs=None),
               dict(mp=0), dict(qkv=None), dict(pos=None), dict(slots=None), dict(q=None), dict(k=None), dict(v=None),
               dict(q=off(a, 16), sc=None)):
        assert call(**kw) == -1, kw
    for kw in (dict(D=64), dict(rot=8), dict(rot=144), dict(rot=-16), dict(wq=a, eps=-1.0), dict(wk=a, eps=float("nan")),
               dict(Hq=65535, stride=1 << 24)):
        assert call(**kw) == -2, kw
    far = ctypes.c_void_p(1 << 40)
    assert call(q=far, pool=1 << 23) == -2 and call(q=far, sc=None) == -1 and call(q=far, sc=off(a, 8)) == -3
    for name in ("qkv", "cs", "q", "k", "v", "wq", "wk"):
        assert call(**{name: off(a, 8)}) == -3, name
    assert call(stride=388) == -3 and call(pos=off(a, 2)) == -3 and call(slots=off(a, 4)) == -3
    assert call(n=0, qkv=None, pos=None, slots=None, q=None, k=None, v=None, cs=None, sc=None) == 0


def test_token_logprobs_argument_checks(lynx_lib, a):
    far = [ctypes.c_void_p((i + 1) << 40) for i in range(8)]

    def call(x=far[0], stride=10, dt=1, n=2, V=10, tok=far[1], top=3, lp=far[2], h=far[3], ids=far[4], tl=far[5]):
        return lynx_lib.lynx_token_logprobs(x, stride, dt, n, V, tok, top, lp, h, ids, tl, None)
    for kw in (dict(n=-1), dict(V=0), dict(top=-1), dict(top=11), dict(dt=2), dict(stride=9), dict(x=None), dict(tok=None),
               dict(lp=None), dict(h=None), dict(ids=None), dict(tl=None)):
        assert call(**kw) == -1, kw
    for kw in (dict(V=(1 << 24) + 1, stride=1 << 25), dict(n=(1 << 24) + 1), dict(top=33, V=40, stride=40)):
        assert call(**kw) == -2, kw
    for name in ("x", "tok", "lp", "h", "ids", "tl"):
        assert call(**{name: off(far[6], 2)}) == -3, name
    assert call(dt=0, x=off(far[6], 1)) == -3
    assert call(n=0, x=None, tok=None, lp=None, h=None, ids=None, tl=None) == 0


def test_outputs_that_share_memory_with_inputs_are_refused(lynx_lib):
    """Spans that meet in one element only; every call is refused before a launch."""
    def at(offset):
        return ctypes.c_void_p((1 << 40) + offset)
    far = [at((i + 1) << 32) for i in range(16)]
    size = lynx_lib.lynx_decode_attn_e4m3_workspace_size(2, 3, 4, 2, 128)

    def decode(q=far[0], out=far[1], lse=far[2], ws=far[3]):
        return lynx_lib.lynx_decode_attn_e4m3(q, 2, 3, 4, 2, 128, far[4], far[5], far[6], 4, far[7], 1, far[8], 0.1, 1, out,
                                              lse, ws, size, None)
    rows = 2 * 3 * 4
    assert decode(q=at(0), out=at(rows * 256 - 16)) == -1 and decode(out=at(0), q=at(rows * 512 - 16)) == -1
    assert decode(q=at(0), lse=at(rows * 256 - 4)) == -1 and decode(q=at(0), ws=at(rows * 256 - 16)) == -1

    def logprobs(x=far[0], tok=far[1], lp=far[2], h=far[3], ids=far[4], tl=far[5]):
        return lynx_lib.lynx_token_logprobs(x, 120, 1, 3, 100, tok, 5, lp, h, ids, tl, None)
    for name, n in (("lp", 12), ("h", 12), ("ids", 60), ("tl", 60)):
        assert logprobs(**{name: at(0), "x": at(n - 4)}) == -1 and logprobs(**{name: at((2 * 120 + 100) * 4 - 4), "x": at(0)}) == -1
        assert logprobs(**{name: at(0), "tok": at(n - 4)}) == -1 and logprobs(**{name: at(8), "tok": at(0)}) == -1


def test_bindings_refuse_host_tensors():
    i = torch.zeros(1, dtype=torch.int32)
    pages, scales = torch.zeros(1, 256, 128, dtype=torch.uint8).view(torch.float8_e4m3fn), torch.zeros(1, 2, 8, dtype=torch.uint8)
    q, table = torch.zeros(1, 1, 1, 128, dtype=torch.bfloat16), torch.zeros(1, 1, 1, dtype=torch.int32)
    with pytest.raises(L.LynxError, match="CUDA"):
        L.lynx_decode_attn_e4m3(q, pages, pages, scales, table, i, 1)
    with pytest.raises(L.LynxError, match="CUDA"):
        L.lynx_chunk_attn_e4m3(q[0], torch.zeros(2, dtype=torch.int32), pages, pages, scales, table, i, 1)
    with pytest.raises(L.LynxError, match="CUDA"):
        L.lynx_qkv_append_e4m3(torch.zeros(1, 384, dtype=torch.bfloat16), 1, 1, None, i, torch.zeros(1, 1, dtype=torch.int64),
                               pages, pages, scales)
    with pytest.raises(L.LynxError, match="CUDA"):
        L.lynx_token_logprobs(torch.zeros(1, 8), i)
