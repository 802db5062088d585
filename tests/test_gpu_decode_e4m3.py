"""Decode and verification attention over pages in 8 bits against float64."""
import math

import numpy as np
import pytest
import torch

from e4m3_testutil import Cache, decode_bound, score_error, to_bf16
from oracle import e4m3
from progressive_kv_quantization_gb300 import lynx as L

pytestmark = pytest.mark.gpu
SCALE = 1 / math.sqrt(128)


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.view(dtype)


def pools_on_gpu(cache):
    k, v, s = cache.pools()
    return dev(k, torch.float8_e4m3fn), dev(v, torch.float8_e4m3fn), dev(s)


def queries(shape, seed, size=1.0):
    return to_bf16(np.random.default_rng(seed).standard_normal(shape) * size)


def check(cache, q, ctx, causal, out, lse, scale=SCALE):
    B, T, Hq, _ = q.shape
    G = Hq // cache.Hkv
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(B):
        for h in range(cache.Hkv):
            k, v = cache.values(b, h)
            rows = q[b, :, h * G:(h + 1) * G].reshape(T * G, 128)
            seen = [ctx[b] - T + i + 1 if causal else ctx[b] for i in range(T) for _ in range(G)]
            ro, rl = e4m3.attention(rows, k, v, scale, seen)
            o, l = out[b, :, h * G:(h + 1) * G].reshape(T * G, 128), lse[b, :, h * G:(h + 1) * G].reshape(-1)
            assert np.abs(o - ro).max() <= decode_bound(rows, k, v, scale), (b, h)
            none = np.isneginf(rl)
            assert np.array_equal(none, np.isneginf(l)), (b, h)
            # the scores' error, log2's and a rounding of the result
            far = score_error(rows, k, scale) + 2.0 ** -19 + 2.0 ** -22 * np.abs(rl[~none])
            assert np.all(np.abs(l[~none] - rl[~none]) <= far), (b, h)


def run(cache, q, ctx, causal, **kw):
    k, v, s = pools_on_gpu(cache)
    return L.lynx_decode_attn_e4m3(dev(q.astype(np.float32)).to(torch.bfloat16), k, v, s, dev(cache.table),
                                   dev(np.array(ctx, dtype=np.int32)), cache.Hkv, causal=causal, **kw)


EDGES = [0, 1, 31, 32, 33, 127, 128, 129, 255, 256, 257, 600]


@pytest.mark.parametrize("Hq,Hkv,T", [(1, 1, 1), (8, 2, 1), (8, 1, 1), (9, 1, 1), (16, 1, 1), (4, 2, 5), (3, 1, 6),
                                      (20, 2, 3)])
def test_contexts_at_every_edge(Hq, Hkv, T):
    cache = Cache(EDGES, Hkv, seed=Hq + T)
    q = queries((len(EDGES), T, Hq, 128), 1)
    for causal in (False, True):
        out, lse = run(cache, q, EDGES, causal)
        check(cache, q, EDGES, causal, out, lse)
    L.lynx_device_status()


@pytest.mark.parametrize("lens,Hq,Hkv,T", [
    ([983], 32, 8, 1),                       # every head cut
    ([20000], 4, 1, 1),                      # one long context over all SMs
    ([5000, 3, 9000, 1, 0, 257], 8, 2, 1),   # ragged
    ([300] * 70, 16, 8, 1),                  # more items than CTAs
    ([700, 2500], 8, 1, 32),                 # 256 rows: sixteen tiles of one head
    ([2500], 2, 2, 64),
    ([1] * 40, 8, 8, 1),
])
def test_splits(lens, Hq, Hkv, T):
    cache = Cache(lens, Hkv, seed=3)
    q = queries((len(lens), T, Hq, 128), 4)
    out, lse = run(cache, q, lens, True)
    check(cache, q, lens, True, out, lse)
    again = run(cache, q, lens, True)        # nothing depends on timing
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    L.lynx_device_status()


def test_scales_of_all_sizes():
    """Blocks from 2^-12 to 2^12 of the usual size, queries of 2^-9: the largest block decides."""
    cache = Cache([1500, 400], 2, seed=5, spread=12)
    q = queries((2, 1, 8, 128), 6, size=2.0 ** -9)
    out, lse = run(cache, q, [1500, 400], False)
    check(cache, q, [1500, 400], False, out, lse)


@pytest.mark.parametrize("byte", [74, 75, 127, 197, 198])
def test_ends_of_the_scales(byte):
    cache = Cache([300], 1, seed=7)
    for s in cache.scales:
        s[:] = byte
    k, _ = cache.values(0, 0)
    size = 1.0 / float(np.abs(k).max())      # scores of a few units
    q = to_bf16(np.random.default_rng(8).standard_normal((1, 1, 4, 128)) * size)
    out, lse = run(cache, q, [300], False)
    check(cache, q, [300], False, out, lse)


def test_queries_of_all_sizes():
    """Rows of one tile between 2^-60 and 2^8, channels of a row between 1 and 2^-20, a row of zeros."""
    cache = Cache([777], 1, seed=9)
    q = queries((1, 1, 8, 128), 10)
    q[0, 0] *= 2.0 ** np.array([0, 8, -8, -30, -60, 4, 0, 0])[:, None]
    q[0, 0, 6] *= 2.0 ** -(np.arange(128) % 21)
    q[0, 0, 7] = 0.0
    out, lse = run(cache, q, [777], False)
    check(cache, q, [777], False, out, lse)


def test_a_key_far_above_the_others():
    """Probabilities down to 2^-30 of the largest count in full: one key's score stands 20 above 20,000 equal ones."""
    n = 20001
    cache = Cache([n], 1, seed=11)
    cache.codes[0][:] = 0x38                 # keys of ones
    page, at = divmod(700, 256)
    cache.codes[0][cache.table[0, 0, page], at] = 0x40   # twos
    for s in cache.scales:
        s[:] = 127
    last = cache.table[0, 0, n // 256]
    cache.codes[0][last, n % 256:] = 0x7F
    q = to_bf16(np.full((1, 1, 4, 128), 20.0 / math.sqrt(128)))
    out, lse = run(cache, q, [n], False)
    check(cache, q, [n], False, out, lse)


def test_far_pages():
    """Byte offsets past 2^32 in a pool of 140,000 pages."""
    small = Cache([520], 2, seed=12, spare=0)
    k, v, s = pools_on_gpu(small)
    n, far = small.codes[0].shape[0], 140000
    big = [torch.zeros(far, 256, 128, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = torch.zeros(far, 2, 8, dtype=torch.uint8, device="cuda")
    for pool, part in zip(big, (k, v)):
        pool[far - n:] = part.view(torch.uint8)
    scales[far - n:] = s
    table = dev(np.where(small.table >= 0, small.table + far - n, small.table))
    q = queries((1, 2, 6, 128), 13)
    out, lse = L.lynx_decode_attn_e4m3(dev(q.astype(np.float32)).to(torch.bfloat16), big[0].view(torch.float8_e4m3fn),
                                       big[1].view(torch.float8_e4m3fn), scales, table,
                                       dev(np.array([520], dtype=np.int32)), 2, causal=True)
    check(small, q, [520], True, out, lse)


def test_outputs_workspace_stream_and_graph():
    """The caller's buffers on a stream of the caller's; one captured call replayed with other
    lengths and queries; two captured calls with a workspace each."""
    lens = [900, 40, 2000]
    cache = Cache(lens, 2, seed=14)
    k, v, s = pools_on_gpu(cache)
    table = dev(cache.table)
    qs = [queries((3, 2, 8, 128), 15 + i) for i in range(2)]
    q = dev(qs[0].astype(np.float32)).to(torch.bfloat16)
    ctx = dev(np.array(lens, dtype=np.int32))
    stream = torch.cuda.Stream()
    bufs = []
    for _ in range(2):
        bufs.append((torch.empty(3, 2, 8, 128, device="cuda"), torch.empty(3, 2, 8, device="cuda"),
                     torch.empty(L.lynx_decode_attn_e4m3_workspace_size(3, 2, 8, 2, 128), dtype=torch.uint8, device="cuda")))

    def call(i, **kw):
        o, l, w = bufs[i]
        return L.lynx_decode_attn_e4m3(q, k, v, s, table, ctx, 2, causal=True, out=o, lse=l, workspace=w, **kw)

    stream.wait_stream(torch.cuda.current_stream())
    out, lse = call(0, stream=stream)
    assert out is bufs[0][0] and lse is bufs[0][1]
    torch.cuda.current_stream().wait_stream(stream)
    check(cache, qs[0], lens, True, out, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(0)
        call(1)
    for lens2, x in ((lens, qs[1]), ([300, 0, 1999], qs[0]), ([2, 33, 512], qs[1])):
        q.copy_(dev(x.astype(np.float32)).to(torch.bfloat16))
        ctx.copy_(dev(np.array(lens2, dtype=np.int32)))
        for o, l, w in bufs:
            o.fill_(7.0)
            w.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        part = Cache(lens, 2, seed=14, poison=False)   # keys past a shorter context are there, and not seen
        full = part.lens
        part.lens = lens2
        check(part, x, lens2, True, *bufs[0][:2])
        part.lens = full
        assert torch.equal(bufs[0][0], bufs[1][0]) and torch.equal(bufs[0][1], bufs[1][1])
    L.lynx_device_status()


def test_calls_without_an_lse_and_with_bad_pages():
    cache = Cache([400], 1, seed=17)
    q = queries((1, 1, 4, 128), 18)
    k, v, s = pools_on_gpu(cache)
    table = dev(cache.table).clone()
    table[0, 0, 1] = k.shape[0]              # outside the pool: page 0 is read, and the word set
    args = [dev(q.astype(np.float32)).to(torch.bfloat16), k, v, s, table, dev(np.array([400], dtype=np.int32)), 1]
    L.lynx_decode_attn_e4m3(*args)
    with pytest.raises(L.LynxError, match="= 2 "):
        L.lynx_device_status()
    table[0, 0, 1] = -1
    L.lynx_decode_attn_e4m3(*args)
    with pytest.raises(L.LynxError, match="= 2 "):
        L.lynx_device_status()
    args[4] = dev(cache.table)
    for n in (-5, 513):                      # counts as 0 and as two pages
        args[5] = dev(np.array([n], dtype=np.int32))
        out, lse = L.lynx_decode_attn_e4m3(*args)
        with pytest.raises(L.LynxError, match="= 3 "):
            L.lynx_device_status()
        assert n > 0 or (torch.all(out == 0) and torch.all(torch.isneginf(lse)))


def test_a_wait_that_runs_out():
    """The context stays usable, and the next call gives its answer."""
    cache = Cache([3000, 100], 2, seed=19)
    q = queries((2, 1, 8, 128), 20)
    L._check(L.load().lynx_test_inject_wait_timeout(1), "inject")
    run(cache, q, [3000, 100], False)
    with pytest.raises(L.LynxError, match="= 1 "):
        L.lynx_device_status()
    out, lse = run(cache, q, [3000, 100], False)
    check(cache, q, [3000, 100], False, out, lse)
    L.lynx_device_status()


def test_refusals():
    cache = Cache([400], 1, seed=21)
    k, v, s = pools_on_gpu(cache)
    q = torch.zeros(1, 1, 4, 128, dtype=torch.bfloat16, device="cuda")
    table, ctx = dev(cache.table), dev(np.array([400], dtype=np.int32))
    good = dict(q=q, k_pages=k, v_pages=v, scales=s, page_table=table, ctx_len=ctx, n_kv_heads=1)
    L.lynx_decode_attn_e4m3(**good)
    bad = [
        (dict(q=q.float()), "q"), (dict(q=q[0]), "q"), (dict(q=q.cpu()), "CUDA"), (dict(k_pages=k.view(torch.uint8)), "k_pages"),
        (dict(v_pages=v[:1]), "v_pages"), (dict(scales=s[:, 0]), "scales"), (dict(scales=s.to(torch.int32)), "scales"),
        (dict(page_table=table.long()), "page_table"), (dict(page_table=table[0]), "page_table"), (dict(ctx_len=ctx.long()), "ctx_len"),
        (dict(ctx_len=ctx.repeat(2)), "ctx_len"), (dict(n_kv_heads=3), "page_table"), (dict(sm_scale=0.0), "sm_scale"),
        (dict(sm_scale=math.inf), "sm_scale"), (dict(out=torch.empty(1, 1, 4, 128, dtype=torch.bfloat16, device="cuda")), "out"),
        (dict(lse=torch.empty(4, device="cuda")), "lse"), (dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda")), "workspace"),
        (dict(q=torch.zeros(1, 65, 1, 128, dtype=torch.bfloat16, device="cuda")), "T=65"),
        (dict(q=torch.zeros(1, 1, 257, 128, dtype=torch.bfloat16, device="cuda")), "256"),
    ]
    for change, word in bad:
        with pytest.raises(L.LynxError, match=word):
            L.lynx_decode_attn_e4m3(**{**good, **change})
    shared = torch.zeros(1, 1, 4, 128, device="cuda")
    with pytest.raises(L.LynxError, match="overlaps"):
        L.lynx_decode_attn_e4m3(**{**good, "q": shared.view(torch.bfloat16).view(-1)[:512].view(1, 1, 4, 128),
                                   "out": shared})
    L.lynx_device_status()
