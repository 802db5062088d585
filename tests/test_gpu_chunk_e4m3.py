"""GPU parity of lynx_chunk_attn_e4m3 with the float64 oracle over the values that the
codes stand for, by the rules of the same attention over BF16 pages (the values
are BF16 numbers)."""
import math

import numpy as np
import pytest
import torch

from oracle import e4m3
from progressive_kv_quantization_gb300 import lynx as L
from test_gpu_chunk_attn import batch, check, oracle

pytestmark = pytest.mark.gpu
SIZES = 2.0 ** np.arange(-3, 4)


def batch8(new, ctx, Hq, Hkv, seed, spread=True, **kw):
    """As batch(), the pages in 8 bits: x["k"] and x["v"] are the values as BF16 pages, finite
    everywhere; x["pools"] holds NaN codes and bytes that are no scales past the contexts."""
    x = batch(new, ctx, Hq, Hkv, seed, **kw)
    rng = np.random.default_rng(seed)
    n = x["k"].shape[0]
    codes, scales = [], []
    for name in ("k", "v"):
        values = torch.nan_to_num(x[name].double(), 0.5, 0.5, -0.5).cpu().numpy().transpose(0, 2, 1).copy()
        if spread:
            values *= np.repeat(rng.choice(SIZES, (n, 8)), 32, axis=1)[:, :, None]
        c, s = e4m3.quantise_pages(values)
        x[name] = torch.from_numpy(e4m3.dequantise_pages(c, s).transpose(0, 2, 1).copy()).cuda().bfloat16()
        codes.append(c)
        scales.append(s)
    table, lens = x["table"].cpu().numpy(), x["ctx"].cpu().numpy()
    for b, length in enumerate(lens):
        if length % 256:
            for page in table[b, :, length // 256]:
                for c, s in zip(codes, scales):
                    c[page, length % 256:] = rng.choice([0x7F, 0xFF])
                    s[page, -(-(length % 256) // 32):] = rng.choice([0, 255])
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    x["pools"] = (up(codes[0]).view(torch.float8_e4m3fn), up(codes[1]).view(torch.float8_e4m3fn), up(np.stack(scales, 1)))
    return x


def call8(x, causal=True, **kw):
    return L.lynx_chunk_attn_e4m3(x["q"], x["cu"], *x["pools"], x["table"], x["ctx"], x["Hkv"], causal=causal, **kw)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,ctx,Hq,Hkv", [
    ([1], [1], 1, 1), ([1], [300], 4, 1), ([5], [5], 8, 2), ([17], [1000], 8, 2), ([64], [64], 4, 1),
    ([65], [191], 4, 2), ([128], [128], 3, 1), ([300], [300], 5, 1), ([256], [2000], 2, 2), ([33], [129], 12, 3),
    ([200], [1111], 10, 2), ([1], [4096], 16, 2), ([1000], [1500], 1, 1), ([90], [500], 16, 1)])
def test_one_request(cuda_device, new, ctx, Hq, Hkv, causal):
    x = batch8(new, ctx, Hq, Hkv, sum(new) + ctx[0])
    check(x, causal, *call8(x, causal))
    check(x, causal, *call8(x, causal, out_dtype=torch.float32))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,ctx,Hq,Hkv,pad", [
    ([3, 0, 200, 1, 64], [10, 40, 513, 700, 64], 4, 2, 0),
    ([1] * 40, [1 + 37 * i for i in range(40)], 8, 2, 3),
    ([0, 0, 5], [0, 3, 5], 2, 1, 9),
    ([130, 1, 131, 2, 132], [1300, 1, 131, 900, 2000], 6, 2, 1),
    ([1, 300] * 60, [200, 400] * 60, 4, 4, 1),       # more items than a list holds, of one and of two groups
    ([0], [100], 2, 1, 5)])
def test_ragged_batches_leave_rows_behind(cuda_device, new, ctx, Hq, Hkv, pad, causal):
    x = batch8(new, ctx, Hq, Hkv, len(new) + pad, pad=pad)
    out = torch.full((sum(new) + pad, Hq, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((sum(new) + pad, Hq), 4.0, device="cuda")
    call8(x, causal, out=out, lse=lse)
    check(x, causal, out, lse)
    assert (out[sum(new):] == 3).all() and (lse[sum(new):] == 4).all()


def test_rows_that_see_no_key(cuda_device):
    x = batch8([40, 7], [25, 3], 4, 2, 1)            # chunks longer than their contexts
    out, lse = call8(x)
    check(x, True, out, lse)
    assert torch.isneginf(lse[0]).all() and (out[0] == 0).all()


def test_long_context_is_taken_out_of_the_sum(cuda_device):
    """Past 16,384 keys the sum of the products leaves tensor memory on the way."""
    x = batch8([3], [40000], 2, 1, 2)
    check(x, True, *call8(x, out_dtype=torch.float32))


@pytest.mark.parametrize("byte", [74, 100, 198])
def test_ends_of_the_scales(cuda_device, byte):
    x = batch8([20], [500], 4, 1, 3, spread=False)
    k, v, s = x["pools"]
    s[:] = byte
    for name, codes, which in (("k", k, 0), ("v", v, 1)):
        values = e4m3.dequantise_pages(np.where((c := codes.view(torch.uint8).cpu().numpy()) % 128 == 127, 0, c),
                                       s[:, which].cpu().numpy())
        x[name] = torch.from_numpy(values.transpose(0, 2, 1).copy()).cuda().bfloat16()
    x["q"] = (x["q"].float() / float(x["k"].float().abs().max())).bfloat16()
    check(x, True, *call8(x, out_dtype=torch.float32))


def test_same_as_over_bf16_pages(cuda_device):
    """The values are BF16 numbers, and the products and sums those of the other kernel."""
    x = batch8([70, 300, 1], [1000, 300, 513], 8, 2, 4)
    out, lse = call8(x)
    o, l = L.lynx_chunk_attn_bf16(x["q"], x["cu"], x["k"], x["v"], x["table"], x["ctx"], 2)
    ref = oracle(x, True)
    check(x, True, out, lse, ref=ref)
    check(x, True, o, l, ref=ref)
    assert (out.float() - o.float()).abs().max() <= 2.0 ** -7 * o.float().abs().max()
    assert (lse - l).abs().max() <= 2.0 ** -18 * 30


def test_strided_queries_workspace_stream_and_graph(cuda_device):
    x = batch8([100, 1, 40], [900, 700, 40], 8, 2, 5, extra_stride=256)
    ws = [torch.empty(L.lynx_chunk_attn_workspace_size(141, 3, 8, 2, 128), dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.empty(141, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    lses = [torch.empty(141, 8, device="cuda") for _ in range(2)]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    call8(x, out=outs[0], lse=lses[0], workspace=ws[0], stream=stream)
    torch.cuda.current_stream().wait_stream(stream)
    check(x, True, outs[0], lses[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for o, l, w in zip(outs, lses, ws):
            call8(x, out=o, lse=l, workspace=w)
    for cu, ctx in (([0, 100, 101, 141], [900, 700, 40]), ([0, 5, 105, 141], [500, 300, 36]), ([0, 141, 141, 141], [141, 1, 0])):
        x["cu"].copy_(torch.tensor(cu, dtype=torch.int32))
        x["ctx"].copy_(torch.tensor(ctx, dtype=torch.int32))
        for o, w in zip(outs, ws):
            o.fill_(9)
            w.fill_(0xFF)
        graph.replay()
        check(x, True, outs[0], lses[0])
        assert torch.equal(outs[0], outs[1]) and torch.equal(lses[0], lses[1])


def test_far_pages(cuda_device):
    """Byte offsets past 2^32 in a pool of 140,000 pages."""
    x = batch8([30], [300], 4, 1, 6)
    k, v, s = x["pools"]
    n, far = k.shape[0], 140000
    big = [torch.zeros(far, 256, 128, dtype=torch.uint8, device="cuda") for _ in range(2)]
    for pool, part in zip(big, (k, v)):
        pool[far - n:] = part.view(torch.uint8)
    scales = torch.zeros(far, 2, 8, dtype=torch.uint8, device="cuda")
    scales[far - n:] = s
    out, lse = L.lynx_chunk_attn_e4m3(x["q"], x["cu"], big[0].view(torch.float8_e4m3fn), big[1].view(torch.float8_e4m3fn),
                                      scales, x["table"].clamp(max=n - 1) + far - n, x["ctx"], 1)
    check(x, True, out, lse)


def test_bad_pages_lengths_and_a_wait_that_runs_out(cuda_device):
    x = batch8([50, 3], [600, 40], 4, 2, 7)
    good = x["table"].clone()
    x["table"][0, 0, 1] = 1 << 20
    call8(x)
    with pytest.raises(L.LynxError, match="= 2 "):
        L.lynx_device_status()
    x["table"].copy_(good)
    x["cu"][1] = 99
    call8(x)
    with pytest.raises(L.LynxError, match="= 6 "):
        L.lynx_device_status()
    x["cu"][1] = 50
    L._check(L.load().lynx_test_inject_wait_timeout(1), "inject")
    call8(x)
    with pytest.raises(L.LynxError, match="= 1 "):
        L.lynx_device_status()
    check(x, True, *call8(x))


def test_refusals(cuda_device):
    x = batch8([5], [300], 4, 2, 8)
    k, v, s = x["pools"]
    good = dict(q=x["q"], cu_q=x["cu"], k_pages=k, v_pages=v, scales=s, page_table=x["table"], ctx_len=x["ctx"], n_kv_heads=2)
    L.lynx_chunk_attn_e4m3(**good)
    for change, word in [
            (dict(q=x["q"].float()), "q must"), (dict(k_pages=x["k"]), "k_pages"), (dict(v_pages=v[:, :128]), "v_pages"),
            (dict(scales=s.float()), "scales"), (dict(scales=s[:1]), "scales"), (dict(cu_q=x["cu"][:1]), "cu_q"),
            (dict(n_kv_heads=1), "page_table"), (dict(ctx_len=x["ctx"].cpu()), "ctx_len"), (dict(out_dtype=torch.float16), "out_dtype"),
            (dict(sm_scale=-1.0), "sm_scale"), (dict(sm_scale=2.0 ** 21), "sm_scale"), (dict(sm_scale=math.nan), "sm_scale"),
            (dict(workspace=torch.empty(8, dtype=torch.uint8, device="cuda")), "workspace")]:
        with pytest.raises(L.LynxError, match=word):
            L.lynx_chunk_attn_e4m3(**{**good, **change})
    L.lynx_device_status()
