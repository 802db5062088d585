"""GPU parity of lynx_chunk_attn_bf16 with the float64 oracle: ragged batches,
one token to several tiles, odd lengths, group sizes that do not divide the
tile, rows that see no key, strided queries, garbage past the context, splits
of long contexts, and the paths around them."""
import math

import numpy as np
import pytest
import torch

from oracle import serving as sv
from progressive_kv_quantization_gb300 import lynx as L

pytestmark = pytest.mark.gpu
D = 128
LSE_TOL = 2.0 ** -11


def batch(new, ctx, Hq, Hkv, seed, pad=0, k_scale=1.0, max_pages=None, extra_stride=0):
    """Random batch on the device; ctx holds all keys.  Pages in shuffled order, and
    everything past a request's context (and unused table entries) is garbage."""
    g = torch.Generator("cuda").manual_seed(seed)
    B = len(new)
    n_rows = sum(new) + pad
    pages = [-(-c // 256) for c in ctx]
    max_pages = max_pages or max(max(pages), 1)
    n_pool = sum(pages) * Hkv + 2
    order = torch.randperm(n_pool, generator=torch.Generator().manual_seed(seed)).int()
    table = torch.full((B, Hkv, max_pages), 2 ** 30, dtype=torch.int32)      # unused entries: far outside the pool
    at = 0
    for b in range(B):
        table[b, :, :pages[b]] = order[at:at + Hkv * pages[b]].view(Hkv, pages[b])
        at += Hkv * pages[b]
    k = (torch.randn(n_pool, D, 256, generator=g, device="cuda") * k_scale).bfloat16()
    v = (torch.randn(n_pool, D, 256, generator=g, device="cuda")
         + torch.randn(1, D, 1, generator=g, device="cuda")).bfloat16()
    for b in range(B):
        if ctx[b] % 256:
            ids = table[b, :, pages[b] - 1].long().cuda()
            k[ids, :, ctx[b] % 256:] = float("nan")
            v[ids, :, ctx[b] % 256:] = float("inf")
    q = torch.randn(n_rows, Hq * D + extra_stride, generator=g, device="cuda").bfloat16()[:, :Hq * D]
    q = q.unflatten(1, (Hq, D))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    cu = i32([sum(new[:b]) for b in range(B + 1)])
    return dict(q=q, cu=cu, k=k, v=v, table=table.cuda(), ctx=i32(list(ctx)), Hkv=Hkv)


def oracle(x, causal, scale=1 / math.sqrt(D)):
    f = lambda t: t.double().cpu().numpy()
    table = x["table"].cpu().numpy().astype(np.int64)
    with np.errstate(invalid="ignore"):
        return sv.chunk_attention(f(x["q"]), x["cu"].cpu().numpy(), f(x["k"]), f(x["v"]), table, x["ctx"].cpu().numpy(),
                                  x["Hkv"], scale, causal)


def call(x, causal, **kw):
    return L.lynx_chunk_attn_bf16(x["q"], x["cu"], x["k"], x["v"], x["table"], x["ctx"], x["Hkv"], causal=causal, **kw)


def check(x, causal, out, lse, v_max=None, scale=1 / math.sqrt(D), ref=None):
    """|out - ref| <= 2^-8 sum_j p_j |v_j| for P's rounding to BF16 (half a step of each)
    + half a BF16 step, 2^-8, of the value.  sum_j p_j |v_j| is put at the largest |v| of
    the pool, which it stays well below wherever more than one key matters (one key:
    P is 1 and not rounded); float32's own errors, 2^-17 of it, have their room there."""
    torch.cuda.synchronize()
    L.lynx_device_status()
    ro, rl = oracle(x, causal, scale) if ref is None else ref
    g, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    rows = ~np.isnan(rl)
    v = x["v"].float()
    vm = float(v[torch.isfinite(v)].abs().max())
    half = 2.0 ** -8 if out.dtype == torch.bfloat16 else 0.0
    lim = 2.0 ** -8 * vm + half * np.abs(ro)
    err = np.abs(g - ro)
    assert np.all(err[rows] <= lim[rows]), f"output off by {np.nanmax(err)}"
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(gl) & rows, empty)
    assert np.all(g[empty] == 0)
    fin = rows & ~empty
    # scores: exact products, 128 float32 additions of partial sums of at most
    # scale * sum |q k| < 30, each off by 2^-23 at worst: 128 * 2^-23 * 30 < 2^-11
    assert np.all(np.abs(gl[fin] - rl[fin]) <= LSE_TOL + 2.0 ** -20 * np.abs(rl[fin])), np.max(np.abs(gl[fin] - rl[fin]))
    # over all: the mean square error of P's rounding is far smaller than its bound
    big = fin & (np.abs(ro).max(-1) > 0)
    if big.sum() > 4:
        rel = np.linalg.norm(err[big]) / np.linalg.norm(ro[big])
        assert rel < 2.0 ** -7, f"relative error {rel}"
    return g


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,ctx,Hq,Hkv", [
    ([1], [1], 1, 1), ([1], [300], 4, 1), ([5], [5], 8, 2), ([17], [1000], 8, 2), ([64], [64], 4, 1),
    ([65], [191], 4, 2), ([128], [128], 3, 1), ([300], [300], 5, 1), ([256], [2000], 2, 2), ([33], [129], 12, 3),
    ([200], [1111], 10, 2), ([1], [4096], 16, 2), ([1000], [1500], 1, 1), ([90], [500], 16, 1)])
def test_one_request(cuda_device, new, ctx, Hq, Hkv, causal):
    x = batch(new, ctx, Hq, Hkv, sum(new) + ctx[0])
    check(x, causal, *call(x, causal))
    check(x, causal, *call(x, causal, out_dtype=torch.float32))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,ctx,Hq,Hkv,pad", [
    ([3, 0, 200, 1, 64], [10, 40, 513, 700, 64], 4, 2, 0),
    ([1] * 40, [1 + 37 * i for i in range(40)], 8, 2, 3),
    ([0, 0, 5], [0, 3, 5], 2, 1, 9),
    ([130, 1, 131, 2, 132], [1300, 1, 131, 900, 2000], 6, 2, 1),
    ([0], [100], 2, 1, 0), ([0], [100], 2, 1, 5)])
def test_ragged_batches_leave_rows_behind(cuda_device, new, ctx, Hq, Hkv, pad, causal):
    x = batch(new, ctx, Hq, Hkv, len(new) + pad, pad=pad)
    out = torch.full((sum(new) + pad, Hq, D), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((sum(new) + pad, Hq), 4.0, device="cuda")
    call(x, causal, out=out, lse=lse)
    check(x, causal, out, lse)
    assert (out[sum(new):] == 3).all() and (lse[sum(new):] == 4).all()


def test_many_requests_of_one_token(cuda_device):
    """More requests than a CTA has threads, and more items than its list holds."""
    rng = np.random.default_rng(0)
    ctx = [int(c) for c in rng.integers(0, 300, 700)]
    x = batch([1] * 700, ctx, 2, 2, 5)
    check(x, True, *call(x, True))
    x = batch([1] * 5000, [int(c) for c in rng.integers(1, 60, 5000)], 1, 1, 6)
    check(x, True, *call(x, True))


def test_requests_of_one_group_between_requests_of_two(cuda_device):
    """Tiles of up to 128 rows between tiles of 256, many tiles of keys each: both
    groups of rows keep step with the ring of key and value tiles."""
    for new, ctx, Hq, Hkv in (([1, 300, 1, 200, 1], [3000, 3000, 2500, 2000, 900], 8, 1),
                              ([1, 1, 1, 129, 2, 513], [9000, 100, 4000, 5000, 6000, 1000], 2, 2),
                              ([64, 1, 65, 1, 66], [4000, 4000, 4000, 4000, 4000], 6, 2)):
        x = batch(new, ctx, Hq, Hkv, sum(new))
        check(x, True, *call(x, True))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,ctx,Hq,Hkv", [
    ([3, 1, 40], [300, 2000, 600], 128, 1), ([2, 5], [700, 5], 300, 1), ([1, 7], [900, 260], 257, 1),
    ([1, 70, 3], [400, 300, 5], 160, 160), ([2, 129], [200, 129], 304, 152), ([1] * 9, [513] * 9, 200, 40)])
def test_many_heads_of_either_kind(cuda_device, new, ctx, Hq, Hkv, causal):
    """More query heads a group than half a tile or a whole one has rows, and more KV
    heads than there are CTAs."""
    x = batch(new, ctx, Hq, Hkv, Hq + Hkv)
    check(x, causal, *call(x, causal))


def test_a_prompt_cut_everywhere(cuda_device):
    """Prompts of every length around the tile's, so that cuts fall near both ends of
    tiles of few keys."""
    rng = np.random.default_rng(3)
    new = [int(n) for n in rng.integers(1, 420, 60)]
    x = batch(new, [n + int(rng.integers(0, 300)) for n in new], 8, 2, 17)
    check(x, True, *call(x, True))
    for n in (1500, 1537, 1999, 2048):
        x = batch([n], [n + n % 5], 16, 8, n)
        check(x, True, *call(x, True))


def test_rows_that_see_no_key(cuda_device):
    # more new tokens than keys: the first rows see none
    x = batch([300, 5], [100, 0], 4, 2, 8)
    out, lse = call(x, True)
    g = check(x, True, out, lse)
    assert (g[:200] == 0).all() and torch.isneginf(lse[:200]).all()
    assert (g[300:] == 0).all() and torch.isneginf(lse[300:]).all()
    check(x, False, *call(x, False))


@pytest.mark.parametrize("k_scale,scale", [(1.0, 1 / math.sqrt(D)), (8.0, 1 / math.sqrt(D)), (1.0, 2.0 ** -14),
                                           (30.0, 0.2)])
def test_score_ranges(cuda_device, k_scale, scale):
    """Flat scores to nearly one-hot rows: the running maximum never moves, or often."""
    x = batch([100, 30], [1500, 900], 4, 2, 11, k_scale=k_scale)
    out, lse = call(x, True, sm_scale=scale)
    ro, rl = oracle(x, True, scale)
    torch.cuda.synchronize()
    g, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    # scores of up to `top`, a float32 sum of 128 exact products each: absolute
    # error 128 * 2^-24 * top; a probability is off by the factor e^that
    top = float(np.abs(rl).max()) + 10
    ds = 128 * 2.0 ** -24 * top * 2
    vm = float(x["v"].float()[torch.isfinite(x["v"].float())].abs().max())
    assert np.all(np.abs(g - ro) <= (2.0 ** -8 + 2 * ds) * vm + 2.0 ** -8 * np.abs(ro))
    assert np.all(np.abs(gl - rl) <= ds + 2.0 ** -20 * np.abs(rl))


@pytest.mark.parametrize("order", ["up", "down"])
def test_running_maximum_moves_on_every_tile(cuda_device, order):
    """Keys whose scores grow (or fall) by far more than the lag from tile to tile."""
    Hq, Hkv, n, T = 4, 1, 2048, 20
    x = batch([T], [n], Hq, Hkv, 12)
    q = x["q"]
    q[:, :, 0] = 8.0
    ramp = torch.arange(n, device="cuda").float() * (0.5 if order == "up" else -0.5)
    ids = x["table"][0, 0].long()
    kk = x["k"][ids].clone()
    kk[:, 0, :] = ramp.view(-1, 256).bfloat16()
    x["k"][ids] = kk
    out, lse = call(x, True)
    ro, rl = oracle(x, True)
    torch.cuda.synchronize()
    top = float(np.abs(rl).max())
    ds = 128 * 2.0 ** -24 * top * 2
    vm = float(x["v"].float()[torch.isfinite(x["v"].float())].abs().max())
    assert np.all(np.abs(out.double().cpu().numpy() - ro) <= (2.0 ** -8 + 2 * ds) * vm + 2.0 ** -8 * np.abs(ro))
    assert np.all(np.abs(lse.double().cpu().numpy() - rl) <= ds + 2.0 ** -20 * np.abs(rl))


def test_strided_queries_and_wide_tables(cuda_device):
    x = batch([70, 9], [600, 300], 4, 2, 13, max_pages=9, extra_stride=5 * 128)
    assert x["q"].stride(0) == 9 * 128
    check(x, True, *call(x, True))


def test_long_context_split_over_the_machine(cuda_device):
    """One token, and a few, over 50,000 keys: every CTA takes a part of the tile."""
    for new in ([1], [3, 40]):
        ctx = [50001, 20000][:len(new)]
        x = batch(new, ctx, 8, 2, 14)
        a = call(x, True)
        check(x, True, *a)
        b = call(x, True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])      # the split does not depend on timing


def test_large_prefill_sampled_rows(cuda_device):
    """4,096 tokens over 9,000 keys with 16 heads: sampled rows against the oracle."""
    new, ctx, Hq, Hkv = [4096], [9000], 16, 4
    x = batch(new, ctx, Hq, Hkv, 15)
    out, lse = call(x, True)
    torch.cuda.synchronize()
    L.lynx_device_status()
    rng = np.random.default_rng(0)
    ids = x["table"][0].long()
    for t in [0, 1, 63, 64, 4095, *rng.integers(0, 4096, 40)]:
        h = int(rng.integers(0, Hq))
        n = 9000 - 4096 + int(t) + 1
        k = x["k"][ids[h // 4]].permute(0, 2, 1).reshape(-1, D)[:n].double()
        v = x["v"][ids[h // 4]].permute(0, 2, 1).reshape(-1, D)[:n].double()
        s = k @ x["q"][int(t), h].double() / math.sqrt(D)
        o = torch.softmax(s, 0) @ v
        assert abs(float(torch.logsumexp(s, 0)) - float(lse[int(t), h])) < LSE_TOL
        lim = 2.0 ** -8 * float(v.abs().max()) + 2.0 ** -8 * o.abs()
        assert bool(((out[int(t), h].double() - o).abs() <= lim).all())


def test_bad_page_ids_lengths_and_bounds_are_reported(cuda_device):
    x = batch([4, 4], [300, 300], 2, 1, 16)
    good = call(x, True)
    torch.cuda.synchronize()
    L.lynx_device_status()
    y = dict(x, table=x["table"].clone())
    y["table"][0, 0, 1] = -5
    call(y, True)
    with pytest.raises(L.LynxError, match="= 2"):
        L.lynx_device_status()
    y = dict(x, ctx=torch.tensor([300, 513], dtype=torch.int32, device="cuda"))
    call(y, True)
    with pytest.raises(L.LynxError, match="= 3"):
        L.lynx_device_status()
    y = dict(x, cu=torch.tensor([0, 4, 9], dtype=torch.int32, device="cuda"))
    out, _ = call(y, True)
    with pytest.raises(L.LynxError, match="= 6"):
        L.lynx_device_status()
    # The request with good bounds is computed.  (Not the same bits: how its keys are
    # cut into parts depends on the batch.  Both results are within check()'s bound
    # of the definition.)
    vm = float(x["v"].float()[torch.isfinite(x["v"].float())].abs().max())
    ro = oracle(x, True)[0][:4]
    assert np.all(np.abs(out[:4].double().cpu().numpy() - ro) <= 2.0 ** -8 * vm + 2.0 ** -8 * np.abs(ro))
    again = call(x, True)
    torch.cuda.synchronize()
    L.lynx_device_status()
    assert torch.equal(again[0], good[0])


def test_a_wait_that_runs_out_is_reported_and_the_context_recovers(cuda_device):
    x = batch([300, 2], [1200, 900], 4, 2, 17)
    good = call(x, True)
    torch.cuda.synchronize()
    L.lynx_device_status()
    assert L.load().lynx_test_inject_wait_timeout(1) == 0
    call(x, True)
    with pytest.raises(L.LynxError, match="= 1"):
        L.lynx_device_status()
    for _ in range(2):
        out, lse = call(x, True)
        torch.cuda.synchronize()
        L.lynx_device_status()
        assert torch.equal(out, good[0]) and torch.equal(lse, good[1])


def test_captured_graph_with_other_lengths(cuda_device):
    new, ctx = [40, 1, 90], [700, 300, 100]
    x = batch(new, ctx, 4, 2, 18, pad=30)
    out = torch.zeros(161, 4, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(161, 4, device="cuda")
    ws = torch.empty(L.lynx_chunk_attn_workspace_size(161, 3, 4, 2, D), dtype=torch.uint8, device="cuda")
    call(x, True, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(x, True, out=out, lse=lse, workspace=ws)
    for new in ([40, 1, 90], [1, 1, 1], [0, 150, 7], [100, 0, 0]):
        x["cu"].copy_(torch.tensor([0, new[0], new[0] + new[1], sum(new)]))
        g.replay()
        a = (out.clone(), lse.clone())
        check(x, True, *a)


def test_back_to_back_calls_share_a_workspace(cuda_device):
    """Calls in one stream, one behind the other, with one workspace."""
    xs = [batch([1, 30], [9000, 2000], 8, 2, 19), batch([64], [8000], 4, 4, 20), batch([1] * 5, [3000] * 5, 16, 2, 21)]
    ws = torch.empty(max(L.lynx_chunk_attn_workspace_size(x["q"].shape[0], len(x["ctx"]), x["q"].shape[1], x["Hkv"], D)
                         for x in xs), dtype=torch.uint8, device="cuda")
    single = [call(x, True) for x in xs]
    torch.cuda.synchronize()
    for _ in range(5):
        outs = [call(x, True, workspace=ws) for x in xs]
        torch.cuda.synchronize()
        for a, b in zip(single, outs):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_two_streams_with_a_workspace_each(cuda_device):
    x, y = batch([200], [3000], 8, 2, 22), batch([1] * 9, [5000] * 9, 8, 2, 23)
    a, b = call(x, True), call(y, True)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        a2, b2 = call(x, True, stream=s1), call(y, True, stream=s2)
        torch.cuda.synchronize()
        assert torch.equal(a[0], a2[0]) and torch.equal(b[0], b2[0])


def test_a_call_on_another_stream_keeps_its_own_memory(cuda_device):
    """Without a workspace, on a stream that is busy: the call returns long before it
    runs, and what torch's current stream allocates and writes meanwhile is not its
    workspace or its output."""
    x = batch([300, 1], [9000, 20000], 8, 2, 91)
    s = torch.cuda.Stream()
    m = torch.ones(4096, 4096, dtype=torch.bfloat16, device="cuda")
    size = L.lynx_chunk_attn_workspace_size(301, 2, 8, 2, D)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(100):
            m = m @ m * 2.0 ** -12
    out, lse = call(x, True, stream=s)
    for _ in range(4):
        torch.full((size,), 0x7F, dtype=torch.uint8, device="cuda")
        torch.full((301, 8, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    assert torch.cuda.current_stream() != s
    check(x, True, out, lse)


def test_workspace_and_guard_bands(cuda_device):
    """Nothing is written outside the outputs and the workspace."""
    x = batch([37, 1], [5000, 700], 8, 2, 24)
    n = 38
    size = L.lynx_chunk_attn_workspace_size(n, 2, 8, 2, D)
    ws = torch.full((size + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    out = torch.full((n + 2, 8, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n + 2, 8), 7.0, device="cuda")
    call(x, True, out=out[1:n + 1], lse=lse[1:n + 1], workspace=ws[256:256 + size])
    check(x, True, out[1:n + 1], lse[1:n + 1])
    assert (ws[:256] == 0x5A).all() and (ws[256 + size:] == 0x5A).all()
    for t in (out, lse):
        assert (t[0] == 7).all() and (t[n + 1] == 7).all()
    with pytest.raises(L.LynxError, match="workspace"):
        call(x, True, workspace=ws[256:256 + size - 16])


def test_agrees_with_the_decode_kernel(cuda_device):
    """A batch of single tokens equals lynx_decode_attn_bf16 within both roundings."""
    B, Hq, Hkv = 6, 8, 2
    x = batch([1] * B, [700, 256, 1, 1300, 2048, 511], Hq, Hkv, 25)
    x["k"] = torch.nan_to_num(x["k"], 0, 0, 0)
    x["v"] = torch.nan_to_num(x["v"], 0, 0, 0)
    o, l = call(x, True, out_dtype=torch.float32)
    table = x["table"].clamp(max=x["k"].shape[0] - 1)
    od, ld = L.lynx_decode_attn_bf16(x["q"].view(B, 1, Hq, D), x["k"], x["v"], table, x["ctx"], Hkv)
    torch.cuda.synchronize()
    L.lynx_device_status()
    vm = float(x["v"].float().abs().max())
    assert float((o.view_as(od) - od).abs().max()) <= 2.0 ** -8 * vm
    assert float((l.view_as(ld) - ld).abs().max()) <= LSE_TOL


def test_context_offsets_pass_32_bits(cuda_device):
    """Pages whose first element lies past 2^31 elements of the pool (9 GB each)."""
    n_pool = 70000
    k = torch.zeros(n_pool, D, 256, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros(n_pool, D, 256, dtype=torch.bfloat16, device="cuda")
    x = batch([5], [600], 2, 1, 26)
    for i, p in enumerate((69999, 65537, 66000)):
        src = int(x["table"][0, 0, i])
        k[p], v[p] = x["k"][src], x["v"][src]
    table = torch.tensor([[[69999, 65537, 66000]]], dtype=torch.int32, device="cuda")
    a = call(x, True)
    b = L.lynx_chunk_attn_bf16(x["q"], x["cu"], k, v, table, x["ctx"], 1)
    torch.cuda.synchronize()
    L.lynx_device_status()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("n", [131072, 400001])
def test_sums_over_long_contexts_do_not_drift(cuda_device, n):
    """2,048 tokens at the end of a long context, float32 output, sampled rows.  With p the
    row's probabilities:
      P's rounding: independent errors of at most 2^-8 p_j, 2^-8 / sqrt(3) p_j in the mean
        square; 7 standard deviations are below 4 * 2^-8 sqrt(sum p_j^2 v_j^2);
      the matrix unit's float32 sums, which are cut off and not rounded, so that their
        errors add up: a unit of 2^-23 for each of 1,024 additions of 16 keys, after which
        the sum is taken out and added up rounded: 2^-13 sum p_j |v_j|;
      scores and all else in float32: 2^-15 sum p_j |v_j|."""
    T, Hq, Hkv = 2048, 16, 4
    x = batch([T], [n], Hq, Hkv, n)
    v = x["v"]
    v.copy_(torch.where(torch.isfinite(v), v.abs() + 0.1, v))     # one sign: what is cut off adds up
    out, lse = call(x, True, out_dtype=torch.float32)
    torch.cuda.synchronize()
    L.lynx_device_status()
    rng = np.random.default_rng(n)
    ids = x["table"][0].long()
    err = []
    for t in [0, 1, T - 1, *rng.integers(0, T, 20)]:
        h = int(rng.integers(0, Hq))
        seen = n - T + int(t) + 1
        k = x["k"][ids[h // 4]].permute(0, 2, 1).reshape(-1, D)[:seen].double()
        v = x["v"][ids[h // 4]].permute(0, 2, 1).reshape(-1, D)[:seen].double()
        s = k @ x["q"][int(t), h].double() / math.sqrt(D)
        p = torch.softmax(s, 0)
        o, d = p @ v, out[int(t), h].double() - p @ v
        lim = 2.0 ** -6 * torch.sqrt(p.square() @ v.square()) + (2.0 ** -13 + 2.0 ** -15) * (p @ v.abs())
        assert bool((d.abs() <= lim).all()), float((d.abs() / lim).max())
        assert abs(float(torch.logsumexp(s, 0)) - float(lse[int(t), h])) < LSE_TOL
        err.append(float((d / o).mean()))
    # and together: P's rounding falls out of the mean over rows and channels
    assert abs(np.mean(err)) < 2.0 ** -13 + 2.0 ** -15


@pytest.mark.parametrize("shape", ["up", "down", "late", "flat"])
@pytest.mark.parametrize("new,n", [([1] * 200, 40000), ([100] * 80, 33000)])
def test_sums_that_are_taken_out_follow_the_running_maximum(cuda_device, new, n, shape):
    """So many requests over one long context that a CTA goes through tens of thousands of
    keys: its sums are taken out against one maximum and go on against another.  One
    group of rows a tile, and both.  The bound is that of the test above."""
    Hq, Hkv, B = 2, 1, len(new)
    x = batch([sum(new)], [n], Hq, Hkv, n)
    ids = x["table"][0, 0].long()
    pos = torch.arange(ids.numel() * 256, device="cuda").float()
    ramp = {"up": pos / 1000, "down": -pos / 1000, "late": 40.0 * (pos == n - 7000), "flat": 0 * pos}[shape]
    k = x["k"][ids]
    k[:, 0, :] = torch.where(torch.isfinite(k[:, 0, :].float()), ramp.view(-1, 256).bfloat16(), k[:, 0, :])
    x["k"][ids] = k
    x["q"][:, :, 0] = 8.0
    x["cu"] = torch.tensor([sum(new[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda")
    x["ctx"] = torch.full((B,), n, dtype=torch.int32, device="cuda")
    x["table"] = x["table"].expand(B, -1, -1).contiguous()
    size = L.lynx_chunk_attn_workspace_size(sum(new), B, Hq, Hkv, D)
    ws = torch.full((size + 512,), 0xFF, dtype=torch.uint8, device="cuda")     # NaN in every place
    a = call(x, True, out_dtype=torch.float32, workspace=ws[256:256 + size])
    torch.cuda.synchronize()
    L.lynx_device_status()
    assert (ws[:256] == 0xFF).all() and (ws[256 + size:] == 0xFF).all()
    b = call(x, True, out_dtype=torch.float32)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    keys = x["k"][ids].permute(0, 2, 1).reshape(-1, D).double()
    vals = x["v"][ids].permute(0, 2, 1).reshape(-1, D).double()
    for i, r in enumerate(np.random.default_rng(n).integers(0, sum(new), 30)):
        t = int(r) % new[0]
        seen = n - new[0] + t + 1
        s = keys[:seen] @ x["q"][int(r), i % 2].double() / math.sqrt(D)
        p, v = torch.softmax(s, 0), vals[:seen]
        d = (a[0][int(r), i % 2].double() - p @ v).abs()
        # scores here go up to 8 * 40 / sqrt(128) = 28 more: 128 additions of 2^-24 of that
        lim = 2.0 ** -6 * torch.sqrt(p.square() @ v.square()) + (2.0 ** -13 + 2.0 ** -15 + 2.0 ** -12) * (p @ v.abs())
        assert bool((d <= lim).all()), float((d / lim).max())
        assert abs(float(torch.logsumexp(s, 0)) - float(a[1][int(r), i % 2])) < 2 * LSE_TOL


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,ctx,Hq,Hkv", [
    ([1], [50001], 8, 2), ([3, 40], [50001, 20000], 8, 2), ([300, 1], [5000, 9000], 6, 3), ([700], [3000], 4, 1),
    ([64] * 5, [1999, 128, 4097, 640, 777], 16, 4), ([1] * 70, [1 + 53 * i for i in range(70)], 4, 2)])
def test_every_tile_and_every_key_has_its_weight(cuda_device, new, ctx, Hq, Hkv, causal):
    """Values that tell the keys apart.  1 in channel c for the keys of tile c (of 128
    tiles at a time): the output is the tiles' probabilities, so that a tile left out, taken
    twice or from another page is off by all of it.  Then 1 in channel c for key c of
    every tile.  Sums of probabilities, each rounded to BF16 (half a step: 2^-8 of it), 2^-12
    for everything in float32 and what the matrix unit cuts off."""
    x = batch(new, ctx, Hq, Hkv, sum(ctx) + Hq)
    n_tiles = max(-(-c // 128) for c in ctx)
    masks = range(-(-n_tiles // 128) + 1)
    eye = torch.eye(128, dtype=torch.bfloat16, device="cuda")
    outs = []
    for w in masks:
        v = torch.zeros_like(x["v"])
        for b, n in enumerate(ctx):
            pages = -(-n // 256)
            if w == masks[-1]:
                one = torch.cat([eye, eye], 1).expand(pages, -1, -1)
            else:
                tile = torch.arange(2 * pages, device="cuda") - 128 * w            # of each half page
                one = (tile.view(-1, 2, 1) == torch.arange(128, device="cuda")).bfloat16()
                one = one.permute(0, 2, 1).repeat_interleave(128, 2)
            for h in range(Hkv):
                v[x["table"][b, h, :pages].long()] = one
        outs.append(call(dict(x, v=v), causal, out_dtype=torch.float32)[0].double())
    torch.cuda.synchronize()
    L.lynx_device_status()
    lo = 0
    for b, (T, n) in enumerate(zip(new, ctx)):
        seen = (n - T + 1 + torch.arange(T, device="cuda")).clamp(min=0) if causal else torch.full((T,), n, device="cuda")
        for hq in range(Hq):
            ids = x["table"][b, hq // (Hq // Hkv), :-(-n // 256)].long()
            k = x["k"][ids].permute(0, 2, 1).reshape(-1, D)[:n].double()
            s = x["q"][lo:lo + T, hq].double() @ k.T / math.sqrt(D)
            s = s.masked_fill(torch.arange(n, device="cuda") >= seen[:, None], -math.inf)
            p = torch.nan_to_num(torch.softmax(s, 1))                              # a row without keys: 0
            p = torch.nn.functional.pad(p, (0, n_tiles * 128 - n)).view(T, n_tiles, 128)
            ref = [torch.nn.functional.pad(p.sum(2), (0, 128 * (len(masks) - 1) - n_tiles)).view(T, -1, 128)[:, w]
                   for w in masks[:-1]] + [p.sum(1)]
            for o, r in zip(outs, ref):
                err = (o[lo:lo + T, hq] - r).abs()
                assert bool((err <= (2.0 ** -8 + 2.0 ** -12) * r + 1e-9).all()), (b, hq, float((err - r / 256).max()))
        lo += T
