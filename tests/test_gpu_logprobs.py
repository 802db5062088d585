"""lynx_token_logprobs against float64: sizes from one token to the largest vocabulary,
rows at any place, ties, masked logits, rows of nothing else."""
import math

import numpy as np
import pytest
import torch

from oracle import serving as sv
from progressive_kv_quantization_gb300 import lynx as L

pytestmark = pytest.mark.gpu


def check(x, tokens, n_top, got, rows=None):
    """Differences x - max are rounded once (2^-24 of up to the row's range), the exponential is off
    by 2^-21 of itself, sums of up to 2^24 terms in 2,048 threads by some 2^-18: so ln s by 2^-17 with
    room, a log probability by that and two roundings of its own; the entropy's mean of differences
    by 2^-17 of its range."""
    torch.cuda.synchronize()
    logprob, entropy, ids, top = (t.double().cpu().numpy().reshape(x.shape[0], *t.shape[t.dim() - (1 if i > 1 else 0):])
                                  for i, t in enumerate(got))
    xd = x.double().cpu().numpy()
    ro, rh, ri, rt = sv.token_logprobs(xd, tokens.cpu().numpy().reshape(-1), n_top)
    assert np.array_equal(ids, ri)
    for g, r in ((logprob, ro), (top, rt)):
        none = np.isneginf(r)
        assert np.array_equal(none, np.isneginf(g))
        assert np.all(np.abs(g - r)[~none] <= 2.0 ** -17 + 2.0 ** -22 * np.abs(r[~none]))
    fin = np.where(np.isfinite(xd), xd, 0)
    span = np.minimum(fin.max(1) - fin.min(1), 100.0) + 1
    assert np.all(np.abs(entropy - rh) <= 2.0 ** -17 * span) and np.all(entropy >= 0)


def logits(N, V, dtype, seed, size=2.5):
    g = torch.Generator("cuda").manual_seed(seed)
    x = (torch.randn(N, V, generator=g, device="cuda") * size).to(dtype)
    tokens = torch.randint(0, V, (N,), generator=g, device="cuda").to(torch.int32)
    return x, tokens


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,V", [(1, 1), (3, 2), (5, 7), (4, 31), (2, 33), (7, 257), (3, 1000), (2, 2049), (5, 8191), (1, 32000),
                                 (3, 50257), (2, 151936), (700, 600), (1, 1 << 20)])
def test_sizes(cuda_device, N, V, dtype):
    x, tokens = logits(N, V, dtype, V)
    for n_top in sorted({0, min(1, V), min(5, V), min(20, V), min(32, V)}):
        check(x, tokens, n_top, L.lynx_token_logprobs(x, tokens, n_top))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset", [1, 2, 3, 5, 7])
def test_rows_at_any_place(cuda_device, dtype, offset):
    """Rows that begin between multiples of 16 bytes, in a wider buffer; the same bits as in one of their own."""
    for N, V in ((3, 4001), (2, 3), (1, 70001)):
        wide, tokens = logits(N, V + 13, dtype, offset)
        x = wide[:, offset:offset + V]
        got = L.lynx_token_logprobs(x, tokens.clamp(max=V - 1), min(8, V))
        check(x, tokens.clamp(max=V - 1), min(8, V), got)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ties_go_to_the_lowest(cuda_device, dtype):
    V = 9000
    equal = torch.zeros(1, V, dtype=dtype, device="cuda")
    few = torch.randint(0, 3, (1, V), device="cuda").to(dtype)
    zeros = torch.where(torch.arange(V, device="cuda") % 2 == 0, 0.0, -0.0)[None].to(dtype)   # -0 is 0
    steps = (torch.arange(V, device="cuda") // 100)[None].to(dtype)
    back = steps.flip(1).contiguous()
    x = torch.cat([equal, few, zeros, steps, back])
    tokens = torch.arange(5, dtype=torch.int32, device="cuda")
    for n_top in (1, 7, 32):
        check(x, tokens, n_top, L.lynx_token_logprobs(x, tokens, n_top))
    big = torch.zeros(1, 300000, dtype=dtype, device="cuda")
    check(big, tokens[:1], 32, L.lynx_token_logprobs(big, tokens[:1], 32))


def test_most_of_the_largest_in_one_place(cuda_device):
    """All the large logits among one thread's pieces, rising and falling: more reach the first bound than find room."""
    V = 1 << 20
    for rising in (True, False):
        x = torch.full((1, V), -50.0, device="cuda")
        i = torch.arange(V, device="cuda")
        mine = (i // 4) % 256 == 77              # one thread's pieces, in any split into CTAs of whole 1024s
        order = torch.arange(int(mine.sum()), device="cuda", dtype=torch.float32) * 2.0 ** -8
        x[0, mine] = order if rising else order.flip(0)
        # so that the bound of the other groups is far below
        x[0, (i // 4) % 256 // 4 != 77 // 4] -= torch.rand(int(((i // 4) % 256 // 4 != 77 // 4).sum()), device="cuda")
        tokens = torch.tensor([77 * 4], dtype=torch.int32, device="cuda")
        check(x, tokens, 32, L.lynx_token_logprobs(x, tokens, 32))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_masked_logits(cuda_device, dtype):
    """-inf and the type's lowest value in most places, all but one place, and all places."""
    V = 5000
    low = torch.finfo(dtype).min
    x, tokens = logits(9, V, dtype, 3)
    keep = torch.rand(9, V, device="cuda") < 0.01
    x[:3] = torch.where(keep[:3], x[:3], -math.inf)
    x[3] = -math.inf
    x[3, 4321] = 2.0
    x[4] = -math.inf
    x[5] = torch.where(keep[5], x[5], low)
    x[6] = low
    x[7] = low
    x[7, 17] = -3.0
    x[8, :4990] = -math.inf
    x[8, 4990:] = low
    tokens[3], tokens[7], tokens[8] = 4321, 17, 4995
    for n_top in (0, 4, 32):
        got = L.lynx_token_logprobs(x, tokens, n_top)
        check(x, tokens, n_top, got)
    assert got[1][4] == 0 and abs(float(got[1][6]) - math.log(V)) < 1e-4


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_row_with_nan_or_infinity_is_nan(cuda_device, bad):
    x, tokens = logits(4, 40000, torch.float32, 4)
    x[1, 39999] = bad
    x[2, 123] = bad
    logprob, entropy, ids, _ = L.lynx_token_logprobs(x, tokens, 3)
    for r in (1, 2):
        assert math.isnan(logprob[r]) and math.isnan(entropy[r])
    keep = [0, 3]
    check(x[keep], tokens[keep], 3, [t[keep] for t in L.lynx_token_logprobs(x, tokens, 3)])
    assert ((ids >= 0) & (ids < 40000)).all()


@pytest.mark.parametrize("V", [40, 3000, 200000])
def test_rows_with_too_few_numbers(cuda_device, V):
    """Fewer values than alternatives that are not NaN: every output is written all the same."""
    x = torch.full((4, V), math.nan, device="cuda")
    x[1, 7] = 1.0
    x[2, V - 5:] = torch.arange(5.0, device="cuda")
    x[3] = torch.randn(V, device="cuda")
    tokens = torch.zeros(4, dtype=torch.int32, device="cuda")
    out = dict(logprob=torch.zeros(4, device="cuda"), entropy=torch.zeros(4, device="cuda"),
               top_ids=torch.full((4, 20), -7, dtype=torch.int32, device="cuda"), top_logprobs=torch.zeros(4, 20, device="cuda"))
    L.lynx_token_logprobs(x, tokens, 20, **out)
    assert out["top_logprobs"][:3].isnan().all() and out["entropy"][:3].isnan().all() and out["logprob"][:3].isnan().all()
    assert ((out["top_ids"] >= 0) & (out["top_ids"] < V)).all()
    check(x[3:], tokens[3:], 20, [t[3:] for t in out.values()])


@pytest.mark.parametrize("N,V", [(1, 1 << 22), (2, 151936), (700, 70001)])
def test_rising_values(cuda_device, N, V):
    """The bound from the front of a row holds nothing back behind it."""
    x = (torch.arange(V, device="cuda", dtype=torch.float32) * 2.0 ** -12).expand(N, V).contiguous()
    x[-1] = x[-1].flip(0)
    tokens = torch.full((N,), V - 1, dtype=torch.int32, device="cuda")
    for n_top in (1, 32):
        got = L.lynx_token_logprobs(x, tokens, n_top)
        rows = sorted({0, N - 1})
        check(x[rows], tokens[rows], n_top, [t[rows] for t in got])


def test_one_token_with_almost_all_weight(cuda_device):
    """Log probabilities near 0 keep their relative precision, down to what float32's sum holds."""
    x, tokens = logits(3, 30000, torch.float32, 5, size=1.0)
    tokens[:] = 777
    for r, lead in enumerate((15.0, 20.0, 60.0)):
        x[r, 777] = lead
    got = L.lynx_token_logprobs(x, tokens, 2)
    check(x, tokens, 2, got)
    assert (got[0] <= 0).all() and got[0][2] == 0 and got[2][:, 0].eq(777).all()


def test_large_values_and_ids_outside(cuda_device):
    x, _ = logits(4, 1000, torch.float32, 6, size=1e6)
    tokens = torch.tensor([-1, 1000, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    got = L.lynx_token_logprobs(x, tokens, 1)
    assert torch.isneginf(got[0]).all()
    check(x, tokens, 1, got)


def test_three_dimensions_outputs_stream_and_graph(cuda_device):
    """Behind verification: [B, T + 1, V] with -1 behind the last token; buffers and a stream of the caller's."""
    x, _ = logits(12, 3000, torch.bfloat16, 7)
    tokens = torch.randint(0, 3000, (3, 4), device="cuda").to(torch.int32)
    tokens[1, 2:] = -1
    out = dict(logprob=torch.empty(3, 4, device="cuda"), entropy=torch.empty(3, 4, device="cuda"),
               top_ids=torch.empty(3, 4, 5, dtype=torch.int32, device="cuda"), top_logprobs=torch.empty(3, 4, 5, device="cuda"))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = L.lynx_token_logprobs(x.view(3, 4, 3000), tokens, 5, stream=stream, **out)
    torch.cuda.current_stream().wait_stream(stream)
    assert all(a is b for a, b in zip(got, out.values()))
    flat = lambda: [t.view(12, *t.shape[2:]) for t in got]
    check(x, tokens, 5, flat())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.lynx_token_logprobs(x.view(3, 4, 3000), tokens, 5, **out)
    for seed in (8, 9):
        x.copy_(logits(12, 3000, torch.bfloat16, seed)[0])
        tokens.copy_(torch.randint(0, 3000, (3, 4), device="cuda"))
        for t in out.values():
            t.zero_()
        graph.replay()
        check(x, tokens, 5, flat())


def test_empty_and_refusals(cuda_device):
    x, tokens = logits(4, 100, torch.float32, 10)
    none = L.lynx_token_logprobs(x[:0], tokens[:0], 3)
    assert none[0].shape == (0,) and none[2].shape == (0, 3)
    good = dict(logits=x, tokens=tokens, n_top=3)
    for change, word in [
            (dict(logits=x.half()), "logits"), (dict(logits=x[0]), "logits"), (dict(logits=x.t()), "logits"), (dict(logits=x.cpu()), "CUDA"),
            (dict(logits=torch.zeros(4, 4, 100, device="cuda")[:, :2], tokens=torch.zeros(4, 2, dtype=torch.int32, device="cuda")), "stride"),
            (dict(tokens=tokens.long()), "tokens"), (dict(tokens=tokens[:3]), "tokens"), (dict(n_top=-1), "n_top"),
            (dict(n_top=33), "n_top"), (dict(logits=x[:, :2], n_top=3), "n_top"), (dict(logprob=torch.empty(3, device="cuda")), "logprob"),
            (dict(top_ids=torch.empty(4, 3, device="cuda")), "top_ids"), (dict(entropy=x.view(-1)[:4]), "overlaps"),
            (dict(top_logprobs=tokens.view(torch.float32).expand(4, 4)[:, :3]), "top_logprobs")]:
        with pytest.raises(L.LynxError, match=word):
            L.lynx_token_logprobs(**{**good, **change})
    L.lynx_device_status()
