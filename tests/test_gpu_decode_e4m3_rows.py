"""Decode and verification attention over pages in 8 bits, each row against bounds of its own."""
import math

import numpy as np
import pytest
import torch

from e4m3_testutil import Cache, attention_and_bounds, equal_keys_case, far_key_case, small_channels_case
from oracle import e4m3
from progressive_kv_quantization_gb300 import lynx as L
from test_gpu_decode_e4m3 import queries, run

pytestmark = pytest.mark.gpu
SCALE = 1 / math.sqrt(128)


def check_rows(cache, q, ctx, causal, out, lse, scale=SCALE):
    B, T, Hq, _ = q.shape
    G = Hq // cache.Hkv
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(B):
        seen = [ctx[b] - T + i + 1 if causal else ctx[b] for i in range(T) for _ in range(G)]
        for h in range(cache.Hkv):
            k, v = cache.values(b, h)
            rows = q[b, :, h * G:(h + 1) * G].reshape(T * G, 128)
            ro, rl, off_o, off_l = attention_and_bounds(rows, k, v, scale, seen)
            assert np.all(np.abs(out[b, :, h * G:(h + 1) * G].reshape(T * G, 128) - ro) <= off_o), (b, h)
            l, none = lse[b, :, h * G:(h + 1) * G].reshape(-1), np.isneginf(rl)
            assert np.array_equal(none, np.isneginf(l)), (b, h)
            assert np.all(np.abs(l[~none] - rl[~none]) <= off_l[~none]), (b, h)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Hq,Hkv,T", [(8, 2, 1), (9, 1, 1), (16, 2, 2), (16, 4, 5), (4, 1, 6), (8, 1, 8)])
def test_blocks_of_very_different_scales(Hq, Hkv, T, causal):
    """Neighbouring blocks and pages up to 2^24 apart, over some thousand keys, in tiles of 8, 16 and 24
    rows: a block under another one's scale is off by powers of two."""
    lens = [5000, 3333, 257]
    cache = Cache(lens, Hkv, seed=Hq + T, spread=12)
    q = queries((len(lens), T, Hq, 128), 2, size=2.0 ** -9)
    for _ in range(3):
        out, lse = run(cache, q, lens, causal)
        check_rows(cache, q, lens, causal, out, lse)
    L.lynx_device_status()


@pytest.mark.parametrize("Hq,T", [(8, 1), (4, 4), (8, 3), (5, 9)])
@pytest.mark.parametrize("scale,low,high", [(2.0 ** -120, 100, 127), (2.0 ** -100, 60, 127), (2.0 ** 100, -126, -90), (1.0, -60, 20)])
def test_rows_of_all_sizes_over_one_key(Hq, T, scale, low, high):
    """One key: the lse is the score, the output the value; sizes from BF16's smallest normal to its largest number.

    Scores below 2^23: the maximum is a score rounded once, off by 2^-24 of it, and with a lead of 2^5 over the running
    one p 2^10 has to stay below FP16's 65,504."""
    cache = Cache([1] * 20, 1, seed=23)
    rng = np.random.default_rng(24)
    q = rng.uniform(0.5, 1.0, (20, T, Hq, 128)) * rng.choice([-1, 1], (20, T, Hq, 128))
    q = q * np.exp2(rng.integers(low, high + 1, (20, T, Hq, 1)).astype(float))
    q[3::4] *= np.exp2(-rng.integers(0, 24, (5, T, Hq, 128)).astype(float))
    q[1, 0, 0] = 0
    q = np.where(np.abs(q) < 2.0 ** -126, 0.0, q)
    q = queries_of(q)
    out, lse = run(cache, q, [1] * 20, False, sm_scale=scale)
    L.lynx_device_status()
    held = 0
    for b in range(20):
        k, v = cache.values(b, 0)
        rows = q[b].reshape(-1, 128)
        fits = np.abs(scale * rows @ k[0]) < 2.0 ** 23
        held += fits.mean() / 20
        ro, rl, off_o, off_l = attention_and_bounds(rows[fits], k, v, scale, [1] * int(fits.sum()))
        o, l = (t[b].double().cpu().numpy() for t in (out, lse))
        assert np.all(np.abs(o.reshape(-1, 128)[fits] - ro) <= off_o)
        assert np.all(np.abs(l.reshape(-1)[fits] - rl) <= off_l)
    assert held > 0.5


def queries_of(x):
    return torch.from_numpy(x.astype(np.float32)).bfloat16().double().numpy()


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("Hq,T,n", [(4, 1, 1), (4, 2, 300), (6, 4, 9000), (8, 3, 2)])
def test_a_row_that_is_not_finite_is_nan(Hq, T, n, bad):
    """Over few keys and many, and nothing but that row; without a key it is 0."""
    cache = Cache([n], 1, seed=25)
    q = queries((1, T, Hq, 128), 26)
    with np.errstate(invalid="ignore"):
        sick = q.copy()
        sick[0, T - 1, 1, 77] = bad
        sick[0, 0, Hq - 1, 3] = bad
    out, lse = run(cache, sick, [n], True)
    L.lynx_device_status()
    for t, h in ((T - 1, 1), (0, Hq - 1)):
        if n - T + t + 1 > 0:
            assert out[0, t, h].isnan().all() and lse[0, t, h].isnan()
        else:
            assert (out[0, t, h] == 0).all() and lse[0, t, h] == -math.inf
        out[0, t, h], lse[0, t, h] = (x[0, t, h] for x in run(cache, q, [n], True))
    check_rows(cache, q, [n], True, out, lse)


@pytest.mark.parametrize("scale", [0.02, 0.04, 0.07, 0.1, 0.2])
@pytest.mark.parametrize("T", [1, 3, 5])
def test_sums_over_long_contexts_do_not_drift(T, scale):
    """131,072 keys that one CTA sums by itself, all but the first page's the same, so that the roundings go
    one way.  In each 32 keys of the first page one has the lead, and the others' p is no round number.

    A row's sum gets one addition a unit of 128 keys, 1,024 in all, each off by 2^-24 of the sum so far
    at most, half of that over all: 2^-15; O's the same.  And what attention_and_bounds counts for the
    scores (of 16 |q| |k| 2^-23) and the exponentials (2^-18)."""
    n, B, Hkv, G = 131072, 304, 2, 4         # two items a CTA of two an SM
    codes = np.full((3, 256, 128), 0x38, dtype=np.uint8)           # keys of ones
    codes[1, ::32] = 0x39                                          # and of 1.125
    rng = np.random.default_rng(27)
    values = rng.integers(0x30, 0x48, (3, 256, 128), dtype=np.uint8)   # 0.5 .. 3.75
    scales = np.full((3, 2, 8), 127, dtype=np.uint8)
    table = torch.full((B, Hkv, n // 256), 2, dtype=torch.int32, device="cuda")
    table[:, :, 0] = 1
    up = lambda a: torch.from_numpy(a).cuda()
    q = torch.full((B, T, G * Hkv, 128), 0.125, dtype=torch.bfloat16, device="cuda")
    out, lse = L.lynx_decode_attn_e4m3(q, up(codes).view(torch.float8_e4m3fn), up(values).view(torch.float8_e4m3fn), up(scales),
                                       table, torch.full((B,), n, dtype=torch.int32, device="cuda"), Hkv, sm_scale=scale)
    L.lynx_device_status()
    scale = float(np.float32(scale))
    w = np.where(np.arange(256) % 32 == 0, np.exp(scale * 18.0), np.exp(scale * 16.0))[:, None]
    first, other = e4m3.decode(values[1]), e4m3.decode(values[2])
    total = w.sum() + (n - 256) * math.exp(scale * 16.0)
    want = ((w * first).sum(0) + math.exp(scale * 16.0) * (n // 256 - 1) * other.sum(0)) / total
    e = 16 * 2.0 ** -23 * scale * 18.0 + 2.0 ** -18
    assert np.abs(lse.double().cpu().numpy() - math.log(total)).max() <= e + 2.0 ** -15 + 2.0 ** -22 * math.log(total)
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= (2 * e + 2.0 ** -14) * want)


def test_the_keys_far_below_the_largest_count():
    cache, q, scale = far_key_case()
    out, lse = run(cache, q, [20001], False, sm_scale=scale)
    check_rows(cache, q, [20001], False, out, lse, scale)


@pytest.mark.parametrize("rows", [4, 12, 20])
def test_both_halves_of_a_probability_count(rows):
    cache, q, scale = equal_keys_case(rows)
    out, lse = run(cache, q, [2000], False, sm_scale=scale)
    check_rows(cache, q, [2000], False, out, lse, float(np.float32(scale)))


def test_small_channels_count():
    cache, q, scale = small_channels_case()
    out, lse = run(cache, q, [777], False, sm_scale=scale)
    check_rows(cache, q, [777], False, out, lse, scale)


@pytest.mark.parametrize("key_size", [-8, 0, 8, 30, 60])
@pytest.mark.parametrize("Hq", [8, 14, 22])
def test_rows_of_other_sizes_in_one_tile(Hq, key_size):
    """Keys of the size that makes the scores of some of the rows ordinary ones."""
    cache = Cache([777], 1, seed=9)
    cache.scales[0][:] = np.clip(cache.scales[0].astype(int) + key_size, 0, 255)
    q = queries((1, 1, Hq, 128), 10) * np.resize(2.0 ** np.array([0, 8, -8, -30, -60, -4, -1, -28]), Hq)[:, None]
    q[0, 0, 7] = 0.0
    rows = np.log2(np.abs(q[0, 0]).max(-1), where=q[0, 0].any(-1), out=np.full(Hq, -99.0)) + key_size < 5
    out, lse = run(cache, q, [777], False)
    k, v = cache.values(0, 0)
    ro, rl, off_o, off_l = attention_and_bounds(q[0, 0], k, v, SCALE, [777] * Hq)
    o, l = out[0, 0].double().cpu().numpy(), lse[0, 0].double().cpu().numpy()
    # larger scores than some hundreds make one key of them all, which a rounding of the scores decides
    assert np.all((np.abs(o - ro) <= off_o)[rows]) and np.all((np.abs(l - rl) <= off_l)[rows])
    fits = np.abs(SCALE * q[0, 0] @ k.T).max(-1) < 2.0 ** 23
    assert np.isfinite(o[fits]).all() and np.all((np.abs(l - rl) <= off_l)[fits])
