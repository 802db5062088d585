"""lynx_chunk_attn_e4m3 with query rows of every size side by side in a tile, each against
bounds of its own."""
import math

import numpy as np
import pytest
import torch

from progressive_kv_quantization_gb300 import lynx as L
from test_gpu_chunk_attn import oracle
from test_gpu_chunk_e4m3 import batch8, call8

pytestmark = pytest.mark.gpu


def score_errors(x, scale):
    """Of each row and key of a batch of one request: a query row is held down to 2^-9 of its largest
    value exactly and to 2^-17 of that below, and of the float32 sum of 128 products each addition is
    off by 2^-23 of the sum of magnitudes at most; two roundings of the scale."""
    q = x["q"].double().cpu().numpy()
    n, Hq, _ = q.shape
    G = Hq // x["Hkv"]
    ctx = int(x["ctx"][0])
    ids = x["table"][0, :, :-(-ctx // 256)].long().cpu().numpy()
    k = x["k"].double().cpu().numpy()[ids].transpose(0, 1, 3, 2).reshape(x["Hkv"], -1, 128)[:, :ctx]
    v = x["v"].double().cpu().numpy()[ids].transpose(0, 1, 3, 2).reshape(x["Hkv"], -1, 128)[:, :ctx]
    s, off, vs = [], [], []
    for h in range(Hq):
        kh, size = k[h // G], np.abs(q[:, h])
        s.append(scale * q[:, h] @ kh.T)
        top = np.maximum(size.max(-1, keepdims=True), 2.0 ** -119)
        rest = np.where(size < 2.0 ** -9 * top, 2.0 ** -17 * top, 0.0)
        off.append(scale * (rest @ np.abs(kh).T + 130 * 2.0 ** -23 * (size @ np.abs(kh).T)))
        vs.append(v[h // G])
    return np.stack(s, 1), np.stack(off, 1), np.stack(vs)


@pytest.mark.parametrize("scale,low,high", [(2.0 ** -100, 0, 127), (2.0 ** -120, 100, 127), (2.0 ** 20, -126, 0), (1.0, -60, 60)])
def test_rows_of_all_sizes_over_one_key(cuda_device, scale, low, high):
    """One key: the lse is the score, the output the value; sizes from BF16's smallest normal to its largest number."""
    x = batch8([300], [1], 3, 1, high - low, spread=False)
    rng = np.random.default_rng(1)
    size = np.exp2(rng.integers(low, high + 1, (300, 3, 1)).astype(float))
    q = rng.uniform(0.5, 1.0, (300, 3, 128)) * rng.choice([-1, 1], (300, 3, 128)) * size
    q[::7] *= np.exp2(-rng.integers(0, 24, (43, 3, 128)).astype(float))      # channels far below the row's largest
    q[5], q[140, 1] = 0, 0
    q[6, 2, :127] = 0
    x["q"] = torch.from_numpy(q.astype(np.float32)).cuda().bfloat16()
    out, lse = call8(x, False, sm_scale=scale, out_dtype=torch.float32)
    L.lynx_device_status()
    s, off, v = score_errors(x, scale)
    lse = lse.double().cpu().numpy()
    # Scores below 2^30 only.  (The maximum is the score rounded once, m (1 + r) with |r| <= 2^-24, and P
    # 2^(-m r): past 2^128, which float32 does not hold, from scores of 2^31 on.)
    held = np.abs(s[:, :, 0]) < 2.0 ** 30
    assert held.mean() > 0.4
    # (a block's factor is at least float32's smallest normal number, on sums of up to 2^24)
    assert np.all((np.abs(lse - s[:, :, 0]) <= off[:, :, 0] + 2.0 ** -22 * np.abs(s[:, :, 0]) + 2.0 ** -102)[held])
    # P is not 1 but 2^(-m r), off by 2^-24 |score| in natural units.  The sum takes it as it is, the
    # product rounded to BF16: to 1 while it is less than half a step off, by half a step of 2^-8 at most
    # behind that.  And the exponential's 2^-22, the sum's inverse and a rounding.
    one = np.broadcast_to(v[:, 0], (300, 3, 128))
    limit = np.minimum(2.0 ** -8, 2.0 ** -23 * np.abs(s[:, :, 0])) + 2.0 ** -21
    assert np.all((np.abs(out.double().cpu().numpy() - one) <= limit[:, :, None] * np.abs(one))[held])


@pytest.mark.parametrize("causal", [True, False])
def test_rows_of_many_sizes_over_many_keys(cuda_device, causal):
    """The softmax of small and large rows, rows of zeros and rows with outlier channels in one tile."""
    scale = 1 / math.sqrt(128)
    x = batch8([120], [500], 4, 1, 2)
    rng = np.random.default_rng(3)
    q = rng.standard_normal((120, 4, 128)) * np.exp2(rng.integers(-20, 2, (120, 4, 1)))
    q[::5, :, 17] *= 64                     # the other channels keep all their bits: 2^-6 and less of the largest
    q[3::5, :, 90] = 2000                   # they fall below 2^-9 of it
    q[::11] = 0
    x["q"] = torch.from_numpy(q.astype(np.float32)).cuda().bfloat16()
    out, lse = call8(x, causal, out_dtype=torch.float32)
    L.lynx_device_status()
    ro, rl = oracle(x, causal, scale)
    s, off, v = score_errors(x, scale)
    seen = np.arange(500) < (np.arange(381, 501)[:, None] if causal else np.full((120, 1), 500))
    e = np.where(seen[:, None], off, 0).max(-1) + 2.0 ** -18           # and the exponential's 2^-21, sums and roundings
    p = np.exp(np.where(seen[:, None], s - rl[:, :, None], -np.inf))
    assert np.all(np.abs(lse.double().cpu().numpy() - rl) <= e + 2.0 ** -22 * np.abs(rl))
    # P to half a step of BF16; the scores' error in P and in its sum, where it is one to first order
    limit = np.einsum("nhk,hkc->nhc", p, np.abs(v)) * (2.0 ** -8 + 2 * e[:, :, None] * (1 + e[:, :, None]))
    some = e < 0.5                          # not the 22 of 120 tokens with 2000, 2^-17 of which is 2^-6
    assert some.mean() > 0.8
    assert np.all((np.abs(out.double().cpu().numpy() - ro) <= limit)[some])


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("ctx", [1, 300, 20000])
def test_a_row_that_is_not_finite_is_nan(cuda_device, bad, ctx):
    """As over BF16 pages, and nothing but that row; without a key it is 0.

    The rows of a warp follow their maxima together, so that a row whose own does not move any more may
    leave the others' P against another reference: both results are within the kernel's bounds (2^-8
    of the values for P's rounding, 2^-11 of the scores for float32's sums), not the same bits."""
    x = batch8([150], [ctx], 2, 1, 4)
    good = [t.clone() for t in call8(x, out_dtype=torch.float32)]
    rows = [149, 148, 100, 0]
    for i, r in enumerate(rows):
        x["q"][r, i % 2, 5 + i] = bad
    out, lse = call8(x, out_dtype=torch.float32)
    L.lynx_device_status()
    for r in range(150):
        for h in range(2):
            if r in rows and h == rows.index(r) % 2:
                sees = ctx - 150 + r + 1 > 0
                assert out[r, h].isnan().all() and lse[r, h].isnan() if sees else (out[r, h] == 0).all() and lse[r, h] == -math.inf
            else:
                assert (out[r, h] - good[0][r, h]).abs().max() <= 2 * 2.0 ** -8 * x["v"].float().abs().max()
                assert lse[r, h] == good[1][r, h] or abs(lse[r, h] - good[1][r, h]) <= 2 * 2.0 ** -11
