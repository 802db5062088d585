"""Decode and verification attention over pages in 8 bits, each row against bounds of its own."""
import math

import numpy as np
import pytest
import torch

from e4m3_testutil import Cache, attention_and_bounds
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
