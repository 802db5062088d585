"""lynx_qkv_append_e4m3 of rows with NaN: the block's other tokens are as without them."""
import numpy as np
import pytest
import torch

from oracle import e4m3
from oracle import serving as sv
from progressive_kv_quantization_gb300 import lynx as L
from test_gpu_append_e4m3 import call, case, pools_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("everywhere", [True, False])
@pytest.mark.parametrize("reqs", [[(40, 1), (0, 1), (31, 1)], [(5, 70), (0, 33)], [(0, 1)] * 20 + [(3, 50)]])
def test_nan_leaves_the_other_tokens_their_scale(cuda_device, reqs, everywhere):
    """Whole rows of NaN, and single channels; a decode step, chunks, runs behind a CTA's first 32 rows."""
    c = case(reqs, 2, 2, len(reqs), norm=False, rot=0)
    n = c["qkv"].shape[0]
    sick = np.unique(np.r_[0, n // 2, n - 1])
    x = c["qkv"].clone()
    for r in sick:
        x[r, slice(256, None) if everywhere else slice(300, None, 37)] = float("nan")
    c["qkv"] = x
    pools = pools_of(c)
    call(c, pools)
    torch.cuda.synchronize()
    L.lynx_device_status()
    rows = x.double().cpu().numpy().reshape(n, -1, 128)
    for which in range(2):
        new = rows[:, 2 + 2 * which:4 + 2 * which]
        codes, scales, _ = e4m3.append(np.nan_to_num(new), c["slots"], c["codes"][which], c["scales"][which])
        got = pools[which].view(torch.uint8).cpu().numpy()
        assert np.array_equal(pools[2].cpu().numpy()[:, which], scales)
        bad = np.zeros(codes.shape, dtype=bool)
        for h in range(2):
            bad[c["slots"][:, h] // 256, c["slots"][:, h] % 256] = np.isnan(new[:, h])
        assert np.all(got[bad] % 128 == 127) and np.array_equal(got[~bad], codes[~bad])


def test_a_key_whose_norm_is_nan(cuda_device):
    """One NaN channel makes the normalised key NaN as a whole; its neighbours in the block are right."""
    c = case([(33, 5)], 1, 1, 3)
    c["qkv"] = c["qkv"].clone()
    c["qkv"][2, 128 + 9] = float("nan")
    pools = pools_of(c)
    call(c, pools)
    L.lynx_device_status()
    x = c["qkv"].double().cpu().numpy().reshape(5, 3, 128)
    cos, sin = c["cs"][c["positions"], :64].astype(float), c["cs"][c["positions"], 64:].astype(float)
    keys = np.nan_to_num(sv.norm_rotate(x[:, 1:2], c["w"][1], 1e-6, cos, sin, False))
    codes, scales, _ = e4m3.append(keys, c["slots"], c["codes"][0], c["scales"][0])
    got = pools[0].view(torch.uint8).cpu().numpy()
    assert np.array_equal(pools[2].cpu().numpy()[:, 0], scales)
    page, at = divmod(int(c["slots"][2, 0]), 256)
    assert np.all(got[page, at] % 128 == 127)
    got[page, at] = codes[page, at]
    # one code in a thousand may be a neighbour, where float32 and float64 round to different sides
    off = got != codes
    assert off.mean() < 1e-3 and np.all(np.abs(e4m3.decode(got) - e4m3.decode(codes))[off] <= 2.0 ** -3 * np.abs(e4m3.decode(codes))[off] + 2.0 ** -9)
