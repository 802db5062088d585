"""lynx_qkv_append_e4m3 with rows in the middle of their blocks that are not written: those
around them are one run, whatever the reason and wherever a CTA's rows end."""
import numpy as np
import pytest
import torch

from progressive_kv_quantization_gb300 import lynx as L
from test_gpu_append_e4m3 import call, case, check, pools_of

pytestmark = pytest.mark.gpu


def refuse(c, rows, how):
    """Makes rows of a case ones that are not written; returns the error word that tells of it."""
    if how == "position":
        c["positions"][rows] = 100000
        return 4
    if how == "slot":
        c["slots"][rows] = c["codes"].shape[1] * 256 + np.arange(c["Hkv"])
        return 5
    if how == "no position":
        c["positions"][rows] = -1
    else:
        c["slots"][rows] = -1
    return 0


def call_and_check(c, words):
    """The call three times on fresh pools: the same bits, and the oracle's with the rows left out."""
    first = None
    for _ in range(3):
        pools = pools_of(c)
        q = call(c, pools)
        torch.cuda.synchronize()
        if words:
            with pytest.raises(L.LynxError, match="= [%s] " % "".join(map(str, sorted(words)))):
                L.lynx_device_status()
        bits = [p.view(torch.uint8).clone() for p in pools]
        assert first is None or all(torch.equal(a, b) for a, b in zip(first, bits))
        first = bits
    left_out = dict(c, positions=np.where(c["positions"] >= 100000, -1, c["positions"]),
                    slots=np.where(c["slots"] >= c["codes"].shape[1] * 256, -1, c["slots"]))
    check(left_out, q, pools)


HOW = ["position", "slot", "no position", "no slot"]


@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("held", [0, 5, 31])
def test_one_row_in_the_middle(cuda_device, how, held):
    for row in (0, 1, 7, 30, 31, 32, 39):
        c = case([(held, 40)], 2, 1, 9 + row)
        word = refuse(c, [row], how)
        call_and_check(c, {word} if word else set())


@pytest.mark.parametrize("how", HOW)
def test_blocks_of_which_little_is_written(cuda_device, how):
    """First and last token of a block, at every place of a CTA's 32 rows; other runs in front and behind."""
    for front in (1, 2, 15, 16, 30, 31, 32, 33, 45):
        c = case([(3, 1)] * front + [(0, 32), (64, 32), (7, 3)], 3, 2, front, norm=False, rot=64)
        word = refuse(c, np.r_[front + 1:front + 31, front + 33:front + 63], how)
        call_and_check(c, {word} if word else set())


@pytest.mark.parametrize("seed", range(6))
def test_rows_left_out_everywhere(cuda_device, seed):
    rng = np.random.default_rng(seed)
    reqs = [(int(rng.integers(0, 300)), int(rng.integers(1, 90))) for _ in range(20)]
    c = case(reqs, 4, 2, seed, interleaved=bool(seed % 2), rot=128 if seed < 3 else 32, pad=3)
    n = sum(r[1] for r in reqs)
    words = set()
    for how in HOW:
        rows = np.flatnonzero(rng.random(n) < 0.12)
        words.add(refuse(c, rows, how))
    c["slots"][c["positions"] < 0] = -1
    call_and_check(c, words - {0})
