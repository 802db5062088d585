"""The 8-bit append's oracle: rows that are not written leave the others of their block one run."""
import numpy as np

from oracle import e4m3


def test_a_row_left_out_leaves_one_run():
    rng = np.random.default_rng(0)
    codes, scales = e4m3.quantise_pages(rng.standard_normal((2, 256, 128)))
    x = rng.standard_normal((30, 1, 128)) * np.exp2(rng.integers(-6, 7, (30, 1, 1)))
    slots = 256 + 35 + np.arange(30)[:, None]           # tokens 35..63 of page 1, and one of the next block
    holes = np.array([4, 5, 17])
    slots[holes] = -1
    c, s, _ = e4m3.append(x, slots, codes, scales)
    kept = np.setdiff1d(np.arange(29), holes)
    want = max(e4m3.scale_byte(np.abs(x[kept]).max()), int(scales[1, 1]))
    assert s[1, 1] == want and s[1, 2] == e4m3.scale_byte(np.abs(x[29]).max())
    assert np.array_equal(c[1, 35 + kept], e4m3.encode(x[kept, 0] * 2.0 ** (127 - want)))
    assert np.array_equal(c[1, 35 + holes], codes[1, 35 + holes])
    assert np.array_equal(c[1, 32:35], e4m3.encode(e4m3.decode(codes[1, 32:35]) * 2.0 ** (int(scales[1, 1]) - want)))
    # nothing but the rows left out: the values behind a gap of another length are a run of their own
    slots[6:29] += 1
    slots[29] = -1
    assert not np.array_equal(e4m3.append(x, slots, codes, scales)[0], c)
