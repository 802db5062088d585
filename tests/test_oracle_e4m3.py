"""The 8-bit pages' oracle against torch's conversion and against its own definition."""
import numpy as np
import torch

from oracle import e4m3


def test_codes_as_torch_has_them():
    codes = torch.arange(256, dtype=torch.uint8)
    there = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(e4m3.decode(codes.numpy()), there, equal_nan=True)
    x = np.concatenate([np.random.default_rng(0).uniform(-448, 448, 20000), np.exp2(np.random.default_rng(1).uniform(-14, 8, 20000))])
    v = e4m3.VALUES[:127]
    x = np.concatenate([x, v, -v, (v[1:] + v[:-1]) / 2, -(v[1:] + v[:-1]) / 2]).astype(np.float32)   # values and ties
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(e4m3.encode(x), want)


def test_scale_is_the_smallest_that_holds_the_block():
    for top in (1.0, 448.0, np.nextafter(448.0, 1e9), 447.9, 896.0, 3e-5, 1e10):
        s = e4m3.scale_byte(top)
        assert top <= 448 * 2.0 ** (s - 127) and top > 448 * 2.0 ** (s - 128)
    assert e4m3.scale_byte(0.0) == 74 and e4m3.scale_byte(1e38) == 198


def test_append_rounds_what_stands_in_front_only_where_the_scale_grows():
    rng = np.random.default_rng(2)
    codes, scales = e4m3.quantise_pages(rng.standard_normal((2, 256, 128)))
    small = rng.standard_normal((1, 1, 128)) * 1e-3
    slots = np.array([[256 + 70]])
    c, s, _ = e4m3.append(small, slots, codes, scales)
    assert np.array_equal(s, scales) and np.array_equal(np.delete(c[1], 70, 0), np.delete(codes[1], 70, 0))
    large = small * 1e7
    c, s, _ = e4m3.append(large, slots, codes, scales)
    assert s[1, 2] > scales[1, 2] and np.array_equal(np.delete(s.ravel(), 10), np.delete(scales.ravel(), 10))
    d, was = e4m3.dequantise_pages(c, s), e4m3.dequantise_pages(codes, scales)
    assert np.abs(d[1, 70] - large[0, 0]).max() <= np.abs(large).max() / 16
    assert np.abs(d[1, 64:70] - was[1, 64:70]).max() <= 2.0 ** (s[1, 2] - 127.0 - 10) + 2.0 ** -4 * np.abs(was).max()
    assert np.array_equal(d[0], was[0]) and np.array_equal(d[1, :64], was[1, :64])
    # the first token of a block: what the block held before does not count
    c, s, _ = e4m3.append(small, np.array([[256 + 64]]), codes, scales)
    assert s[1, 2] < scales[1, 2]


def test_attention_of_no_and_of_one_key():
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((2, 128)), rng.standard_normal((5, 128)), rng.standard_normal((5, 128))
    out, lse = e4m3.attention(q, k, v, 0.1, [0, 1])
    assert np.all(out[0] == 0) and np.isneginf(lse[0])
    assert np.allclose(out[1], v[0]) and np.isclose(lse[1], 0.1 * q[1] @ k[0])
