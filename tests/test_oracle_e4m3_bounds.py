"""The bounds of attention over pages in 8 bits tell a kernel that loses small probabilities,
the second half of a probability, small rows or small channels from one that does not."""
import numpy as np
import pytest

from e4m3_testutil import Cache, attention_and_bounds, equal_keys_case, far_key_case, small_channels_case, to_bf16


def one_head(cache, q, scale):
    k, v = cache.values(0, 0)
    rows = q.reshape(-1, 128)
    return rows, k, v, attention_and_bounds(rows, k, v, scale, [k.shape[0]] * rows.shape[0])


def weights(rows, k, lse, scale):
    return np.exp(scale * rows @ k.T - lse[:, None])


def test_the_keys_far_below_the_largest_count():
    cache, q, scale = far_key_case()
    rows, k, v, (out, lse, off_o, off_l) = one_head(cache, q, scale)
    p = weights(rows, k, lse, scale)
    assert np.abs(p @ v - out).max() <= off_o.min() / 100
    without = np.where(p > 0.5, p, 0) @ v
    assert np.all(np.abs(without - out) > 10 * off_o)


@pytest.mark.parametrize("rows", [4, 12, 20])
def test_both_halves_of_a_probability_count(rows):
    cache, q, scale = equal_keys_case(rows)
    rows, k, v, (out, lse, off_o, off_l) = one_head(cache, q, scale)
    p = weights(rows, k, lse, scale)
    top = p.max()
    half = (p / top * 2.0 ** 10).astype(np.float16).astype(float) * 2.0 ** -10 * top
    assert np.all(np.abs(half @ v - out) > 2 * off_o)


def test_small_channels_count():
    cache, q, scale = small_channels_case()
    rows, k, v, (out, lse, off_o, off_l) = one_head(cache, q, scale)
    for c in (15, 16, 32):
        less = rows.copy()
        less[:, c] = 0
        o = attention_and_bounds(less, k, v, scale, [777] * 8)[0]
        assert np.all((np.abs(o - out) > 10 * off_o).any(1))


@pytest.mark.parametrize("log_size", [-60, -30, -8, 0, 8])
def test_rows_of_any_size_count(log_size):
    cache = Cache([777], 1, seed=9)
    cache.scales[0][:] = np.clip(cache.scales[0].astype(int) - log_size, 0, 255)
    q = to_bf16(np.random.default_rng(10).standard_normal((1, 1, 8, 128)) * 2.0 ** log_size)
    rows, k, v, (out, lse, off_o, off_l) = one_head(cache, q, 128 ** -0.5)
    o, l = attention_and_bounds(0 * rows, k, v, 128 ** -0.5, [777] * 8)[:2]
    assert np.all(np.abs(o - out).max(1) > 100 * off_o.max(1)) and np.all(np.abs(l - lse) > 100 * off_l)
