"""Caches of pages in 8 bits for the tests, and how far attention over them may be
off (no GPU code here)."""
from __future__ import annotations

import math

import numpy as np

from oracle import e4m3

NAN_CODE = 0x7F


def to_bf16(x):
    """The nearest BF16 numbers, as float64."""
    b = np.asarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000
    return b.astype(np.uint32).view(np.float32).astype(np.float64)


class Cache:
    """Pages of requests of the given lengths in a shuffled pool.  Positions behind a
    request's last token hold NaN codes, blocks behind it bytes outside the scales' range."""

    def __init__(self, lens, Hkv, seed, max_pages=None, spare=3, spread=0.0, poison=True):
        rng = np.random.default_rng(seed)
        pages = [-(-max(n, 0) // e4m3.PAGE) for n in lens]
        self.max_pages = max_pages or max(1, max(pages))
        n = sum(pages) * Hkv + spare
        order = rng.permutation(n)
        self.table = np.full((len(lens), Hkv, self.max_pages), -7, dtype=np.int32)
        self.codes, self.scales = [], []
        for _ in range(2):
            x = rng.standard_normal((n, e4m3.PAGE, e4m3.H)) + rng.standard_normal(e4m3.H)
            if spread:   # blocks of other sizes
                size = np.exp2(rng.integers(-spread, spread + 1, (n, e4m3.PAGE // e4m3.BLOCK)))
                x *= np.repeat(size, e4m3.BLOCK, axis=1)[:, :, None]
            c, s = e4m3.quantise_pages(x)
            self.codes.append(c)
            self.scales.append(s)
        at = 0
        for b, length in enumerate(lens):
            for h in range(Hkv):
                for j in range(pages[b]):
                    page = order[at]
                    at += 1
                    self.table[b, h, j] = page
                    left = length - j * e4m3.PAGE
                    if poison and left < e4m3.PAGE:
                        for c, s in zip(self.codes, self.scales):
                            c[page, left:] = NAN_CODE
                            s[page, -(-left // e4m3.BLOCK):] = rng.choice([0, 255, 73, 199])
        self.lens, self.Hkv = lens, Hkv

    def values(self, b, h):
        """Keys and values of a request and head, float64 [len, 128]."""
        n = self.lens[b]
        ids = self.table[b, h, :-(-n // e4m3.PAGE)]
        return [e4m3.dequantise_pages(c[ids], s[ids]).reshape(-1, e4m3.H)[:n] for c, s in zip(self.codes, self.scales)]

    def pools(self):
        """(k codes, v codes, scales [n, 2, 8])"""
        return self.codes[0], self.codes[1], np.stack(self.scales, 1)


def score_error(q, k, scale):
    """How far a score may be off: products of the codes and BF16 numbers are exact, and of
    the float32 sum of 128 of them eight partial sums (one a product of 16) are cut off at
    2^-23 of what they hold at most, with a few roundings of factors behind them."""
    return 16 * 2.0 ** -23 * scale * float((np.abs(q) @ np.abs(k).T).max(initial=0.0))


def decode_bound(q, k, v, scale):
    """How far an output may be off, for probabilities of 22 bits: twice the scores' error
    (in p and in the sum), the exponential's 2^-21 and the sums' roundings."""
    return (2 * score_error(q, k, scale) + 2.0 ** -18) * float(np.abs(v).max(initial=0.0))


def attention_and_bounds(q, k, v, scale, seen):
    """One KV head, row by row: (out, lse, how far each output may be off, how far each lse).

    Row r's scores are off by e_r at most: score_error's 16 steps of 2^-23, of that row's own
    scale |q| |k| over the keys that it sees.  A probability, relative to itself, by e_r, by 2^-19 of the exponent's
    argument (rounded once, in 32..64 where it is largest) and by 2^-21 of the exponential, 2^-18 in
    all with the float32 sums behind them; and by 2^-35 of the largest one, since it is held as two
    FP16 numbers of 2^10 p whose steps end at 2^-24 (half a step each).  So with sum p = 1
        |out error| <= 2 (e_r + 2^-18) sum p |v| + 2 * 2^-35 max p sum |v|
    (the factors 2: once for the sum of p v, once for the sum of p)."""
    out, lse = e4m3.attention(q, k, v, scale, seen)
    off_o, off_l = np.zeros_like(out), np.zeros_like(lse)
    size = np.abs(v)
    for r in range(q.shape[0]):
        n = min(max(int(seen[r]), 0), k.shape[0])
        if n == 0:
            continue
        p = np.exp(scale * (k[:n] @ q[r]) - lse[r])
        e = 16 * 2.0 ** -23 * scale * float((np.abs(k[:n]) @ np.abs(q[r])).max()) + 2.0 ** -18
        off_o[r] = 2 * e * (p @ size[:n]) + 2.0 ** -34 * p.max() * size[:n].sum(0)
        off_l[r] = e + 2.0 ** -22 * abs(lse[r])
    return out, lse, off_o, off_l


def far_key_case():
    """One key's score stands 20 above those of 20,000 equal ones, whose values are 2^12 times as large:
    (cache, queries [1, 1, 4, 128], scale).  Products and sums of the scores are exact."""
    n, far = 20001, 700
    cache = Cache([n], 1, seed=11)
    rng = np.random.default_rng(12)
    cache.codes[0][:] = 0x38                                           # keys of ones
    cache.codes[0][cache.table[0, 0, far // 256], far % 256] = 0x40    # twos
    cache.codes[1][:] = rng.integers(0x30, 0x48, cache.codes[1].shape, dtype=np.uint8)   # 0.5 .. 3.75
    cache.scales[0][:] = 127
    cache.scales[1][:] = 127 + 12
    cache.scales[1][cache.table[0, 0, far // 256], far % 256 // 32] = 127
    cache.codes[0][cache.table[0, 0, n // 256], n % 256:] = NAN_CODE
    return cache, np.full((1, 1, 4, 128), 0.125), 1.25


def equal_keys_case(rows):
    """2,000 keys, all but one in 32 of the first page alike, a little below those: their p is no round
    number, and its rounding to FP16 the same for all: (cache, queries [1, 1, rows, 128], scale)."""
    cache = Cache([2000], 1, seed=13, poison=False)
    rng = np.random.default_rng(14)
    cache.codes[0][:] = 0x38
    cache.codes[0][cache.table[0, 0, 0], ::32] = 0x39                  # 1.125
    cache.codes[1][:] = rng.integers(0x30, 0x48, cache.codes[1].shape, dtype=np.uint8)
    for s in cache.scales:
        s[:] = 127
    return cache, np.full((1, 1, rows, 128), 0.125), 0.1


def small_channels_case():
    """Channel c of the queries is 2^-(c mod 17) of the usual size, and the keys' 2^(c mod 17) times: all count
    alike.  (cache, queries [1, 1, 8, 128], scale)"""
    cache = Cache([777], 1, seed=15)
    rng = np.random.default_rng(16)
    size = np.exp2(np.arange(128) % 17)
    x = rng.standard_normal(cache.codes[0].shape) * size
    cache.codes[0], cache.scales[0] = e4m3.quantise_pages(x)
    last = cache.table[0, 0, 3]
    cache.codes[0][last, 777 % 256:] = NAN_CODE
    q = rng.uniform(0.5, 1.5, (1, 1, 8, 128)) * rng.choice([-1, 1], (1, 1, 8, 128))
    return cache, to_bf16(q / size), 1 / math.sqrt(128)
