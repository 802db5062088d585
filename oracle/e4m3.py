"""Pages in 8 bits, in plain numpy: E4M3 codes, blocks of 32 tokens with a
power-of-two scale, the append of new tokens to them in float64, and attention
of a few query rows over the paged cache in float64."""
from __future__ import annotations

import math

import numpy as np

PAGE, BLOCK, H = 256, 32, 128
TOP = 448.0
SCALE_LO, SCALE_HI = 74, 198


def _values():
    """What the codes 0..127 stand for (127: NaN)."""
    v = []
    for code in range(128):
        e, m = code >> 3, code & 7
        v.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    v[127] = math.nan
    return np.array(v)


VALUES = _values()


def decode(codes):
    """uint8 codes -> float64."""
    codes = np.asarray(codes)
    return np.where(codes & 0x80, -1.0, 1.0) * VALUES[codes & 0x7F]


def encode(x):
    """float64 in -448..448 -> the nearest codes, ties to the even one."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), TOP)
    # codes are ordered as their values: the position among the middles
    v = VALUES[:127]
    middle = (v[1:] + v[:-1]) / 2
    low = np.searchsorted(middle, a, side="left")
    high = np.searchsorted(middle, a, side="right")
    code = np.where(low == high, low, np.where(low % 2 == 0, low, high))
    return (code + 128 * np.signbit(x)).astype(np.uint8)


def scale_byte(top):
    """The smallest s in SCALE_LO..SCALE_HI with top <= 448 * 2^(s - 127), or SCALE_HI."""
    s = SCALE_LO
    while s < SCALE_HI and float(top) > TOP * 2.0 ** (s - 127):
        s += 1
    return s


def quantise_pages(x):
    """float64 [n, 256, 128] -> (codes uint8 [n, 256, 128], scale bytes [n, 8])."""
    n = x.shape[0]
    blocks = x.reshape(n, PAGE // BLOCK, BLOCK, H)
    top = np.abs(blocks).max((2, 3))
    s = np.array([[scale_byte(t) for t in row] for row in top], dtype=np.int64).reshape(n, PAGE // BLOCK)
    codes = encode(blocks * 2.0 ** (127 - s)[:, :, None, None])
    return codes.reshape(x.shape), s.astype(np.uint8)


def dequantise_pages(codes, scales):
    """codes [n, 256, 128], scale bytes [n, 8] -> float64."""
    s = np.clip(scales.astype(np.int64), SCALE_LO, SCALE_HI)
    return decode(codes) * np.repeat(2.0 ** (s - 127), BLOCK, axis=1)[:, :, None]


def append(x, slots, codes, scales):
    """Rows x float64 [n, heads, 128] written to slots [n, heads] (negative: not written) of
    codes [pool, 256, 128] and scales [pool, 8]; returns new arrays and, for each code, the
    value that it stands for before it is rounded (the codes' own where nothing was written).
    A row that is not written, where a block's rows go on behind it one row a token, leaves
    them one run."""
    codes, scales = codes.copy(), scales.copy()
    wanted = decode(codes)
    for h in range(x.shape[1]):
        r = 0
        while r < x.shape[0]:
            slot = int(slots[r, h])
            if slot < 0:
                r += 1
                continue
            page, first = divmod(slot, PAGE)
            block, at = divmod(first, BLOCK)
            run = [0]   # the rows behind it that go on in its block
            for n in range(1, min(BLOCK - at, x.shape[0] - r)):
                if int(slots[r + n, h]) == slot + n:
                    run.append(n)
                elif slots[r + n, h] >= 0:
                    break
            run = np.array(run)
            was = min(max(int(scales[page, block]), SCALE_LO), SCALE_HI)
            s = scale_byte(np.abs(x[r + run, h]).max())
            if at > 0:
                s = max(s, was)
                old = slice(block * BLOCK, first)
                wanted[page, old] = decode(codes[page, old]) * 2.0 ** (was - s)
                codes[page, old] = encode(wanted[page, old])
            new = x[r + run, h] * 2.0 ** (127 - s)
            wanted[page, first + run] = np.clip(new, -TOP, TOP)
            codes[page, first + run] = encode(np.clip(new, -TOP, TOP))
            scales[page, block] = s
            r += int(run[-1]) + 1
    return codes, scales, wanted


def attention(q, k, v, scale, seen):
    """One KV head: q [rows, 128] over k, v [n, 128] float64, row r over its first seen[r]
    keys -> (out [rows, 128], lse [rows]); no keys: zeros and -inf."""
    out = np.zeros((q.shape[0], H))
    lse = np.full(q.shape[0], -np.inf)
    for r in range(q.shape[0]):
        n = min(max(int(seen[r]), 0), k.shape[0])
        if n == 0:
            continue
        s = scale * (k[:n] @ q[r])
        m = s.max()
        p = np.exp(s - m)
        lse[r] = m + math.log(p.sum())
        out[r] = p @ v[:n] / p.sum()
    return out, lse
