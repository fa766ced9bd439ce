"""CPU oracle of e4m3 pages (one f32 scale per block and KV head): the number format, the
append that quantises, and the values the decode attends over (test infrastructure only,
like the rest of ``oracle/``; numpy only).

An e4m3 code is a byte: sign, 4 exponent bits (bias 7), 3 fraction bits; exponent 0 holds
the multiples of 2^-9 below 2^-6, the pattern 0x7F (and 0xFF) is NaN, the largest value is
448 and there are no infinities.

Appending rows to a block: with ``a`` the largest magnitude of the new rows and ``s`` the
block's scale (0 when it holds no earlier row),

    s'   = max(s, 2^e), e the smallest integer >= -126 with a <= 448 * 2^e (0 if a = 0)
    code = e4m3(x / s') for new rows, e4m3(code * (s / s')) for earlier ones when s' > s

each quotient and product rounded to f32 as the GPU takes it, then to the nearest code,
ties to the even one. ``tests/test_oracle_block_scaled.py`` pins all of it.
"""

from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0


def _positive_values() -> np.ndarray:
    c = np.arange(127)  # codes 0x00 .. 0x7E
    e, f = c >> 3, (c & 7).astype(np.float64)
    return np.where(e == 0, np.ldexp(f / 8, -6), np.ldexp(1 + f / 8, e - 7))


POSITIVE = _positive_values()


def e4m3_values(codes) -> np.ndarray:
    """Values of e4m3 codes (uint8), float64."""
    codes = np.asarray(codes).astype(np.uint8)
    table = np.concatenate([POSITIVE, [np.nan], -POSITIVE, [np.nan]])
    return table[codes]


def e4m3_codes(x) -> np.ndarray:
    """Codes nearest to finite ``x``, ties to the even code, magnitudes above 448 to 448."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), E4M3_MAX)
    up = np.searchsorted(POSITIVE, a, side="left")  # first code with value >= a
    down = np.maximum(up - 1, 0)
    mid = (POSITIVE[down] + POSITIVE[up]) / 2  # exact: neighbours have few bits
    code = np.where(a > mid, up, np.where(a < mid, down, np.where(down % 2 == 0, down, up)))
    code = np.where(POSITIVE[up] == a, up, code)
    return (code | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def block_scale(a: float) -> np.float32:
    """The smallest power of two s >= 2^-126 with a <= 448 s; 0 for a = 0."""
    if a == 0:
        return np.float32(0)
    e = -126
    while E4M3_MAX * 2.0 ** e < a:
        e += 1
    return np.float32(2.0 ** e)


def append_blocks(new, block_tables, seq_lens, pool, scales):
    """One plane's append: ``new`` [B, HK, n, D] at positions len_b .. of each sequence;
    returns copies (pool codes uint8 [NB, HK, BS, D], scales f32 [NB, HK])."""
    new = np.asarray(new, dtype=np.float32)
    B, HK, n, _ = new.shape
    pool, scales = np.array(pool, dtype=np.uint8), np.array(scales, dtype=np.float32)
    BS = pool.shape[2]
    for b in range(B):
        start = int(seq_lens[b])
        for j in range(start // BS, (start + n - 1) // BS + 1 if n else 0):
            lo, hi = max(start, j * BS), min(start + n, (j + 1) * BS)
            blk = int(block_tables[b][j])
            for h in range(HK):
                x = new[b, h, lo - start:hi - start]
                old = scales[blk, h] if lo > j * BS else np.float32(0)
                s = max(old, block_scale(float(np.abs(x).max())))
                if lo > j * BS and s > old:
                    kept = e4m3_values(pool[blk, h, :lo - j * BS]).astype(np.float32)
                    pool[blk, h, :lo - j * BS] = e4m3_codes(kept * np.float32(old / s))
                pool[blk, h, lo - j * BS:hi - j * BS] = e4m3_codes(x / s) if s > 0 else 0
                scales[blk, h] = s
    return pool, scales


def block_values(pool, scales) -> np.ndarray:
    """Values of e4m3 pages, float64 [NB, HK, BS, D]: scale of the block times the code's value."""
    return e4m3_values(pool) * np.asarray(scales, dtype=np.float64)[:, :, None, None]
