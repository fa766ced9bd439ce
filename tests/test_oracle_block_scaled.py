"""CPU pins of the e4m3 page oracle: the number format against its definition and torch's,
the scale rule, and what appending in pieces must agree with."""

import numpy as np
import pytest
import torch

from oracle import block_scaled as O


def test_values_match_the_format():
    v = O.e4m3_values(np.arange(256))
    ref = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(v), np.isnan(ref)) and np.array_equal(v[~np.isnan(v)], ref[~np.isnan(ref)])
    assert v[0x7E] == 448 and v[0x01] == 2.0 ** -9 and v[0x08] == 2.0 ** -6


def test_codes_are_nearest_with_ties_to_even():
    v = O.e4m3_values(np.arange(0x7F))
    assert np.array_equal(O.e4m3_codes(v), np.arange(0x7F)) and np.array_equal(O.e4m3_codes(-v[1:]), 0x80 + np.arange(1, 0x7F))
    mid = (v[:-1] + v[1:]) / 2
    even = np.where(np.arange(0x7E) % 2 == 0, np.arange(0x7E), np.arange(1, 0x7F))
    assert np.array_equal(O.e4m3_codes(mid), even)
    assert np.array_equal(O.e4m3_codes(np.nextafter(mid, 1e9)), np.arange(1, 0x7F))
    assert np.array_equal(O.e4m3_codes(np.nextafter(mid, 0)), np.arange(0x7E))
    assert O.e4m3_codes(1e30) == 0x7E and O.e4m3_codes(-449.0) == 0xFE
    x = np.random.default_rng(1).normal(size=5000) * 100
    x = np.clip(x, -448, 448).astype(np.float32)
    ref = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(O.e4m3_codes(x), ref)


@pytest.mark.parametrize("a,s", [(0.0, 0.0), (448.0, 1.0), (448.5, 2.0), (1.0, 2.0 ** -8), (1.75, 2.0 ** -8),
                                 (1.7578125, 2.0 ** -7), (3.0e38, 2.0 ** 120), (1e-40, 2.0 ** -126)])
def test_block_scale(a, s):
    assert O.block_scale(a) == np.float32(s)


def test_append_row_by_row_ends_where_one_append_does():
    # scales are powers of two, so a grown scale shifts the earlier codes; rows whose codes stay
    # in the normal range (magnitudes within 2^12 of the block's largest) keep every bit
    rng = np.random.default_rng(3)
    new = rng.choice([-1, 1], size=(2, 2, 40, 64)) * rng.uniform(1, 2, size=(2, 2, 40, 64)) * \
        2.0 ** rng.integers(0, 5, size=(2, 2, 40, 1))
    tables, lens = [[3, 0, 5], [4, 1, 2]], [0, 7]
    pool = rng.integers(0, 126, size=(6, 2, 32, 64)).astype(np.uint8)
    scales = np.full((6, 2), 2.0 ** -9, dtype=np.float32)
    at_once, s1 = O.append_blocks(new, tables, lens, pool, scales)
    p, s = pool, scales
    for j in range(40):
        p, s = O.append_blocks(new[:, :, j:j + 1], tables, [l + j for l in lens], p, s)
    for blk in (0, 3, 1):  # blocks that held no row before
        assert np.array_equal(s[blk], s1[blk])
        rows = 32 if blk == 3 else 8 if blk == 0 else 15
        assert np.array_equal(O.block_values(p, s)[blk, :, :rows], O.block_values(at_once, s1)[blk, :, :rows])


def test_appended_values_are_within_half_a_step():
    rng = np.random.default_rng(5)
    new = rng.normal(size=(1, 1, 50, 64))
    pool, scales = O.append_blocks(new, [[0, 1]], [0], np.zeros((2, 1, 32, 64), np.uint8), np.ones((2, 1), np.float32))
    got = O.block_values(pool, scales)[:, 0].reshape(64, 64)[:50]
    ref = new[0, 0].astype(np.float32)
    step = np.maximum(2.0 ** -4 * np.abs(ref), scales.max() * 2.0 ** -10)  # half a step: relative, or of the smallest values
    assert (np.abs(got - ref) <= step).all()
