"""CPU pins of the sparse oracle: outward rounding, bounds, scores that bound every product,
the choice's rules, and attention that is the dense one when every block is chosen."""

import numpy as np
import pytest
import torch

import oracle
from oracle import sparse as S


def bf16(x):
    return torch.from_numpy(np.asarray(x)).to(torch.bfloat16).double().numpy()


def test_outward_rounding():
    rng = np.random.default_rng(0)
    x = rng.normal(size=4000) * 10.0 ** rng.integers(-6, 6, size=4000)
    lo, hi = S.bf16_outward(x, False), S.bf16_outward(x, True)
    assert (lo <= x).all() and (hi >= x).all()
    assert np.array_equal(bf16(lo), lo) and np.array_equal(bf16(hi), hi)
    near = bf16(x)
    assert ((near == lo) | (near == hi)).all()  # the nearest value is one of the two
    same = bf16(x)
    assert np.array_equal(S.bf16_outward(same, False), same) and np.array_equal(S.bf16_outward(same, True), same)


def test_bounds_widen_as_rows_arrive():
    rng = np.random.default_rng(1)
    values = bf16(rng.normal(size=(4, 2, 16, 8)))
    start = np.full((4, 2, 2, 8), 99.0)
    at_once = S.update_bounds(start, values, [[2, 0], [1, 3]], [30, 17], 30)
    step = start
    for n in range(1, 31):
        step = S.update_bounds(step, values, [[2, 0], [1, 3]], [n, min(n, 17)], 1 if n <= 17 else 0)
        if n > 17:  # the second sequence has stopped
            step = S.update_bounds(step, values, [[2, 0]], [n], 1)
    assert np.array_equal(step, at_once)
    assert np.array_equal(at_once[0, :, 0], values[0, :, :14].min(1))
    assert np.array_equal(at_once[3, :, 1], values[3, :, 0])


def test_scores_bound_every_product():
    rng = np.random.default_rng(2)
    keys = bf16(rng.normal(size=(20, 16, 32)))
    q = bf16(rng.normal(size=(3, 32)))
    s = S.block_scores(q, keys.min(1), keys.max(1))
    assert (np.asarray(s) >= np.einsum("nbd,rd->nbr", keys, q).max((1, 2)) - 1e-12).all()
    one = S.block_scores(q, keys[:, 0], keys[:, 0])  # blocks of one key: the product itself
    assert np.allclose(one, (keys[:, 0] @ q.T).max(1))


@pytest.mark.parametrize("n,k,first,last,want", [
    (3, 4, 1, 1, [0, 1, 2]), (6, 4, 1, 1, [0, 3, 4, 5]), (6, 2, 1, 1, [0, 5]), (6, 3, 0, 1, [0, 3, 5]),
    (6, 5, 2, 2, [0, 1, 3, 4, 5])])
def test_choice(n, k, first, last, want):
    assert S.choose([9, 1, 2, 5, 5, 0][:n], k, first, last) == want


def test_ties_go_to_the_lower_block():
    assert S.choose([0, 7, 7, 7, 7, 0], 4, 1, 1) == [0, 1, 2, 5]


def test_every_block_chosen_is_the_dense_read():
    rng = np.random.default_rng(4)
    k, v = rng.normal(size=(6, 2, 16, 8)), rng.normal(size=(6, 2, 16, 8))
    q = rng.normal(size=(2, 4, 3, 8))
    tables, lens = [[5, 0, 2], [1, 4, 3]], [40, 19]
    ref = oracle.paged_decode_attention(q, k, v, tables, lens, 0.3, 3)
    got = S.sparse_attention(q, k, v, tables, lens, 0.3, [[[0, 1, 2]] * 2, [[0, 1]] * 2])
    assert np.abs(got - ref).max() < 1e-12
