"""The float64 oracle of norm and rotation, held against properties of the formula."""

import numpy as np
import pytest

from oracle import rotate


def test_scores_depend_on_the_distance_alone():
    rng = np.random.default_rng(0)
    q, k = rng.normal(size=(1, 1, 64)), rng.normal(size=(1, 1, 64))
    freq = 1e4 ** (-np.arange(32) / 32)
    for adjacent in (False, True):
        at = lambda x, p: rotate.norm_rotate(x, [p], freq, adjacent=adjacent)[0]
        s0 = (at(q, 7) * at(k, 3)).sum()
        s1 = (at(q, 1007) * at(k, 1003)).sum()
        assert abs(s0 - s1) < 1e-9
        assert abs((at(q, 0) - q)).max() == 0.0


def test_norm_gives_rows_of_unit_mean_square():
    x = np.random.default_rng(1).normal(size=(3, 2, 128)) * 17.0
    y, _ = rotate.norm_rotate(x, [0, 1, 2], 1e4 ** (-np.arange(64) / 64), weight=np.zeros(128), offset=1.0, eps=0.0)
    assert np.allclose((y * y).mean(-1), 1.0)


@pytest.mark.parametrize("sections,cycle,axes", [
    ([2, 1, 1], False, [0, 0, 1, 2]),
    ([2, 1, 1], True, [0, 1, 2, 0]),
    ([4, 2, 2], True, [0, 1, 2, 0, 1, 2, 0, 0]),
    ([0, 4], False, [1, 1, 1, 1]),
    ([4], True, [0, 0, 0, 0]),
])
def test_axes_of_frequencies(sections, cycle, axes):
    assert [rotate.axis_of(i, sections, cycle) for i in range(len(axes))] == axes


def test_equal_positions_on_all_axes_are_one_axis():
    rng = np.random.default_rng(2)
    x, freq, pos = rng.normal(size=(5, 3, 64)), 1e4 ** (-np.arange(32) / 32), np.arange(5) * 11
    one = rotate.norm_rotate(x, pos, freq)[0]
    for cycle in (False, True):
        assert np.array_equal(rotate.norm_rotate(x, np.stack([pos] * 3), freq, sections=[12, 10, 10], cycle=cycle)[0], one)
