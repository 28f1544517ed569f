"""The key-by-key checks of long contexts find what they are for: mistakes planted in the numbers that they check."""
import numpy as np
import pytest

from tests.paged_keys import STAGE, count_errors, count_keys


def row(length, d, weight=None, seed=0):
    """(out, lse) of a row whose stages are counted `weight` times each, and the true counts."""
    feature = np.random.default_rng(seed).integers(0, d, -(-length // STAGE))
    true = count_keys(feature, length, d)
    got = true if weight is None else count_keys(feature, length, d, weight)
    total = got.sum()
    return (got / total)[None], np.array([np.log(total)]), true[None], np.array([length])


@pytest.mark.parametrize("length", [1, 16, 208, 9001, 12345, 20011, 31200, 60000])
@pytest.mark.parametrize("d", [64, 128])
def test_right_numbers_pass(length, d):
    assert count_errors(*row(length, d)) == (0.0, 0.0)


@pytest.mark.parametrize("length", [9001, 12345, 20011, 31200, 60000])
@pytest.mark.parametrize("d", [64, 128])
def test_a_lost_or_doubled_stage_shows(length, d):
    """By twice what is allowed at least: a kernel's own error does not hide it."""
    stages = -(-length // STAGE)
    for at in (0, 1, stages // 3, stages // 2, stages - 2):
        for times in (0, 2):
            weight = np.ones(stages, int)
            weight[at] = times
            out, lse = count_errors(*row(length, d, weight, seed=at))
            assert out > 2 and lse > 2


@pytest.mark.parametrize("length", [9001, 31200, 60000])
@pytest.mark.parametrize("d", [64, 128])
def test_a_stage_in_anothers_place_shows(length, d):
    stages = -(-length // STAGE)
    weight = np.ones(stages, int)
    weight[stages // 2], weight[stages // 2 + 1] = 0, 2
    out, lse = count_errors(*row(length, d, weight))
    assert out > 2 and lse == 0.0
