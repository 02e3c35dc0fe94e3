"""The join of a decode step whose cache is split over workgroups: odd counts and widths, and pages that
are not there."""

import pytest

import test_gpu_attn_step as base

pytestmark = pytest.mark.gpu

# heads, groups, dim, lengths, capacity, page (0: dense), window
CASES = [
    (1, 1, 64, [1279], 1280, 0, 0),  # an odd number of splits
    (3, 3, 7, [3000, 1], 3001, 0, 0),
    (2, 1, 50, [4000, 900, -1], 4096, 100, 0),
    (9, 3, 36, [2500, 0], 2560, 17, 2200),
    (17, 1, 128, [30000], 30001, 1, 0),  # more splits than are read ahead, two blocks of heads
    (1, 1, 1, [700], 701, 0, 600),
]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("name", list(base.TYPES))
def test_step(case, name):
    base.test_step(case, name)
