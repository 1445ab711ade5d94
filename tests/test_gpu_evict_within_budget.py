"""Eviction in wide matrices, whose sequences take a cluster of blocks each:
sequences within their budget beside longer ones.  The former leave after the
cluster's first barrier, and many of their blocks have no entry to copy."""

import numpy as np
import pytest

import test_gpu_evict as base
from test_gpu_evict import dev  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("longest,budget", [(4200, 700), (9000, 2048), (20000, 1000), (66000, 3000)])
@pytest.mark.parametrize("in_place", [False, True])
def test_within_the_budget_beside_longer_ones(dev, longest, budget, in_place):
    lens = [longest, budget, budget - 1, 0, 1, budget + 1, 33] + [budget // 3] * 5
    base.Problem(lens, budget, 4, 32, 1, seed=longest).check(dev, in_place=in_place)


def test_a_batch_that_evicts_nothing(dev):
    rng = np.random.default_rng(1)
    p = base.Problem([int(n) for n in rng.integers(0, 400, 300)], 400, 4, 16, 1, seed=2, extra=8000)
    # a table as wide as the matrix: clusters are chosen by both
    wide = np.full((300, 130), -1, np.int32)
    wide[:, :p.table.shape[1]] = p.table
    p.table = wide
    for _ in range(3):
        p.check(dev)
