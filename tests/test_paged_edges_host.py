"""Edges of the paged cache without a GPU."""
import numpy as np

import paged_ref as ref


def test_forced_pages_come_before_infinite_scores():
    """Ten pages, six of them of scale inf, four kept: the first and the last are among them."""
    zero = np.zeros((10, 128), dtype=np.int64)
    scale = np.ones(10, dtype=np.float32)
    scale[2:8] = np.inf
    q = np.ones((1, 128), dtype=np.float32)
    assert ref.select(q, zero, zero, scale, 4, 1, 1) == [0, 2, 3, 9]
    assert ref.select(q, zero, zero, scale, 1, 0, 1) == [9]
    assert ref.select(q, zero, zero, scale, 1, 1, 0) == [0]
    assert ref.select(q, zero, zero, scale, 4, 0, 0) == [2, 3, 4, 5]
    scale[[0, 9]] = -1  # not even a page outside the pool loses its place
    assert ref.select(q, zero, zero, scale, 3, 1, 1) == [0, 2, 9]
