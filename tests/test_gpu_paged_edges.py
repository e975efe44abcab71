"""Edges of the paged-cache operators on the GPU: calls that the interface allows and
that test_gpu_paged.py does not make.  Plain implementations and tolerances as there.
"""
import numpy as np
import pytest

from long_context_sparse_rtp_b200 import rtp_paged_plan
from test_gpu_paged import _gpu, check_plan, ints  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------- a batch without tokens
@pytest.mark.parametrize("B", [1, 1024, 1025, 2500])
@pytest.mark.parametrize("release", [False, True])
def test_plan_without_tokens(B, release):
    """max_tokens = 0: nothing is taken, released pages go back, requests that want tokens are
    refused."""
    g = np.random.default_rng(B)
    lens = g.integers(0, 60, B).tolist()
    rel = (g.random(B) < 0.5).astype(int).tolist() if release else None
    for in_place in (False, True):
        check_plan(lens, [0] * B, ps=16, width=5, free=7, cap=12000, max_tokens=0, release=rel,
                   in_place=in_place)
    check_plan(lens, (g.integers(0, 2, B)).tolist(), ps=16, width=5, free=7, cap=12000, max_tokens=0,
               release=rel)


def test_plan_without_tokens_pads_its_spans():
    B = 2000
    spans = ints([[9, 9, 9, 9]] * 5)
    r = rtp_paged_plan(ints([3] * B), ints([0] * B), ints([[1]] * B), ints([0]), ints([0]), page_size=16,
                       max_tokens=0, out=dict(spans=spans))
    assert r["spans"].tolist() == [[-1, 0, 0, 0]] * 5
