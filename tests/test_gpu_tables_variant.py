"""Block tables on both sides of where one CTA leaves the pages to a cluster, against the
definition on lists: few requests with many pages, that go and come back, with tokens
placed and without."""

import numpy as np
import pytest

from test_gpu_page_tables import Both

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch

    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("R,W", [(1, 32768), (1, 32769), (5, 6553), (5, 6554), (32, 1024), (32, 1025), (25, 3000)])
@pytest.mark.parametrize("shared", [0, 7])
def test_all_pages_go_and_come_back(R, W, shared):
    rng = np.random.default_rng(W)
    b = Both(R, W, 1, R * W, shared=shared, rng=rng, stride=3)
    full = np.full(R, W)
    b.call(full)
    b.call(np.zeros(R, dtype=int))
    b.call(full, np.ones(R, dtype=int), 2 * R)
    half = rng.integers(0, W + 1, R)
    b.call(half, np.minimum(half, 3), 4 * R)
    b.call(np.where(np.arange(R) % 3 == 1, -1, W))
    b.call(half)
