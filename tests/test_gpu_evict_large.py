"""Freeing in hot buffers up to the largest, where a thread holds 32 slots."""

import pytest
import torch

from test_gpu_evict import test_evict_frees_and_the_resolver_goes_on as frees

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("protect", [0, 2])
@pytest.mark.parametrize("D,k,lens", [(16384, 900, [30000, 16500]), (16385, 900, [30000, 16385, 16386]),
                                      (20000, 2000, [45000, 21000]), (32768, 4000, [60000, 33000])])
def test_evict_frees_in_the_largest_buffers(D, k, lens, protect):
    frees(D, k, lens, protect)
