"""Attention with a scale that is no number: NaN where there is a row to weigh,
and what an empty request always gets where there is none."""

import pytest
import torch

from hierarchical_sparse_kv_request_gb300 import hisparse as H
from test_gpu_attend import TYPES, make_q, make_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("heads,k", [(20, 50), (20, 700), (130, 700)])
def test_a_nan_scale_gives_nan(dtype, heads, k):
    R, D = 3, k + 10
    rows = make_rows(R * D, dtype, 3).view(R, D, 416)
    q = make_q(R, heads, dtype, 4)
    ids = torch.stack([torch.randperm(D)[:k] for _ in range(R)]).int().cuda()
    ids[0, ::3] = -1
    ids[1] = -1
    out = torch.full((R, heads, 512), 7.0, dtype=TYPES[dtype], device="cuda")
    lse = torch.zeros((R, heads), device="cuda")
    H.attend(q, rows, ids, out, float("nan"), lse=lse)
    assert torch.isnan(out[[0, 2]]).all() and torch.isnan(lse[[0, 2]]).all()
    assert (out[1] == 0).all() and (lse[1] == float("-inf")).all()
