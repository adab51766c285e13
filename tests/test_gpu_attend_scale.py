"""Attention with scales at the ends of their type.  Tolerances as in
test_gpu_attend.py, whose check() compares."""

import numpy as np
import pytest
import torch

from hierarchical_sparse_kv_request_gb300 import hisparse as H
from test_gpu_attend import check, make_rows

pytestmark = pytest.mark.gpu
R, HEADS, K, D = 3, 20, 130, 140


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def attend(q, scale, hole=None):
    rows = make_rows(R * D, "bf16", 3).view(R, D, 416)
    ids = torch.stack([torch.randperm(D)[:K] for _ in range(R)]).int().cuda()
    if hole is not None:
        ids[hole] = -1
    out = torch.empty((R, HEADS, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((R, HEADS), device="cuda")
    H.attend(q, rows, ids, out, scale, lse=lse)
    return rows, ids, out, lse


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("scale", [2.3e38, 3.0e38, 3.4e38])
def test_scales_up_to_the_largest(scale, sign):
    """With queries that bring the scores back to ordinary size."""
    g = torch.Generator(device="cuda").manual_seed(5)
    q = torch.randn((R, HEADS, 576), generator=g, device="cuda", dtype=torch.float64) * 1e-38 / 24
    q = (3 * q).to(torch.bfloat16)
    rows, ids, out, lse = attend(q, sign * scale)
    check(q, rows, ids, out, float(np.float32(sign * scale)), "bf16", lse)
