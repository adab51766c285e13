"""Attention at the ends of its ranges: queries and scales as large or small as
their types hold, many heads, many requests.  Tolerances as in
test_gpu_attend.py, whose check() compares."""

import numpy as np
import pytest
import torch

from hierarchical_sparse_kv_request_gb300 import hisparse as H
from test_gpu_attend import TYPES, call, check, make_q, make_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def attend(q, rows, scale, k, dtype):
    """One call over k random rows a request, compared with the definition."""
    R, D = rows.shape[:2]
    ids = torch.stack([torch.randperm(D)[:k] for _ in range(R)]).int().cuda()
    out = torch.empty((R, q.shape[1], 512), dtype=TYPES[dtype], device="cuda")
    lse = torch.empty(q.shape[:2], device="cuda")
    H.attend(q, rows, ids, out, scale, lse=lse)
    check(q, rows, ids, out, float(np.float32(scale)), dtype, lse)


@pytest.mark.parametrize("top", [126, 127, 128])
def test_queries_up_to_the_largest_bf16_values(top):
    """Values just below 2^top; the scale brings scores back to ordinary size."""
    R, heads, k, D = 2, 9, 130, 140
    rows = make_rows(R * D, "bf16", 3).view(R, D, 416)
    g = torch.Generator(device="cuda").manual_seed(top)
    q = 1.98 * torch.rand((R, heads, 576), generator=g, device="cuda", dtype=torch.float64) - 0.99
    q[:, :, 7] = 0.99
    q = (q * 2.0 ** top).to(torch.bfloat16)
    assert torch.isfinite(q).all()
    attend(q, rows, 2.0 ** (-4 - top), k, "bf16")


@pytest.mark.parametrize("R,heads,k", [(1, 1, 90), (1, 1, 1000), (1, 20, 300), (3, 1, 300)])
def test_strides_of_a_single_head_or_request_mean_nothing(R, heads, k):
    D = k + 9
    rows = make_rows(R * D, "bf16", 3).view(R, D, 416)
    q, out = make_q(R, heads, "bf16", 4), torch.empty((R, heads, 512), dtype=torch.bfloat16, device="cuda")

    def odd(x, n):
        return torch.as_strided(x, x.shape, (n * heads if R > 1 else 3, n if heads > 1 else 1, 1))

    odd_rows = torch.as_strided(rows, rows.shape, (D * 416 if R > 1 else 5, 416, 1))
    ids = torch.stack([torch.randperm(D)[:k] for _ in range(R)]).int().cuda()
    acc = torch.zeros((R, D), device="cuda")
    H.attend(odd(q, 576), odd_rows, ids, odd(out, 512), 0.05, weights=acc, positions=ids)
    check(q, rows, ids, out, float(np.float32(0.05)), "bf16", None, acc, torch.zeros_like(acc), ids)
