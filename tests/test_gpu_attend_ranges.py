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


@pytest.mark.parametrize("heads", [257, 960, 1000, 1024])
def test_as_many_heads_as_a_call_takes(heads):
    call(2, heads, 150, 170, "f16" if heads % 2 else "bf16", seed=heads, pad=0.1, weights=True)


def test_as_many_heads_and_rows_as_a_call_takes():
    call(1, 1024, 8192, 8192, "bf16", seed=1, weights=True)


@pytest.mark.parametrize("R,heads,k", [(8192, 3, 5), (8192, 66, 70), (8191, 17, 1)])
def test_as_many_requests_as_a_call_takes(R, heads, k):
    """Compared: the first, the last, those around whole waves, and some between."""
    D, tokens = k + 4, 2 * k + 20
    rows = make_rows(R * D, "bf16", 1).view(R, D, 416)
    q = make_q(R, heads, "bf16", 2)
    order = torch.rand((R, D), device="cuda").argsort(1)
    ids = order[:, :k].int().contiguous()
    ids[::7, 0] = -1
    pos = torch.rand((R, tokens), device="cuda").argsort(1)[:, :k].int().contiguous()
    out = torch.empty((R, heads, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((R, heads), device="cuda")
    acc = torch.rand((R, tokens), device="cuda")
    before, status = acc.clone(), torch.zeros(R, dtype=torch.int32, device="cuda")
    H.attend(q, rows, ids, out, 0.05, lse=lse, weights=acc, positions=pos, status=status)
    some = sorted({0, 1, 151, 152, 153, 4095, 4096, R - 2, R - 1, *range(R // 152 * 152 - 3, min(R // 152 * 152 + 3, R)),
                   *np.random.default_rng(R).integers(0, R, 100).tolist()})
    check(q, rows, ids, out, float(np.float32(0.05)), "bf16", lse, acc, before, pos, requests=some)
    assert (status == 0).all()
