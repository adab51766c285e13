"""Attention over the sub-steps of a speculative verification: three swap-ins of
the same layer are resolved before any of them is attended, with the rows of the
earlier ones protected, so that every sub-step's ids still name its rows."""

import numpy as np
import pytest
import torch

from hierarchical_sparse_kv_request_gb300 import hisparse as H
from test_gpu_attend import check, make_q, make_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def test_sub_steps_with_protected_rows():
    R, k, D, tokens, heads, steps = 4, 100, 400, 1500, 20, 3
    hs = H.HiSparse(R, 1, H.ROW4_BYTES, k, D, host_to_device_ratio=4, host_capacity=[tokens] * R)
    rows = make_rows(R * tokens, "bf16", 5).view(R, tokens, 416)
    for r in range(R):
        hs.host_rows(0, r)[:] = rows[r].cpu().numpy()
    seq = torch.full((R,), tokens, dtype=torch.int32, device="cuda")
    hs.prefill(seq)
    hs.set_protected_calls(steps - 1)
    weights = torch.zeros((R, tokens), device="cuda")
    for _ in range(3):
        topk = [torch.stack([torch.randperm(tokens)[:k] for _ in range(R)]).int().cuda() for _ in range(steps)]
        ids = [torch.empty((R, k), dtype=torch.int32, device="cuda") for _ in range(steps)]
        for n in range(steps):
            hs.swap_in(0, topk[n], seq, ids[n])
        for n in range(steps):
            q = make_q(R, heads, "bf16", n)
            out = torch.empty((R, heads, 512), dtype=torch.bfloat16, device="cuda")
            before = weights.clone()
            hs.attend(0, q, ids[n], out, 0.05, weights=weights, positions=topk[n])
            check(q, rows, topk[n], out, float(np.float32(0.05)), "bf16", None, weights, before, topk[n])
    assert not any(int(s) for s in hs.status())
    hs.close()
