"""Attention whose workspace is allocated by the call itself, on a stream that
is not the current one: neither side's later allocations meet the other's work.
Tolerances as in test_gpu_attend.py, whose check() compares."""

import numpy as np
import pytest
import torch

from hierarchical_sparse_kv_request_gb300 import hisparse as H
from test_gpu_attend import check, make_q, make_rows

pytestmark = pytest.mark.gpu
CYCLES = 20_000_000      # of a delay, some 10 ms: the host is done long before


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("kind", ["Stream", "address"])
@pytest.mark.parametrize("R,heads,k", [(4, 100, 400), (170, 5, 130)])
def test_a_workspace_of_the_call_on_another_stream(R, heads, k, kind):
    D = k + 30
    rows = make_rows(R * D, "bf16", 1).view(R, D, 416)
    ids = torch.stack([torch.randperm(D)[:k] for _ in range(R)]).int().cuda()
    q = make_q(R, heads, "bf16", 2)
    out = torch.empty((R, heads, 512), dtype=torch.bfloat16, device="cuda")
    acc = torch.zeros((R, D), device="cuda")
    size = H.attend_workspace_bytes(R, heads, k, True)
    side = torch.cuda.Stream()
    old = torch.full((size,), 3, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(CYCLES)            # on the current stream: `old` is read late
    kept = old.clone()
    del old
    with torch.cuda.stream(side):
        torch.cuda._sleep(2 * CYCLES)    # and the call works later still
    H.attend(q, rows, ids, out, 0.05, weights=acc, positions=ids,
             stream=side if kind == "Stream" else side.cuda_stream)
    later = [torch.full((size,), 7, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert (kept == 3).all()
    assert all((x == 7).all() for x in later)
    check(q, rows, ids, out, float(np.float32(0.05)), "bf16", None, acc, torch.zeros_like(acc), ids)


def test_the_default_stream_by_its_address():
    R, heads, k, D = 3, 16, 200, 230
    rows = make_rows(R * D, "bf16", 1).view(R, D, 416)
    ids = torch.stack([torch.randperm(D)[:k] for _ in range(R)]).int().cuda()
    q = make_q(R, heads, "bf16", 2)
    out = torch.empty((R, heads, 512), dtype=torch.bfloat16, device="cuda")
    acc = torch.zeros((R, D), device="cuda")
    torch.cuda.synchronize()
    H.attend(q, rows, ids, out, 0.05, weights=acc, positions=ids, stream=0)
    torch.cuda.synchronize()
    check(q, rows, ids, out, float(np.float32(0.05)), "bf16", None, acc, torch.zeros_like(acc), ids)


def test_a_handle_knows_its_device():
    hs = H.HiSparse(2, 1, H.ROW4_BYTES, 4, 8, host_to_device_ratio=2, host_capacity=[16, 16])
    assert hs.device == torch.cuda.current_device()
    hs.close()
