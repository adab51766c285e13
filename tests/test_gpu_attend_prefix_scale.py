"""Attention over a shared prefix with scales and queries at the ends of their types,
brought back to ordinary scores by each other.  Tolerances as in
test_gpu_attend_prefix.py, whose check() compares: a query times a power of two is
exact, so that nothing is rounded that is not counted there."""

import numpy as np
import pytest
import torch

import pages_model as M
from hierarchical_sparse_kv_request_gb300 import hisparse as H
from test_gpu_attend_prefix import TYPES, check, make_part, make_rows, named

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def attend(q, n, scale, dtype="bf16", row=M.ROW8, part=True, bs=16, rows=None):
    R, heads, _ = q.shape
    used = -(-n // bs)
    rng = np.random.default_rng(n)
    if rows is None:
        rows = make_rows((used + 2) * bs, dtype, row, 3)
    table = torch.from_numpy(rng.permutation(used + 2)[:used].astype(np.int32)).cuda()
    table[::5] = -1
    p, pl = make_part(R, heads, dtype, 7) if part else (None, None)
    out = torch.empty((R, heads, 512), dtype=TYPES[dtype], device="cuda")
    lse = torch.empty((R, heads), device="cuda")
    H.attend_prefix(q, rows, table, bs, n, out, scale, lse=lse, part=p, part_lse=pl)
    check(q, named(rows, table, bs, n), out, lse, float(np.float32(scale)), dtype, p, pl)


def randn(R, heads, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((R, heads, 576), generator=g, device="cuda", dtype=torch.float64)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("scale", [1e30, 2.3e38, 3.0e38, 3.4e38])
@pytest.mark.parametrize("n", [130, 1500])
def test_scales_up_to_the_largest(n, scale, sign):
    attend((3 * randn(3, 20, 5) / scale / 24).to(torch.bfloat16), n, sign * scale)


@pytest.mark.parametrize("scale", [1e-30, 1e-37, 5e-39, 1e-40, 1e-42])
def test_scales_down_to_the_smallest(scale):
    """(times the largest queries: scores of some units down to 10^-3)"""
    top = min(3 / scale / 24, 5e37)
    attend((top * randn(3, 20, 6)).to(torch.bfloat16), 700, scale)


def test_a_scale_of_zero_weighs_all_rows_alike():
    for dtype, spread in (("bf16", 1e36), ("bf16", 1.0), ("f16", 1e4)):
        attend((spread * randn(3, 20, 8)).to(TYPES[dtype]), 300, 0.0, dtype, part=False)
        attend((spread * randn(3, 20, 8)).to(TYPES[dtype]), 300, -0.0, dtype)


@pytest.mark.parametrize("top", [126, 127, 128])
@pytest.mark.parametrize("row", [M.ROW4, M.ROW16])
def test_queries_up_to_the_largest_bf16_values(top, row):
    """Values just below 2^top; the scale brings scores back to ordinary size."""
    g = torch.Generator(device="cuda").manual_seed(top)
    q = 1.98 * torch.rand((2, 9, 576), generator=g, device="cuda", dtype=torch.float64) - 0.99
    q[:, :, 7] = 0.99
    q = (q * 2.0 ** top).to(torch.bfloat16)
    assert torch.isfinite(q).all()
    attend(q, 300, 2.0 ** (-4 - top), row=row)
