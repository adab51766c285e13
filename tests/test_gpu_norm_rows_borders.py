"""Codes and scales of normalised rows where they are easily the wrong ones: values
exactly on a border between two codes, and means at the ends of the range that the calls
promise them for."""

import numpy as np
import pytest
import torch

import pages_model as M
from hierarchical_sparse_kv_request_gb300 import hisparse as H
from test_gpu_norm_rows import TYPES, exact_values, make

pytestmark = pytest.mark.gpu
CODES = {M.ROW4: np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6]), M.ROW8: M.E4M3[:127]}


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def norm(x, w, eps, row):
    rows = torch.empty((x.shape[0], row), dtype=torch.uint8, device="cuda")
    H.norm_rows(x, rows, weight=w, eps=eps)
    return rows.cpu().numpy()


def nearest_even(v, table):
    hi = np.clip(np.searchsorted(table, v), 1, len(table) - 1)
    a, b = v - table[hi - 1], table[hi] - v
    return table[np.where((a < b) | ((a == b) & (hi % 2 == 1)), hi - 1, hi)]


@pytest.mark.parametrize("row", [M.ROW4, M.ROW8])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("size", [1.0, 3.0, 0.625, 11.0, 1.4375])
def test_values_exactly_on_a_border(size, dtype, row):
    """All |x| the same and eps 0: y is the weight, with the sign of x.  Weights are the
    borders between neighbouring codes, times powers of two that bring groups to scale 1."""
    codes = CODES[row]
    codes = codes[codes >= 2.0 ** -6] if row == M.ROW8 else codes
    borders = (codes[1:] + codes[:-1]) / 2
    top = codes[-1]
    group = 128 if row == M.ROW8 else 16
    w = np.resize(borders, 512)
    w[::group] = top                               # the group's scale is 1
    w16 = torch.from_numpy(w).to(TYPES[dtype]).cuda()
    assert np.array_equal(w16.double().cpu().numpy(), w)          # borders are exact in both types
    x = torch.full((8, 576), size, dtype=TYPES[dtype], device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    x[4:] *= torch.where(torch.rand((4, 576), generator=g, device="cuda") < 0.5, -1, 1).to(TYPES[dtype])
    x[1::2] *= 2
    rows = norm(x, w16, 0.0, row)
    got, _ = M.values_of_rows(rows, dtype)
    want = nearest_even(w, codes) if row == M.ROW4 else nearest_even(w, CODES[row])
    assert np.array_equal(np.abs(got), np.broadcast_to(want, got.shape))


@pytest.mark.parametrize("k", [-3, 0, 4])
def test_a_largest_magnitude_exactly_on_a_border_of_the_scale(k):
    """y is the weight: 448 of a power of two keeps that power as its scale."""
    w = torch.full((512,), 0.25 * 2.0 ** k, dtype=torch.bfloat16, device="cuda")
    w[::128] = 448.0 * 2.0 ** k
    for size in (1.0, 3.0, 0.625, 11.0, 1.4375):
        x = torch.full((3, 576), size, dtype=torch.bfloat16, device="cuda")
        rows = norm(x, w, 0.0, M.ROW8)
        scale = np.ascontiguousarray(rows[:, 512:528]).view(np.float32)
        assert (scale == 2.0 ** k).all(), (size, scale)
        # (6 times the border between two e4m3 values: the even one)
        w4 = torch.full((512,), 2.0 ** -6, dtype=torch.bfloat16, device="cuda")
        w4[::16] = 6 * 1.0625 * 2.0 ** k
        scale4 = M.E4M3[norm(x, w4, 0.0, M.ROW4)[:, 256:288]]
        assert (scale4 == 2.0 ** k).all(), (size, scale4)


@pytest.mark.parametrize("row", [M.ROW4, M.ROW8])
@pytest.mark.parametrize("power", [-50, -49, 48, 49])
def test_means_at_the_ends_of_the_range(row, power):
    """Means between 2^-100 and 2^100, eps 0: every code is that of the exact value."""
    g = torch.Generator(device="cuda").manual_seed(power + 100)
    x = torch.randn((20000, 576), generator=g, device="cuda").to(torch.bfloat16)
    mean = x[:, :512].double().square().mean(1)
    x = x[(mean > 1) & (mean < 2)][:8000] * 2.0 ** power
    w = (1 + 0.2 * torch.randn((512,), generator=g, device="cuda")).to(torch.bfloat16)
    rows = norm(x, w, 0.0, row)
    y = M.norm(x[:, :512].double().cpu().numpy(), w.double().cpu().numpy(), 0.0)
    got, _ = M.values_of_rows(rows, "bf16")
    assert x.shape[0] > 4000
    assert np.array_equal(got, exact_values(y, row))
