"""The signs of normalised rows' codes: those of the values, also of zeros."""

import numpy as np
import pytest
import torch

import pages_model as M
from hierarchical_sparse_kv_request_gb300 import hisparse as H
from test_gpu_norm_rows import make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def signs(rows, row):
    """bool [n][512]: the sign bits of the codes."""
    if row == M.ROW8:
        return rows[:, :512] >= 128
    bits = np.empty((rows.shape[0], 512), dtype=bool)
    bits[:, 0::2], bits[:, 1::2] = rows[:, :256] & 8, rows[:, :256] & 128
    return bits


@pytest.mark.parametrize("row", [M.ROW4, M.ROW8])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("spread", [1.0, 2.0 ** -6])
def test_the_sign_of_zeros_and_of_values_that_become_zero(dtype, row, spread):
    """In every row, whether or not one of its other codes took a second look."""
    x, w = make(20000, dtype, 21, spread)
    x[:, 3:512:7] = 0
    x[:, 3:512:14] = -0.0
    x[:, 1:512:11] *= 2.0 ** -12                   # codes of 0 with a sign
    x[::5, 128:256] = -0.0                         # groups of zeros, whose scale is 0 or the least
    w[5::9] *= -1
    rows = torch.empty((x.shape[0], row), dtype=torch.uint8, device="cuda")
    H.norm_rows(x, rows, weight=w, eps=1e-5)
    rows = rows.cpu().numpy()
    want = (torch.signbit(x[:, :512]) ^ torch.signbit(w)).cpu().numpy()
    assert np.array_equal(signs(rows, row), want)
