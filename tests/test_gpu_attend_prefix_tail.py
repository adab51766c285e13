"""Attention over a shared prefix with a long flat tail of small weights, as far as the
longest prefix: what the tail adds up to is in the output as it is in the sum.

Each weight enters the second product in the model's type: half a step of itself, or,
in f16 below 2^-14, 2^-25 absolutely.  The largest is at least 2^7 there, so that a tail
of n weights is off by at most n 2^-32 of the largest (2^-12 with 2^20), not by n 2^-25.
Sums: the weights of a tile (a few steps) and the tiles, one step each, at most 8,192; the
second product adds 16 rows a step, at most 65,536 steps of at most 2^-23 (the tensor
core's sums may be cut off where a rounding would go up)."""

import math

import numpy as np
import pytest
import torch

import pages_model as M
from hierarchical_sparse_kv_request_gb300 import hisparse as H
from test_gpu_attend_prefix import HALF, TYPES

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads", [(1, 3), (19, 512)])      # tiles shared by all pairs; a group or more a pair
@pytest.mark.parametrize("n", [40000, 1 << 20])
@pytest.mark.parametrize("below", [24.4, 25.01, 28.0, 32.5])
def test_a_flat_tail_below_one_row(below, n, heads, dtype):
    """Row 0 once, at a place in the middle, the others 2^-below of it."""
    x = torch.zeros((2, 576), device="cuda")
    x[1, 512] = -below * math.log(2.0)
    x[0, :256], x[1, :256] = 0.0, 1.0               # out is the tail's share
    x[0, 256:512], x[1, 256:512] = 1.0, 0.0         # and the top's
    x16 = x.to(TYPES[dtype])
    rows = torch.empty((2, M.ROW16), dtype=torch.uint8, device="cuda")
    H.norm_rows(x16, rows)
    table = torch.ones(n, dtype=torch.int32, device="cuda")
    table[n // 2 + 77] = 0
    q = torch.zeros((*heads, 576), dtype=TYPES[dtype], device="cuda")
    q[:, :, 512] = 1.0
    out = torch.empty((*heads, 512), dtype=TYPES[dtype], device="cuda")
    lse = torch.empty(heads, device="cuda")
    H.attend_prefix(q, rows, table, 1, n, out, 1.0, lse=lse)
    tail = (n - 1) * math.exp(float(x16[1, 512]))
    share = tail / (1 + tail)
    steps = n / 128
    sums = (steps + 100) * U32 + n / 16 * 2.0 ** -23
    off = (HALF[dtype] + sums) * share + n * 2.0 ** -32 * (dtype == "f16")
    got = out.double()
    err = (got[..., :256] - share).abs().max().item()
    assert err <= HALF[dtype] * share + (1 + HALF[dtype]) * off + 2.0 ** -25, (err / share, off / share)
    err = (got[..., 256:] - (1 - share)).abs().max().item()
    assert err <= HALF[dtype] + 2 * (HALF[dtype] + sums), err
    assert (lse.double() - math.log1p(tail)).abs().max() <= (steps + 100) * U32 * (1 + below)
    print("tail", below, n, heads, dtype, "relative error", ((got[..., :256] - share).abs().max() / share).item(), "lse",
          (lse.double() - math.log1p(tail)).abs().max().item())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("step", [0.5, 2.9, 3.1, 5.9, 6.1, 8.1, 14.0, 20.0])
def test_the_top_rises_a_little_in_every_tile(step, dtype):
    """In units of a factor of 2, over 40 tiles: the reference follows, before a weight is too
    large for its type."""
    n = 40 * 128
    up = torch.arange(n, device="cuda") // 128 * step * math.log(2.0)
    x = torch.zeros((n, 576), device="cuda")
    x[:, 512] = up / 16
    g = torch.Generator(device="cuda").manual_seed(2)
    x[:, :512] = torch.randn((n, 512), generator=g, device="cuda")
    x16 = x.to(TYPES[dtype])
    rows = torch.empty((n, M.ROW16), dtype=torch.uint8, device="cuda")
    H.norm_rows(x16, rows)
    heads = 76 * 128        # a pair goes through all tiles
    q = torch.zeros((19, 512, 576), dtype=TYPES[dtype], device="cuda")
    q[:, :, 512] = 16.0
    out = torch.empty((19, 512, 512), dtype=TYPES[dtype], device="cuda")
    lse = torch.empty((19, 512), device="cuda")
    table = torch.arange(n, dtype=torch.int32, device="cuda")
    H.attend_prefix(q, rows, table, 1, n, out, 1.0, lse=lse)
    s = 16.0 * x16[:, 512].double()
    p = torch.exp(s - s.max())
    want, spread = (p @ x16[:, :512].double()) / p.sum(), (p @ x16[:, :512].double().abs()) / p.sum()
    ds = 8 * U32 * s.abs().max()
    tol = HALF[dtype] * want.abs() + (1 + HALF[dtype]) * (torch.expm1(2 * ds) + HALF[dtype] + 1000 * U32) * spread + 2.0 ** -25
    assert ((out.double() - want).abs() <= tol).all()
    w_lse = s.max() + torch.log(p.sum())
    assert (lse.double() - w_lse).abs().max() <= ds + 1000 * U32 + 16 * U32 * w_lse.abs()
    assert heads == out.shape[0] * out.shape[1]
