"""Attention over a shared prefix with scores so large that their 32-bit steps are
many units: the largest one's row is the output, whatever the product with the scale
was rounded by.  Scores here are products of two values, exact before the scale."""

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


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n", [100, 1000])
@pytest.mark.parametrize("scale", [1e3, -3e4, 1e5, 7e5, 3e6, -1.1e7, 5e7, 1e8, 1e9, -1e10, 1e15, 1e25, 3e35])
def test_the_largest_score_takes_all(scale, n, dtype):
    """Each head q = a e0 with its own a, rows with a value of their own in place 0 (at
    least 1/256 from the next), half of them twice: the output is the mean of the best row's
    two, or that row."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.zeros((n, 576), device="cuda")
    x[:, 1:] = torch.randn((n, 575), generator=g, device="cuda")
    values = (1 + torch.arange(128, device="cuda") / 128.0)              # exact in both types
    some = values[torch.randint(0, 120, (n,), generator=g, device="cuda")] - 1.5
    x[:, 0] = some
    x[n // 3, 0], x[2 * n // 3, 0] = 1.9375 - 1.5, 1.9375 - 1.5          # the largest, twice
    x[n // 2, 0] = -0.625                                                # the smallest, once
    rows16 = x.to(TYPES[dtype])
    rows = torch.empty((n, M.ROW16), dtype=torch.uint8, device="cuda")
    H.norm_rows(rows16, rows)
    heads = 70
    a = 1 + torch.arange(heads, device="cuda") / 128.0
    q = torch.zeros((1, heads, 576), dtype=TYPES[dtype], device="cuda")
    q[0, :, 0] = a.to(TYPES[dtype])
    q[0, 1::2, 0] *= -1
    order = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
    out = torch.empty((1, heads, 512), dtype=TYPES[dtype], device="cuda")
    lse = torch.empty((1, heads), device="cuda")
    H.attend_prefix(q, rows, order, 1, n, out, scale, lse=lse)
    s = float(np.float32(scale))
    lat = rows16[:, :512].double()
    score = s * q[0, :, 0].double()[:, None] * rows16[:, 0].double()[None]
    top = score.amax(1, keepdim=True)
    gap = torch.where(score == top, float("inf"), top - score).amin()
    assert gap > 3      # (s / 1024 at 10^3: the rest weighs at most n e^-gap, counted below)
    p = torch.exp(score - top)
    total = p.sum(1, keepdim=True)
    want = (p / total) @ lat
    spread = (p / total) @ lat.abs()
    # a score is one rounding of its product with the factor, and the factor's two: 3 half
    # steps of the score, which the other rows' weights get in their logarithm
    ds = 3 * U32 * score.abs().amax()
    rest = (total - (score == top).sum(1, keepdim=True)) / total
    tol = (HALF[dtype] * want.abs() + (1 + HALF[dtype]) * (HALF[dtype] + 200 * U32) * spread + 2.0 ** -25
           + torch.expm1(2 * ds).clamp(max=1e9) * rest * lat.abs().amax())
    assert torch.isfinite(out).all()
    assert ((out[0].double() - want).abs() <= tol).all()
    w_lse = top[:, 0] + torch.log(total[:, 0])
    assert ((lse[0].double() - w_lse).abs() <= 6 * U32 * w_lse.abs() + 200 * U32 + torch.expm1(2 * ds).clamp(max=1e9) * rest[:, 0]).all()


@pytest.mark.parametrize("scale", [2.3e38, 3.4e38, -3.4e38])
def test_largest_scales_in_f16(scale):
    """f16's smallest queries and rows: scores near 2^127 times 2^-48, one row's far above
    the others': the output is that row."""
    rows = torch.zeros((64, 576), dtype=torch.float16, device="cuda")
    rows[:, 0] = torch.arange(64, device="cuda") * 2.0 ** -24
    rows[:, 1:512] = torch.randn((64, 511), generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    packed = torch.empty((64, M.ROW16), dtype=torch.uint8, device="cuda")
    H.norm_rows(rows, packed)
    q = torch.zeros((1, 70, 576), dtype=torch.float16, device="cuda")
    q[0, :, 0] = 2.0 ** -24
    out = torch.empty((1, 70, 512), dtype=torch.float16, device="cuda")
    lse = torch.empty((1, 70), device="cuda")
    H.attend_prefix(q, packed, torch.arange(4, dtype=torch.int32, device="cuda"), 16, 64, out, scale, lse=lse)
    best = 63 if scale > 0 else 0
    assert torch.equal(out, rows[best, :512].expand_as(out))
    want = float(np.float32(scale)) * 2.0 ** -48 * best
    assert (lse.double() - want).abs().max() <= 4 * 2.0 ** -24 * abs(want) + 2.0 ** -20


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("order", ["rising", "falling", "shuffled"])
@pytest.mark.parametrize("scale", [1e4, 3e6, 1e9, -1e9, 1e20, 3e38])
def test_a_pair_goes_through_several_tiles(scale, order, dtype):
    """Heads for all pairs, eight tiles each, the reference moving between them; joined with
    parts far above (even heads), far below (odd ones), and of no weight."""
    n, R, heads = 1000, 19, 512
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((n, 576), generator=g, device="cuda")
    x[:, 0] = (torch.arange(n, device="cuda") // 10) / 128.0 - 0.4       # tens of rows alike
    x[-10:-1, 0], x[1:10, 0] = 0.3, -0.3                                 # but the largest and the smallest
    x[:, 512:] = 0
    x16 = x.to(TYPES[dtype])
    rows = torch.empty((n, M.ROW16), dtype=torch.uint8, device="cuda")
    H.norm_rows(x16, rows)
    table = {"rising": torch.arange(n), "falling": torch.arange(n).flip(0),
             "shuffled": torch.randperm(n, generator=torch.Generator().manual_seed(1))}[order].to(torch.int32).cuda()
    q = torch.zeros((R, heads, 576), dtype=TYPES[dtype], device="cuda")
    size = 2.0 ** -10 if abs(scale) > 1e38 else 1.0                      # (scores stay in range)
    q[:, :, 0] = size * torch.where(torch.arange(heads, device="cuda") % 4 < 2, 1.0, -1.0).to(TYPES[dtype])
    s32 = float(np.float32(scale))
    score = s32 * q[0, :4, 0].double()[:, None] * x16[:, 0].double()[None]      # (the same for every fourth head)
    top = score.amax(1)
    part = torch.randn((R, heads, 512), generator=g, device="cuda").to(TYPES[dtype])
    lse = (top.repeat(heads // 4) + torch.where(torch.arange(heads, device="cuda") % 2 == 0, 1.0, -1.0) * top.abs().max() / 4)
    part_lse = lse.float().expand(R, heads).clone()
    part_lse[5] = -float("inf")
    part[5] = float("nan")
    out, sums = torch.empty((R, heads, 512), dtype=TYPES[dtype], device="cuda"), torch.empty((R, heads), device="cuda")
    alone, sums0 = torch.empty_like(out), torch.empty_like(sums)
    H.attend_prefix(q, rows, table, 1, n, alone, scale, lse=sums0)
    H.attend_prefix(q, rows, table, 1, n, out, scale, lse=sums, part=part, part_lse=part_lse)
    # at 10^4 the next score is 10^4 / 256 or more away: what it weighs is below f16's step
    weights = (score == top[:, None]).double()
    weights /= weights.sum(1, keepdim=True)
    want = (weights @ x16[:, :512].double()).repeat(heads // 4, 1)
    spread = (weights @ x16[:, :512].double().abs()).repeat(heads // 4, 1)
    tol = HALF[dtype] * want.abs() + (1 + HALF[dtype]) * (HALF[dtype] + 200 * U32) * spread + 2.0 ** -25 + 1e-12
    assert ((alone.double() - want).abs() <= tol).all()
    count = (score == top[:, None]).sum(1).double().log().repeat(heads // 4)
    w = top.repeat(heads // 4) + count
    assert ((sums0.double() - w).abs() <= 6 * U32 * w.abs() + 200 * U32).all()
    rest = [r for r in range(R) if r != 5]
    assert torch.equal(out[5], alone[5]) and torch.equal(sums[5], sums0[5])
    assert torch.equal(out[rest][:, ::2], part[rest][:, ::2])
    assert torch.equal(out[rest][:, 1::2], alone[rest][:, 1::2])
    assert ((sums[rest][:, ::2] - part_lse[rest][:, ::2]).abs() <= 4 * U32 * part_lse[rest][:, ::2].abs()).all()
