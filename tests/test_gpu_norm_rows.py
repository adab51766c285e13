"""Rows normalised and stored by slot, and read back, against the definition in 64
bits.  The roundings that the tolerances count:

- y: the mean of 512 squares in 32 bits (a lane's 16 terms, then 5 sums: 20 half steps
  of 2^-24, halved by the root), the root and its inverse (2), the last product (1):
  13 half steps, E = 13 * 2^-24 relative to y;
- 16-bit rows: one rounding more, half a step of the type;
- 8-bit rows: y / scale is exact but for y's error; a code is the nearest to it, half a
  step of 2^-4 of the value (and 2^-10 of the scale below 2^-6 of it, where codes are
  spaced evenly); where y's error takes the largest magnitude over a power of two, the
  group has twice or half the scale, and as good codes;
- 4-bit rows: the scale is the e4m3 value nearest to the largest magnitude / 6, half a
  step of 2^-4 of it (of 2^-10 below 2^-6); a code is the nearest to value / scale, at
  most 1, 1/2 or 1/4 away (above 4, above 2, below), and where the scale fell below the
  largest magnitude / 6, at most 6 * 2^-4 < 1 below it."""

import numpy as np
import pytest
import torch

import pages_model as M
import rows4_model as M4
from hierarchical_sparse_kv_request_gb300 import hisparse as H

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
E = 13 * 2.0 ** -24
ROWS = [M.ROW4, M.ROW8, M.ROW16]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def make(n, dtype, seed, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((n, 576), generator=g, device="cuda")
    x = x * torch.exp(0.5 * torch.randn((n, 1), generator=g, device="cuda")) * spread
    w = 1 + 0.2 * torch.randn((512,), generator=g, device="cuda")
    return x.to(TYPES[dtype]), w.to(TYPES[dtype])


def check(y, rope, rows, dtype, row):
    """The stored rows against y (float64 [n][512]) and the rope values' bits."""
    rows = rows.cpu().numpy()
    assert np.array_equal(rows[:, row - 128:], rope.contiguous().view(torch.uint8).cpu().numpy())
    got, _ = M.values_of_rows(rows, dtype)
    size = np.abs(y) * E
    if row == M.ROW16:
        tol = size + HALF[dtype] * np.abs(y) * (1 + E) + 2.0 ** -25 * (dtype == "f16") + 1e-38
    else:
        group = 128 if row == M.ROW8 else 16
        top = np.repeat(np.abs(y).reshape(len(y), -1, group).max(2), group, axis=1)
        if row == M.ROW8:
            scale = np.ascontiguousarray(rows[:, 512:528]).view(np.float32).astype(np.float64)
            want = M.scale8(np.abs(y).reshape(len(y), 4, 128).max(2))
            at_edge = np.abs(np.log2(top.reshape(len(y), 4, 128)[:, :, 0] / 448 / want)) < 2 * E
            near_half = np.abs(np.log2(np.maximum(top.reshape(len(y), 4, 128)[:, :, 0], 1e-300) / 224 / want)) < 2 * E
            assert ((scale == want) | (at_edge & (scale == 2 * want)) | (near_half & (scale == want / 2))).all()
            tol = size + 2.0 ** -4 * np.abs(y) * (1 + E) + 2.0 ** -10 * np.repeat(scale, 128, axis=1)
        else:
            scale = np.repeat(M.E4M3[rows[:, 256:288]], 16, axis=1)
            assert (np.abs(scale - top / 6) <= 2.0 ** -4 * scale + E * top + 2.0 ** -10).all()
            q = np.abs(y) * (1 + E) / np.maximum(scale, 2.0 ** -10)
            step = np.where(q > 4, 1.0, np.where(q > 2, 0.5, 0.25))
            tol = size + step * scale * (1 + E) + 6 * 2.0 ** -10 * (scale < 2.0 ** -6)
    bad = ~(np.abs(got - y) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], y[bad][:4], tol[bad][:4])


@pytest.mark.parametrize("row", ROWS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 127, 1000])
def test_rows_at_slots(n, dtype, row):
    x, w = make(n, dtype, n)
    count = 2 * n + 3
    g = torch.Generator(device="cuda").manual_seed(n + 1)
    slots = torch.randperm(count, generator=g, device="cuda")[:n].to(torch.int32)
    rows = torch.full((count, row), 0xA5, dtype=torch.uint8, device="cuda")
    H.norm_rows(x, rows, slots=slots, weight=w, eps=1e-5)
    y = M.norm(x[:, :512].double().cpu().numpy(), w.double().cpu().numpy(), float(np.float32(1e-5)))
    check(y, x[:, 512:], rows[slots.long()], dtype, row)
    untouched = torch.ones(count, dtype=torch.bool, device="cuda")
    untouched[slots.long()] = False
    assert (rows[untouched] == 0xA5).all()
    # and back
    values = torch.full((n, 576), 7.0, dtype=TYPES[dtype], device="cuda")
    H.gather_rows(rows, values, slots=slots)
    lat, rope = M.values_of_rows(rows[slots.long()].cpu().numpy(), dtype)
    assert np.array_equal(values[:, :512].double().cpu().numpy(), lat)
    assert np.array_equal(values[:, 512:].double().cpu().numpy(), rope)


def nearest(v, table):
    """The entries of table (rising; ties to the even one) nearest to v >= 0."""
    hi = np.clip(np.searchsorted(table, v), 1, len(table) - 1)
    a, b = v - table[hi - 1], table[hi] - v
    return table[np.where((a < b) | ((a == b) & (hi % 2 == 1)), hi - 1, hi)]


def exact_values(y, row):
    """What codes and scales of unlimited precision stand for."""
    group = 128 if row == M.ROW8 else 16
    g = np.abs(y).reshape(len(y), -1, group)
    top = g.max(2)
    codes = M.E4M3[:127] if row == M.ROW8 else np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    scale = (M.scale8(top) if row == M.ROW8 else nearest(np.minimum(top / 6, 448.0), M.E4M3[:127]))[:, :, None]
    q = np.minimum(g / np.where(scale > 0, scale, 1.0), codes[-1])
    return np.where(scale > 0, nearest(q, codes) * scale, 0.0).reshape(y.shape) * np.sign(y)


@pytest.mark.parametrize("row", [M.ROW4, M.ROW8])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("spread", [1.0, 2.0 ** -6])
def test_codes_and_scales_are_those_of_unlimited_precision(dtype, row, spread):
    """Every one of 10 million (4 million of them beside groups of zeros, whose scale is
    far from the row's): one that 32 bits cannot tell is worked out with more."""
    x, w = make(20000, dtype, 11, spread)
    x[::5, 128:256] = 0
    rows = torch.empty((20000, row), dtype=torch.uint8, device="cuda")
    H.norm_rows(x, rows, weight=w, eps=1e-5)
    y = M.norm(x[:, :512].double().cpu().numpy(), w.double().cpu().numpy(), float(np.float32(1e-5)))
    got, _ = M.values_of_rows(rows.cpu().numpy(), dtype)
    assert np.array_equal(got, exact_values(y, row))


def test_infinities_and_nan_of_the_weight_stay_in_their_groups():
    x, w = make(5000, "bf16", 12)
    x[:, 40] = torch.where(x[:, 40] == 0, 1, x[:, 40])
    w[40], w[200] = float("inf"), float("nan")
    finite = w.double().cpu().numpy()
    finite[[40, 200]] = 1.0
    y = M.norm(x[:, :512].double().cpu().numpy(), finite, float(np.float32(1e-6)))
    for row, group in ((M.ROW8, 128), (M.ROW4, 16)):
        rows = torch.empty((5000, row), dtype=torch.uint8, device="cuda")
        back = torch.empty((5000, 576), dtype=torch.bfloat16, device="cuda")
        H.norm_rows(x, rows, weight=w)
        H.gather_rows(rows, back)
        got, want = back[:, :512].double().cpu().numpy(), exact_values(y, row)
        of = np.arange(512) // group
        there = (of != 40 // group) & (of != 200 // group)
        assert np.array_equal(got[:, there], want[:, there])
        assert np.isnan(got[:, of == 200 // group]).all()
        most = float("inf") if row == M.ROW8 else 2688.0      # (448 * 2^120, beyond bf16; 6 * 448)
        assert (np.abs(got[:, 40]) == most).all()
        rest = (of == 40 // group) & (np.arange(512) != 40)
        assert (got[:, rest] == 0).all()


@pytest.mark.parametrize("row", ROWS)
def test_slots_that_are_none(row):
    """Negative, and not below the number of rows: nothing is written, nothing read."""
    x, w = make(9, "bf16", 3)
    slots = torch.tensor([-1, 4, -2 ** 31, 5, 6, 2 ** 31 - 1, 0, -7, 8], dtype=torch.int32, device="cuda")
    rows = torch.full((9, row), 0x5A, dtype=torch.uint8, device="cuda")
    H.norm_rows(x, rows[:6], slots=slots, weight=w)
    ok = torch.tensor([1, 3, 6], device="cuda")
    y = M.norm(x[:, :512].double().cpu().numpy(), w.double().cpu().numpy(), 1e-6)[[1, 3, 6]]
    check(y, x[ok, 512:], rows[[4, 5, 0]], "bf16", row)
    assert (rows[[1, 2, 3, 6, 7, 8]] == 0x5A).all()
    values = torch.full((9, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    H.gather_rows(rows[:6], values, slots=slots)
    assert (values[[0, 2, 4, 5, 7, 8]] == 7.0).all()
    assert torch.equal(values[ok, 512:], x[ok, 512:])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_without_a_norm_rows_are_stored_as_they_are(dtype):
    x, _ = make(300, dtype, 5)
    rows = torch.empty((300, M.ROW16), dtype=torch.uint8, device="cuda")
    H.norm_rows(x, rows)
    assert torch.equal(rows.view(TYPES[dtype]), x)
    four, packed = (torch.empty((300, M.ROW4), dtype=torch.uint8, device="cuda") for _ in range(2))
    x[::7] *= 0.001
    x[3, :16] = 0
    x[4, 17] = -0.0
    H.norm_rows(x, four)
    H.pack_rows(x, packed)
    assert torch.equal(four, packed)          # bit for bit
    eight = torch.empty((300, M.ROW8), dtype=torch.uint8, device="cuda")
    H.norm_rows(x, eight)
    y = x[:, :512].double().cpu().numpy()
    check(y, x[:, 512:], eight, dtype, M.ROW8)
    want = M.scale8(np.abs(y).reshape(300, 4, 128).max(2))
    assert np.array_equal(eight[:, 512:528].contiguous().view(torch.float32).double().cpu().numpy(), want)


def test_borders_of_the_8_bit_scale():
    """A group's largest magnitude at, next above and next below 448 of a power of two."""
    x = torch.zeros((6, 576), dtype=torch.float16, device="cuda")
    for i, top in enumerate((448.0, 448.25, 447.75, 0.4375, 7.0, 2.0 ** -24)):
        x[i, :512:128] = top
        x[i, 5] = -top
    rows = torch.empty((6, M.ROW8), dtype=torch.uint8, device="cuda")
    H.norm_rows(x, rows)
    scale = rows[:, 512:528].contiguous().view(torch.float32).cpu().numpy()
    assert (scale == np.array([1, 2, 1, 2.0 ** -10, 2.0 ** -6, 2.0 ** -32])[:, None]).all()
    check(x[:, :512].double().cpu().numpy(), x[:, 512:], rows, "f16", M.ROW8)


@pytest.mark.parametrize("row", ROWS)
def test_zeros_infinities_and_nan(row):
    x, w = make(8, "bf16", 1)
    x[0, :512] = 0
    x[1, 100] = float("nan")
    x[2, 300] = float("inf")
    x[3, :512] = float("inf")
    x[4, 520] = float("nan")                  # a rope value: stored as it is
    rows = torch.empty((8, row), dtype=torch.uint8, device="cuda")
    back = torch.empty((8, 576), dtype=torch.bfloat16, device="cuda")
    H.norm_rows(x, rows, weight=w)
    H.gather_rows(rows, back)
    assert (back[0, :512] == 0).all()
    assert torch.isnan(back[1, :512]).all()
    assert torch.isnan(back[2, 300]) and torch.isnan(back[3, :512]).all()
    assert torch.isfinite(back[4:, :512]).all() and torch.isnan(back[4, 520])
    assert torch.equal(back[5:, 512:], x[5:, 512:])
    # without a norm an infinity is one value's, or its group's
    H.norm_rows(x, rows)
    H.gather_rows(rows, back)
    if row == M.ROW8:
        assert back[2, 300] == float("inf") and (back[2, :256] != float("inf")).all()
        assert torch.isnan(back[1, :128]).all() and torch.isfinite(back[1, 128:512]).all()
    if row == M.ROW16:
        assert torch.equal(back[2], x[2])
    if row == M.ROW4:
        assert back[2, 300] == 2688.0          # clipped, as pack_rows does


@pytest.mark.parametrize("spread", [1e-18, 1e-4, 1e4, 1e15])
def test_sizes_far_from_one(spread):
    """The norm takes them out, down to where eps counts."""
    x, w = make(40, "bf16", 2, spread)
    for row in ROWS:
        rows = torch.empty((40, row), dtype=torch.uint8, device="cuda")
        H.norm_rows(x, rows, weight=w, eps=0.0)
        y = M.norm(x[:, :512].double().cpu().numpy(), w.double().cpu().numpy(), 0.0)
        if spread > 1e-10:       # (below, squares are below 32 bits' normal numbers)
            check(y, x[:, 512:], rows, "bf16", row)
        else:
            assert np.isfinite(M.values_of_rows(rows.cpu().numpy(), "bf16")[0]).all()


@pytest.mark.parametrize("row", ROWS)
@pytest.mark.parametrize("spread", [1e-15, 1e-18, 1e-19, 2e-20, 1e15])
def test_means_next_to_what_32_bits_hold(row, spread):
    """As many rows as have codes that take a second look: all of them numbers, and with
    squares that are normal numbers none far off."""
    x, w = make(3000, "bf16", 13, spread)
    rows = torch.empty((3000, row), dtype=torch.uint8, device="cuda")
    H.norm_rows(x, rows, weight=w, eps=0.0)
    assert np.isfinite(M.values_of_rows(rows.cpu().numpy(), "bf16")[0]).all()
    if spread in (1e-15, 1e15):
        check(M.norm(x[:, :512].double().cpu().numpy(), w.double().cpu().numpy(), 0.0), x[:, 512:], rows, "bf16", row)


@pytest.mark.parametrize("row", ROWS)
def test_a_mean_of_zero_without_eps(row):
    x, w = make(3, "bf16", 14)
    x[0, :512], x[1, :512] = 0, 1e-25
    rows = torch.empty((3, row), dtype=torch.uint8, device="cuda")
    back = torch.empty((3, 576), dtype=torch.bfloat16, device="cuda")
    H.norm_rows(x, rows, weight=w, eps=0.0)
    H.gather_rows(rows, back)
    assert torch.isnan(back[:2, :512]).all() and torch.isfinite(back[2]).all()
    assert torch.equal(back[:, 512:], x[:, 512:])


@pytest.mark.parametrize("row", ROWS)
def test_strides_streams_and_graphs(row):
    n = 50
    x, w = make(n, "bf16", 8)
    wide = torch.zeros((n, 640), dtype=torch.bfloat16, device="cuda")
    wide[:, :576] = x
    pool = torch.zeros((n, row + 48), dtype=torch.uint8, device="cuda")
    slots = torch.arange(n - 1, -1, -1, dtype=torch.int32, device="cuda")
    back = torch.zeros((n, 584), dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    H.norm_rows(wide[:, :576], pool[:, :row], slots=slots, weight=w, stream=side)
    H.gather_rows(pool[:, :row], back[:, :576], slots=slots, stream=side.cuda_stream)
    torch.cuda.synchronize()
    plain = torch.empty((n, row), dtype=torch.uint8, device="cuda")
    H.norm_rows(x, plain, weight=w)
    assert torch.equal(pool[:, :row].flip(0), plain)
    assert (pool[:, row:] == 0).all() and (back[:, 576:] == 0).all()
    graph = torch.cuda.CUDAGraph()
    plain.zero_()
    with torch.cuda.graph(graph):
        H.norm_rows(x, plain, weight=w)
    for k in range(3):
        x.copy_(x.roll(1, 0))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(pool[:, :row].flip(0).roll(k + 1, 0), plain)


def test_pinned_host_rows():
    """The rows of a step, straight into a handle's pinned pool."""
    hs = H.HiSparse(2, 1, H.ROW8_BYTES, 4, 8, host_to_device_ratio=2, host_capacity=[16, 16])
    x, w = make(16, "bf16", 4)
    host = torch.from_numpy(hs.host_rows(0, 1))
    H.norm_rows(x, host, weight=w)
    torch.cuda.synchronize()
    rows = torch.empty((16, M.ROW8), dtype=torch.uint8, device="cuda")
    H.norm_rows(x, rows, weight=w)
    assert np.array_equal(hs.host_rows(0, 1), rows.cpu().numpy())
    hs.close()


def test_gather_rounds_scales_that_are_no_powers_of_two():
    """One rounding, half a step of the type."""
    g = torch.Generator(device="cuda").manual_seed(0)
    rows = torch.zeros((200, M.ROW8), dtype=torch.uint8, device="cuda")
    codes = torch.randint(0, 256, (200, 512), generator=g, device="cuda", dtype=torch.uint8)
    rows[:, :512] = torch.where((codes & 0x7F) == 0x7F, 0, codes)
    scale = torch.exp(torch.randn((200, 4), generator=g, device="cuda"))
    rows[:, 512:528] = scale.view(torch.uint8)
    lat, _ = M.values_of_rows(rows.cpu().numpy(), "bf16")
    for dtype in TYPES:
        values = torch.empty((200, 576), dtype=TYPES[dtype], device="cuda")
        H.gather_rows(rows, values)
        # (the product with the scale, in 32 bits, is one more half step)
        tol = np.abs(lat) * (HALF[dtype] + 2.0 ** -24) + 2.0 ** -25
        assert (np.abs(values[:, :512].double().cpu().numpy() - lat) <= tol).all()


@pytest.mark.slow
def test_rows_past_two_gigabytes():
    """Offsets beyond 32 bits: the last rows of a pool of 4.3 GB."""
    count = (1 << 32) // 656 + 1000
    rows = torch.empty((count, M.ROW8), dtype=torch.uint8, device="cuda")
    x, w = make(6, "bf16", 6)
    slots = torch.tensor([count - 1, 0, count - 1000, (1 << 31) // 656, 77, count - 2], dtype=torch.int32, device="cuda")
    H.norm_rows(x, rows, slots=slots, weight=w)
    y = M.norm(x[:, :512].double().cpu().numpy(), w.double().cpu().numpy(), 1e-6)
    check(y, x[:, 512:], rows[slots.long()], "bf16", M.ROW8)
    back = torch.empty((6, 576), dtype=torch.bfloat16, device="cuda")
    H.gather_rows(rows, back, slots=slots)
    assert torch.equal(back[:, 512:], x[:, 512:])
