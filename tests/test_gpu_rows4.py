"""Packing to 4-bit rows and back, bit for bit against the definition in 64
bits (tests/rows4_model.py)."""

import numpy as np
import pytest
import torch

import rows4_model as M
from hierarchical_sparse_kv_request_gb300 import hisparse as H

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def make_values(n, dtype, seed):
    """Rows whose groups span many magnitudes, with zeros, signed zeros and
    values on the borders between two codes."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, 576)) * np.exp2(rng.integers(-9, 9, (n, 36)).repeat(16, axis=1))
    x[rng.random((n, 576)) < 0.05] = 0.0
    x[rng.random((n, 576)) < 0.02] = -0.0
    for i in range(0, n, 3):     # a group of borders: its largest value is 6 * scale
        s = M.E4M3[rng.integers(1, 100)]
        x[i, :16] = s * np.array([6, .25, -.25, .75, -.75, 1.25, 1.75, -1.75, 2.5, -2.5, 3.5, -3.5, 5, -5, 0, -0.0])
    return torch.from_numpy(x).to(TYPES[dtype]).cuda()


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n", [1, 2, 15, 17, 33, 1000, 5003])
def test_pack_unpack_match_the_definition(n, dtype):
    x = make_values(n, dtype, n)
    rows = torch.full((n, 416), 0xA5, dtype=torch.uint8, device="cuda")
    H.pack_rows(x, rows)
    got = rows.cpu().numpy()
    want = M.pack(bits(x), dtype)
    assert np.array_equal(got, want)
    back = torch.empty_like(x)
    H.unpack_rows(rows, back)
    lat, rope = M.unpack(want, dtype)
    assert np.array_equal(back.double().cpu().numpy(), np.concatenate([lat, rope], axis=1))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_every_code_and_scale_unpacks_exactly(dtype):
    rows = np.zeros((256, 416), dtype=np.uint8)
    rows[:, :256] = np.arange(256, dtype=np.uint8)          # every pair of codes
    rows[:, 256:288] = np.arange(256, dtype=np.uint8)[:, None]   # every scale byte, signs and NaN too
    rows[:, 256:288] &= 0x7F
    rows[:, 288:] = np.frombuffer(np.arange(64, dtype=np.float16).tobytes(), dtype=np.uint8)
    back = torch.empty((256, 576), dtype=TYPES[dtype], device="cuda")
    H.unpack_rows(torch.from_numpy(rows).cuda(), back)
    lat, rope = M.unpack(rows, dtype)
    np.testing.assert_array_equal(back.double().cpu().numpy(), np.concatenate([lat, rope], axis=1))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_infinities_clip_and_nan_stays_in_its_group(dtype):
    x = make_values(8, dtype, 3)
    x[1, 20], x[2, 40], x[3, 100] = float("inf"), float("-inf"), float("nan")
    x[4, :16] = 0
    x[5, :512] = torch.finfo(x.dtype).max
    x[6, :512] = torch.finfo(x.dtype).smallest_normal
    rows = torch.empty((8, 416), dtype=torch.uint8, device="cuda")
    H.pack_rows(x, rows)
    back = torch.empty_like(x)
    H.unpack_rows(rows, back)
    v = back.double().cpu().numpy()
    assert v[1, 20] == 6 * 448 and v[2, 40] == -6 * 448
    nan = np.isnan(v)
    assert nan[3, 96:112].all() and nan.sum() == 16
    assert (v[4, :16] == 0).all() and (v[5, :512] == 6 * 448).all() and (v[6, :512] == 0).all()
    ok = [0, 1, 2, 4, 5, 6, 7]
    assert np.array_equal(rows.cpu().numpy()[ok], M.pack(bits(x), dtype)[ok])


def test_strides_and_neighbours():
    """Rows and values inside wider buffers; bytes between them stay."""
    n = 77
    x = make_values(n, "bf16", 5)
    wide = torch.zeros((n, 640), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:584] = x
    rows = torch.full((n, 656), 0x5A, dtype=torch.uint8, device="cuda")
    H.pack_rows(wide[:, 8:584], rows[:, 16:432])
    got = rows.cpu().numpy()
    assert np.array_equal(got[:, 16:432], M.pack(bits(x), "bf16"))
    assert (got[:, :16] == 0x5A).all() and (got[:, 432:] == 0x5A).all()
    back = torch.full((n, 600), 7.0, dtype=torch.bfloat16, device="cuda")
    H.unpack_rows(rows[:, 16:432], back[:, 16:592])
    lat, rope = M.unpack(got[:, 16:432], "bf16")
    v = back.double().cpu().numpy()
    assert np.array_equal(v[:, 16:592], np.concatenate([lat, rope], axis=1))
    assert (v[:, :16] == 7).all() and (v[:, 592:] == 7).all()


def test_pinned_rows_another_stream_and_a_graph():
    x = make_values(40, "bf16", 9)
    want = M.pack(bits(x), "bf16")
    pinned = torch.zeros((40, 416), dtype=torch.uint8, pin_memory=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    H.pack_rows(x, pinned, stream=side)
    side.synchronize()
    assert np.array_equal(pinned.numpy(), want)
    rows = torch.zeros((40, 416), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        H.pack_rows(x, rows)
    x.copy_(make_values(40, "bf16", 10))
    g.replay()
    assert np.array_equal(rows.cpu().numpy(), M.pack(bits(x), "bf16"))


def test_offsets_past_32_bits():
    """Row i of a strided buffer more than 4 GB behind row 0."""
    big = torch.empty(5 << 30, dtype=torch.uint8, device="cuda")
    rows = torch.as_strided(big, (2, 416), ((4 << 30) + (1 << 20), 1))
    rows.zero_()
    x = make_values(2, "bf16", 1)
    H.pack_rows(x, rows)
    assert np.array_equal(rows.cpu().numpy(), M.pack(bits(x), "bf16"))
    back = torch.empty_like(x)
    H.unpack_rows(rows, back)
    lat, rope = M.unpack(rows.cpu().numpy(), "bf16")
    assert np.array_equal(back.double().cpu().numpy(), np.concatenate([lat, rope], axis=1))


def test_no_rows():
    H.pack_rows(torch.empty((0, 576), dtype=torch.bfloat16, device="cuda"),
                torch.empty((0, 416), dtype=torch.uint8, device="cuda"))
