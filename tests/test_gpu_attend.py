"""Attention over 4-bit rows against the definition in 64 bits, with
tolerances that count the roundings of the computation:

- a score is a sum of 576 products held in 32 bits: off by at most 580 half
  steps of fp32 (2^-24) of scale * sum |q||row|, and by a few of itself;
- a probability is that far off in its logarithm, and enters the product
  with the latent values as f16 (half a step: 2^-11);
- below 2^-14 of the largest, a probability's f16 step no longer shrinks
  with it: half a step is 2^-25 of the largest probability, for each row;
- the sums over rows and heads are in 32 bits; out is rounded once to its
  type (half a step: 2^-8 bf16, 2^-11 f16, and 2^-25 for f16 below 2^-14)."""

import numpy as np
import pytest
import torch

import rows4_model as M
from hierarchical_sparse_kv_request_gb300 import hisparse as H

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
U32 = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def make_rows(n, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((n, 576), generator=g, device="cuda")
    x = (x * torch.exp(0.5 * torch.randn((n, 1), generator=g, device="cuda"))).to(TYPES[dtype])
    rows = torch.empty((n, 416), dtype=torch.uint8, device="cuda")
    H.pack_rows(x, rows)
    return rows


def make_q(R, heads, dtype, seed, spread=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (spread * torch.randn((R, heads, 576), generator=g, device="cuda")).to(TYPES[dtype])


def check(q, rows, ids, out, scale, dtype, lse=None, weights=None, before=None, positions=None,
          resident=None, requests=None):
    """Compare a call's results with the definition."""
    qn, idn = q.double().cpu().numpy(), ids.cpu().numpy().astype(np.int64)
    o = out.double().cpu().numpy()
    R, heads, _ = qn.shape
    D = rows.shape[1]
    for r in range(R) if requests is None else requests:
        use = np.nonzero(idn[r] >= 0)[0]
        got = []
        for x in idn[r, use]:
            got.append(resident[int(x) & (M.FLAG - 1)] if x & M.FLAG else rows[r, int(x)])
        packed = torch.stack(got).cpu().numpy() if got else np.zeros((0, 416), dtype=np.uint8)
        lat, rope = M.unpack(packed, dtype)
        w_out, w_lse, w_p, sp = M.attend(qn[r], lat, rope, scale)
        n = max(use.size, 1)
        ds = 580 * U32 * sp["dot"] + 8 * U32 * np.abs(np.where(np.isfinite(w_lse), w_lse, 0)) + 1e-30
        rel = np.expm1(2 * ds) + 2.0 ** -11 + (2 * n + 16) * U32
        tiny = 2.0 ** -25 * np.abs(lat).sum(0) if use.size else 0.0
        tol = (HALF[dtype] * np.abs(w_out) + (1 + HALF[dtype]) * (rel[:, None] * sp["abs"] + tiny)
               + 2.0 ** -25)
        assert np.isfinite(o[r]).all(), r
        bad = np.abs(o[r] - w_out) > tol
        assert not bad.any(), (r, np.argwhere(bad)[:4], o[r][bad][:4], w_out[bad][:4])
        if lse is not None:
            l = lse[r].double().cpu().numpy()
            if use.size == 0:
                assert (l == -np.inf).all()
            else:
                ltol = ds + (2 * n + 16) * U32 + 8 * U32 * np.abs(w_lse)
                assert (np.abs(l - w_lse) <= ltol).all(), (r, np.abs(l - w_lse).max(), ltol.min())
        if weights is not None:
            got_w = weights[r].double().cpu().numpy()
            want = before[r].double().cpu().numpy().copy()
            pos = positions[r].cpu().numpy()[use]
            np.add.at(want, pos, w_p)
            wrel = np.expm1(2 * ds.max()) + (2 * n + heads + 16) * U32
            wtol = wrel * (want - before[r].double().cpu().numpy()) + 4 * U32 * np.abs(want)
            assert (np.abs(got_w - want) <= wtol).all(), (r, np.abs(got_w - want).max())


def call(R, heads, k, D, dtype="bf16", seed=0, pad=0.0, weights=False, resident=0, scale=576 ** -0.5,
         tokens=None, spread=2.0):
    rng = np.random.default_rng(seed)
    rows = make_rows(R * D, dtype, seed).view(R, D, 416)
    q = make_q(R, heads, dtype, seed + 1, spread)
    ids = np.stack([rng.permutation(D)[:k] for _ in range(R)]).astype(np.int32)
    res = None
    if resident:
        res = make_rows(resident, dtype, seed + 2)
        flag = rng.random((R, k)) < 0.5
        ids = np.where(flag, rng.integers(0, resident, (R, k)) | M.FLAG, ids).astype(np.int32)
    tokens = tokens or 2 * D
    pos = np.stack([rng.permutation(tokens)[:k] for _ in range(R)]).astype(np.int32)
    if pad:
        hole = rng.random((R, k)) < pad
        if R > 1:
            hole[R // 2] = True
        ids[hole] = -1
        pos[hole] = -1
    ids, pos = torch.from_numpy(ids).cuda(), torch.from_numpy(pos).cuda()
    out = torch.full((R, heads, 512), 9.0, dtype=TYPES[dtype], device="cuda")
    lse = torch.full((R, heads), 9.0, device="cuda")
    acc = before = None
    if weights:
        acc = torch.rand((R, tokens), device="cuda")
        before = acc.clone()
    status = torch.zeros(R, dtype=torch.int32, device="cuda")
    H.attend(q, rows, ids, out, scale, lse=lse, positions=pos if weights else None, weights=acc,
             resident_rows=res, status=status)
    torch.cuda.synchronize()
    assert (status == 0).all()
    check(q, rows, ids, out, scale, dtype, lse, acc, before, pos, res)
    return q, rows, ids, out, lse


@pytest.mark.parametrize("k", [1, 2, 3, 15, 16, 31, 63, 64, 65, 127, 128, 129, 200, 1001])
def test_lengths(k):
    call(3, 16, k, k + 3, seed=k, weights=True)


@pytest.mark.parametrize("heads", [1, 2, 7, 8, 15, 16, 17, 31, 32, 33, 40, 63, 64, 65, 100, 127, 128, 129, 200])
def test_heads(heads):
    call(2, heads, 150, 160, "f16" if heads % 2 else "bf16", seed=heads, weights=True)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("R,heads,k,D", [(1, 16, 2048, 2100), (5, 128, 700, 900), (40, 16, 300, 310),
                                         (170, 8, 65, 70), (2, 128, 8192, 8192), (1, 1, 8192, 8200)])
def test_batches(R, heads, k, D, dtype):
    call(R, heads, k, D, dtype, seed=R, weights=R < 10)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("pad", [0.05, 0.5, 0.97])
@pytest.mark.parametrize("heads", [16, 70])
def test_padding_empty_requests_and_resident_rows(pad, heads, dtype):
    call(5, heads, 333, 400, dtype, seed=int(pad * 100), pad=pad, weights=True, resident=50)


def test_a_single_row_of_a_single_slot():
    q, rows, ids, out, lse = call(1, 3, 1, 1, seed=4, weights=True)
    lat, _ = M.unpack(rows[0].cpu().numpy(), "bf16")
    # one row: the output is that row, exactly
    assert np.array_equal(out[0].double().cpu().numpy(), np.broadcast_to(lat[0], (3, 512)))


@pytest.mark.parametrize("spread", [0.0, 1e-6, 30.0, 300.0])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_flat_and_sharp_scores(spread, dtype):
    """From equal scores to a single row taking all the weight."""
    call(2, 20, 300, 310, dtype, seed=8, spread=spread, weights=True)


@pytest.mark.parametrize("dtype,q_scale", [("bf16", 1e30), ("bf16", 1e-30), ("f16", 2000.0), ("f16", 1e-4)])
def test_queries_far_from_one(dtype, q_scale):
    """The softmax's scale brings scores back to ordinary size."""
    R, heads, k, D = 2, 9, 130, 140
    rows = make_rows(R * D, dtype, 3).view(R, D, 416)
    q = (make_q(R, heads, dtype, 4, 1.0).float() * q_scale).to(TYPES[dtype])
    ids = torch.stack([torch.randperm(D)[:k] for _ in range(R)]).int().cuda()
    out = torch.empty((R, heads, 512), dtype=TYPES[dtype], device="cuda")
    lse = torch.empty((R, heads), device="cuda")
    H.attend(q, rows, ids, out, 0.04 / q_scale, lse=lse)
    check(q, rows, ids, out, float(np.float32(0.04 / q_scale)), dtype, lse)


def test_scores_rise_from_tile_to_tile():
    """Each later row outweighs all earlier ones: the running maximum moves
    with every tile, up to the last row."""
    R, heads, k = 1, 5, 700
    rng = np.random.default_rng(0)
    base = rng.standard_normal(576)
    x = np.outer(np.linspace(0.02, 4.0, k), base)
    rows = torch.empty((k, 416), dtype=torch.uint8, device="cuda")
    H.pack_rows(torch.from_numpy(x).to(torch.bfloat16).cuda(), rows)
    q = torch.from_numpy(np.stack([base * s for s in (1, 3, -1, -3, 0.1)])[None]).to(torch.bfloat16).cuda()
    for order in (np.arange(k), np.arange(k)[::-1].copy(), rng.permutation(k)):
        ids = torch.from_numpy(order.astype(np.int32))[None].cuda()
        out = torch.empty((R, heads, 512), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((R, heads), device="cuda")
        acc = torch.zeros((R, k), device="cuda")
        pos = torch.arange(k, dtype=torch.int32, device="cuda")[None]
        H.attend(q, rows[None], ids, out, 0.2, lse=lse, weights=acc, positions=pos)
        check(q, rows[None], ids, out, float(np.float32(0.2)), "bf16", lse, acc, torch.zeros_like(acc), pos)


def test_rows_that_are_not_named_do_not_matter():
    """NaN rows in the cache, outside the named slots and in holes."""
    q, rows, ids, out, lse = call(3, 20, 100, 260, seed=2, pad=0.3)
    named = torch.zeros((3, 260), dtype=torch.bool, device="cuda")
    for r in range(3):
        v = ids[r][ids[r] >= 0].long()
        named[r, v] = True
    rows2 = torch.where(named.unsqueeze(2), rows, 0xFF)
    out2, lse2 = torch.empty_like(out), torch.empty_like(lse)
    H.attend(q, rows2, ids, out2, 576 ** -0.5, lse=lse2)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_nan_and_infinite_queries_stay_in_their_head():
    q, rows, ids, out, lse = call(2, 70, 90, 100, seed=6)
    q2 = q.clone()
    q2[0, 3, 5] = float("nan")
    q2[0, 64, 570] = float("nan")
    q2[1, 9, 17] = float("inf")
    out2, lse2 = torch.empty_like(out), torch.empty_like(lse)
    H.attend(q2, rows, ids, out2, 576 ** -0.5, lse=lse2)
    hit = torch.zeros((2, 70), dtype=torch.bool, device="cuda")
    hit[0, 3] = hit[0, 64] = hit[1, 9] = True
    assert torch.isnan(out2[hit]).all()
    assert torch.equal(out2[~hit], out[~hit]) and torch.equal(lse2[~hit], lse[~hit])


def test_a_nan_row_reaches_every_head_of_its_request_only():
    q, rows, ids, out, lse = call(2, 10, 70, 80, seed=7)
    rows2 = rows.clone()
    rows2[1, int(ids[1, 5]), 256:288] = 0x7F
    out2 = torch.empty_like(out)
    H.attend(q, rows2, ids, out2, 576 ** -0.5)
    assert torch.isnan(out2[1]).all() and torch.equal(out2[0], out[0])


@pytest.mark.parametrize("heads", [12, 66])
def test_strided_tensors(heads):
    """q, out, rows, ids, positions and weights inside wider buffers."""
    R, k, D, tokens = 3, 77, 90, 200
    dtype = "bf16"
    rows = torch.zeros((R, D + 2, 448), dtype=torch.uint8, device="cuda")
    rows[:, :D, :416] = make_rows(R * D, dtype, 1).view(R, D, 416)
    rows_v = rows[:, :D, :416]
    q = torch.zeros((R, heads + 3, 600), dtype=TYPES[dtype], device="cuda")
    q[:, 1:heads + 1, 8:584] = make_q(R, heads, dtype, 2)
    q_v = q[:, 1:heads + 1, 8:584]
    out = torch.full((heads + 1, R, 528), 5.0, dtype=TYPES[dtype], device="cuda")
    out_v = out[:heads, :, 8:520].transpose(0, 1)
    wide = torch.full((R, k + 5), 7, dtype=torch.int32, device="cuda")
    wide[:, :k] = torch.stack([torch.randperm(D)[:k] for _ in range(R)]).int().cuda()
    pos = torch.full((R, k + 9), 7, dtype=torch.int32, device="cuda")
    pos[:, :k] = torch.stack([torch.randperm(tokens)[:k] for _ in range(R)]).int().cuda()
    acc = torch.rand((R, tokens + 30), device="cuda")
    before = acc.clone()
    lse = torch.empty((R, heads), device="cuda")
    H.attend(q_v, rows_v, wide[:, :k], out_v, 0.05, lse=lse, weights=acc[:, :tokens], positions=pos[:, :k])
    check(q_v, rows_v, wide[:, :k], out_v, float(np.float32(0.05)), dtype, lse, acc[:, :tokens],
          before[:, :tokens], pos[:, :k])
    assert torch.equal(acc[:, tokens:], before[:, tokens:])
    assert (out[heads] == 5).all() and (out[:, :, :8] == 5).all() and (out[:, :, 520:] == 5).all()


def test_offsets_past_32_bits():
    """Requests more than 4 GB apart, and slots of one request likewise."""
    dtype, k, D = "bf16", 70, 80
    step = (4 << 30) + (1 << 20)
    big = torch.empty(2 * step, dtype=torch.uint8, device="cuda")
    rows = torch.as_strided(big, (2, D, 416), (step, 416, 1))
    rows.copy_(make_rows(2 * D, dtype, 1).view(2, D, 416))
    q = make_q(2, 4, dtype, 2)
    ids = torch.stack([torch.randperm(D)[:k] for _ in range(2)]).int().cuda()
    out = torch.empty((2, 4, 512), dtype=TYPES[dtype], device="cuda")
    H.attend(q, rows, ids, out, 0.05)
    check(q, rows, ids, out, float(np.float32(0.05)), dtype)
    far = torch.as_strided(big, (1, 3, 416), (0, step - 4096, 1))
    far.copy_(make_rows(3, dtype, 3).view(1, 3, 416))
    ids = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    out = torch.empty((1, 4, 512), dtype=TYPES[dtype], device="cuda")
    H.attend(q[:1], far, ids, out, 0.05)
    check(q[:1], far, ids, out, float(np.float32(0.05)), dtype)


def test_bad_ids_are_skipped_and_recorded():
    """A bad id counts as -1; each kind sets its bit; other requests' do not."""
    R, heads, k, D, tokens = 5, 6, 80, 100, 150
    rows = make_rows(R * D, "bf16", 1).view(R, D, 416)
    res = make_rows(7, "bf16", 2)
    q = make_q(R, heads, "bf16", 3)
    good = torch.stack([torch.randperm(D)[:k] for _ in range(R)]).int().cuda()
    pos = torch.stack([torch.randperm(tokens)[:k] for _ in range(R)]).int().cuda()
    ids, clean = good.clone(), good.clone()
    for r, i, v in [(1, 3, D), (1, 70, -2), (2, 0, M.FLAG | 7), (3, 79, -(1 << 31))]:
        ids[r, i], clean[r, i] = v, -1
    pos2 = pos.clone()
    pos2[4, 10], pos2[4, 11] = tokens, -5
    acc, ref = torch.zeros((R, tokens), device="cuda"), torch.zeros((R, tokens), device="cuda")
    out, want = (torch.empty((R, heads, 512), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    status = torch.zeros(R, dtype=torch.int32, device="cuda")
    H.attend(q, rows, ids, out, 0.05, weights=acc, positions=pos2, resident_rows=res, status=status)
    H.attend(q, rows, clean, want, 0.05, weights=ref, positions=pos)
    assert torch.equal(out, want)
    for i in (10, 11):      # their weight is dropped
        ref[4, int(pos[4, i])] = 0
    assert torch.equal(acc, ref)
    bit = H.STATUS_BIT
    assert status.tolist() == [0, bit(H.STATUS_BAD_INDEX), bit(H.STATUS_BAD_RESIDENT),
                               bit(H.STATUS_BAD_INDEX), bit(H.STATUS_BAD_POSITION)]


@pytest.mark.parametrize("R,heads,k", [(160, 5, 130), (155, 40, 129), (80, 70, 200), (310, 3, 130)])
def test_more_requests_than_a_wave(R, heads, k):
    """The requests behind the last whole wave go in a launch of their own, with
    their own places in every array."""
    call(R, heads, k, k + 9, "f16" if R % 2 else "bf16", seed=R, pad=0.2, weights=True, resident=20)


def test_status_and_weights_of_requests_behind_a_wave():
    R, heads, k, D, tokens = 160, 5, 130, 140, 300
    rows = make_rows(R * D, "bf16", 3).view(R, D, 416)
    q = make_q(R, heads, "bf16", 4)
    ids = torch.stack([torch.randperm(D)[:k] for _ in range(R)]).int().cuda()
    pos = torch.stack([torch.randperm(tokens)[:k] for _ in range(R)]).int().cuda()
    ids[3, 5], ids[157, 7] = D, -9
    pos[4, 0], pos[159, 1] = tokens, -2
    out = torch.empty((R, heads, 512), dtype=torch.bfloat16, device="cuda")
    acc = torch.zeros((R, tokens), device="cuda")
    status = torch.zeros(R, dtype=torch.int32, device="cuda")
    H.attend(q, rows, ids, out, 0.05, weights=acc, positions=pos, status=status)
    bit, want = H.STATUS_BIT, [0] * R
    want[3] = want[157] = bit(H.STATUS_BAD_INDEX)
    want[4] = want[159] = bit(H.STATUS_BAD_POSITION)
    assert status.tolist() == want
    for r in (0, 3, 151, 152, 157, 158):      # the same request by itself
        alone, mine = torch.empty((1, heads, 512), dtype=torch.bfloat16, device="cuda"), torch.zeros((1, tokens), device="cuda")
        H.attend(q[r:r + 1], rows[r:r + 1], ids[r:r + 1], alone, 0.05, weights=mine, positions=pos[r:r + 1])
        torch.testing.assert_close(alone[0], out[r], rtol=2.0 ** -7, atol=1e-3)
        torch.testing.assert_close(mine[0], acc[r], rtol=1e-4, atol=1e-6)


def test_repeated_rows_count_twice_and_results_repeat():
    R, heads, k, D = 2, 16, 500, 600
    rows = make_rows(R * D, "bf16", 1).view(R, D, 416)
    q = make_q(R, heads, "bf16", 2)
    ids = torch.randint(0, 40, (R, k), dtype=torch.int32, device="cuda")
    out = torch.empty((R, heads, 512), dtype=torch.bfloat16, device="cuda")
    H.attend(q, rows, ids, out, 0.05)
    check(q, rows, ids, out, float(np.float32(0.05)), "bf16")
    a = call(9, 24, 700, 800, seed=5, weights=True)
    b = call(9, 24, 700, 800, seed=5, weights=True)
    assert torch.equal(a[3], b[3]) and torch.equal(a[4], b[4])


def test_another_stream_a_graph_and_a_reused_workspace():
    R, heads, k, D = 4, 64, 400, 500
    rows = make_rows(R * D, "bf16", 1).view(R, D, 416)
    ids = torch.stack([torch.randperm(D)[:k] for _ in range(R)]).int().cuda()
    pos = ids.clone()
    q = make_q(R, heads, "bf16", 2)
    ws = torch.full((H.attend_workspace_bytes(R, heads, k, True),), 0xFF, dtype=torch.uint8, device="cuda")
    out, acc = torch.empty((R, heads, 512), dtype=torch.bfloat16, device="cuda"), torch.zeros((R, D), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    H.attend(q, rows, ids, out, 0.05, weights=acc, positions=pos, workspace=ws, stream=side)
    side.synchronize()
    check(q, rows, ids, out, float(np.float32(0.05)), "bf16", None, acc, torch.zeros_like(acc), pos)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        H.attend(q, rows, ids, out, 0.05, weights=acc, positions=pos, workspace=ws)
    for seed in (7, 8):
        q.copy_(make_q(R, heads, "bf16", seed))
        acc.zero_()
        g.replay()
        torch.cuda.synchronize()
        check(q, rows, ids, out, float(np.float32(0.05)), "bf16", None, acc, torch.zeros_like(acc), pos)


def test_pinned_ids():
    R, heads, k, D = 2, 8, 100, 128
    rows = make_rows(R * D, "bf16", 1).view(R, D, 416)
    q = make_q(R, heads, "bf16", 2)
    ids = torch.stack([torch.randperm(D)[:k] for _ in range(R)]).int().pin_memory()
    out = torch.empty((R, heads, 512), dtype=torch.bfloat16, device="cuda")
    H.attend(q, rows, ids, out, 0.05)
    torch.cuda.synchronize()
    check(q, rows, ids, out, float(np.float32(0.05)), "bf16")


def test_the_workspace_must_be_large_enough():
    R, heads, k, D = 2, 8, 100, 128
    rows = make_rows(R * D, "bf16", 1).view(R, D, 416)
    q = make_q(R, heads, "bf16", 2)
    ids = torch.zeros((R, k), dtype=torch.int32, device="cuda")
    out = torch.empty((R, heads, 512), dtype=torch.bfloat16, device="cuda")
    n = H.attend_workspace_bytes(R, heads, k, True)
    with pytest.raises(H.HiSparseError) as e:
        H.attend(q, rows, ids, out, 0.05, weights=torch.zeros((R, 10), device="cuda"), positions=ids,
                 workspace=torch.empty(n - 16, dtype=torch.uint8, device="cuda"))
    assert e.value.code == H.ERR_CAPACITY
