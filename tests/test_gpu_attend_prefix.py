"""Attention over a shared prefix against the definition in 64 bits, with tolerances
that count the roundings of the computation:

- a score is a sum of 576 products held in 32 bits: off by at most 580 half steps of
  fp32 (2^-24) of scale * sum |q||row|, and by a few of itself;
- a probability is that far off in its logarithm, and enters the product with the
  latent values in the model's type (half a step: 2^-8 bf16, 2^-11 f16);
- in f16, below 2^-14 of the running reference, which is at least 2^-8 of the largest,
  its step no longer shrinks with it: half a step is 2^-25 of the reference, at most
  2^-25 of the largest, for each row;
- the sums over rows, and over the parts of a head, are in 32 bits, one step a row; out
  is rounded once to its type (and 2^-25 for f16 below 2^-14)."""

import numpy as np
import pytest
import torch

import pages_model as M
from hierarchical_sparse_kv_request_gb300 import hisparse as H

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
U32 = 2.0 ** -24
ROWS = [M.ROW4, M.ROW8, M.ROW16]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def make_rows(n, dtype, row, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((n, 576), generator=g, device="cuda")
    x = (x * torch.exp(0.5 * torch.randn((n, 1), generator=g, device="cuda"))).to(TYPES[dtype])
    rows = torch.empty((n, row), dtype=torch.uint8, device="cuda")
    H.norm_rows(x, rows)
    return rows


def make_q(R, heads, dtype, seed, spread=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (spread * torch.randn((R, heads, 576), generator=g, device="cuda")).to(TYPES[dtype])


def make_part(R, heads, dtype, seed, lse=6.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    part = torch.randn((R, heads, 512), generator=g, device="cuda").to(TYPES[dtype])
    sums = lse + 2 * torch.randn((R, heads), generator=g, device="cuda")
    if R > 1:
        sums[R // 2] = -float("inf")
        part[R // 2] = float("nan")          # not looked at
    return part, sums


def named(rows, table, bs, length):
    """The rows that a prefix's tokens name, those that are there."""
    t = np.arange(length)
    page = table.cpu().numpy()[t // bs].astype(np.int64)
    at = page * bs + t % bs
    ok = (page >= 0) & (at < rows.shape[0])
    return rows[torch.from_numpy(at[ok]).cuda()].cpu().numpy()


def check(q, packed, out, lse, scale, dtype, part=None, part_lse=None, requests=None):
    R, heads, _ = q.shape
    lat, rope = M.values_of_rows(packed, dtype)
    n = max(packed.shape[0], 1) + 1
    for r in range(R) if requests is None else requests:
        p = None if part is None else part[r].double().cpu().numpy()
        pl = None if part is None else part_lse[r].double().cpu().numpy()
        want, w_lse, sp = M.attend_prefix(q[r].double().cpu().numpy(), lat, rope, scale, p, pl)
        o = out[r].double().cpu().numpy()
        ds = 580 * U32 * sp["dot"] + 16 * U32 * np.abs(np.where(np.isfinite(w_lse), w_lse, 0)) + 1e-30
        rel = np.expm1(2 * ds) + HALF[dtype] + (2 * n + 200) * U32
        tiny = 2.0 ** -25 * np.abs(lat).sum(0) * (dtype == "f16") if packed.shape[0] else 0.0
        tol = HALF[dtype] * np.abs(want) + (1 + HALF[dtype]) * (rel[:, None] * sp["abs"] + tiny) + 2.0 ** -25
        assert np.isfinite(o).all(), r
        bad = np.abs(o - want) > tol
        assert not bad.any(), (r, np.argwhere(bad)[:4], o[bad][:4], want[bad][:4])
        if lse is not None:
            l = lse[r].double().cpu().numpy()
            none = np.isneginf(w_lse)
            assert np.isneginf(l[none]).all()
            ltol = ds + (2 * n + 200) * U32 + 16 * U32 * np.abs(w_lse)
            off = np.abs(l[~none] - w_lse[~none])
            assert (off <= ltol[~none]).all(), (r, off.max())


def call(R, heads, n, row=M.ROW8, dtype="bf16", bs=16, seed=0, part=True, holes=0.0, scale=576 ** -0.5, spread=2.0,
         requests=None, extra=3):
    rng = np.random.default_rng(seed)
    used = -(-n // bs)
    rows = make_rows(max((used + extra) * bs, 1), dtype, row, seed)
    table = torch.from_numpy(rng.permutation(used + extra)[:used].astype(np.int32)).cuda()
    if holes:
        table = torch.where(torch.from_numpy(rng.random(used) < holes).cuda(), -1, table)
    q = make_q(R, heads, dtype, seed + 1, spread)
    p, pl = make_part(R, heads, dtype, seed + 2) if part else (None, None)
    out = torch.full((R, heads, 512), 9.0, dtype=TYPES[dtype], device="cuda")
    lse = torch.full((R, heads), 9.0, device="cuda")
    status = torch.zeros(R, dtype=torch.int32, device="cuda")
    H.attend_prefix(q, rows, table, bs, n, out, scale, lse=lse, part=p, part_lse=pl, status=status)
    torch.cuda.synchronize()
    assert (status == 0).all()
    check(q, named(rows, table, bs, n), out, lse, float(np.float32(scale)), dtype, p, pl, requests)
    return q, rows, table, out, lse, p, pl


@pytest.mark.parametrize("n", [1, 2, 31, 32, 63, 64, 65, 127, 128, 129, 191, 255, 256, 257, 1000])
@pytest.mark.parametrize("row", ROWS)
def test_lengths(n, row):
    call(3, 16, n, row, seed=n)


@pytest.mark.parametrize("R,heads", [(1, 1), (1, 63), (1, 64), (1, 65), (1, 127), (1, 128), (1, 129), (3, 43), (2, 100),
                                     (5, 128), (33, 4), (129, 1), (37, 40), (2, 1024)])
def test_heads(R, heads):
    call(R, heads, 300, M.ROW4, "f16" if heads % 2 else "bf16", seed=heads,
         requests=None if R * heads < 2000 else [0, 1, R // 2, R - 1])


@pytest.mark.parametrize("heads", [1, 2, 3, 31, 33, 34, 64, 65, 72, 96, 97, 130, 191, 193, 200])
@pytest.mark.parametrize("n", [100, 1500])
def test_the_last_heads_are_shared_out(heads, n):
    """Groups of heads that are not full, in one pair and in parts."""
    call(1, heads, n, M.ROW8, "bf16", seed=heads, part=heads % 2 == 0)


@pytest.mark.parametrize("n", [4256, 4257, 6272, 6273, 8448, 8449])
@pytest.mark.parametrize("row", ROWS)
def test_lengths_where_the_rows_come_in_another_way(n, row):
    call(2, 4, n, row, bs=64, seed=n, holes=0.1)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("row", ROWS)
@pytest.mark.parametrize("R,heads,n", [(4, 16, 2048), (37, 40, 5003), (200, 128, 130), (9, 128, 9000)])
def test_batches(R, heads, n, row, dtype):
    """One tile a pair and many, groups of heads in one pair, in two and in many."""
    call(R, heads, n, row, dtype, bs=64, seed=R, requests=sorted({0, 1, R // 2, R - 1}))


@pytest.mark.parametrize("bs", [1, 2, 7, 17, 64, 100, 128, 1000])
@pytest.mark.parametrize("holes", [0.0, 0.3, 0.95])
def test_pages_and_holes(bs, holes):
    call(3, 20, 777, M.ROW8, "f16", bs=bs, seed=bs, holes=holes)


def test_nothing_to_attend_to():
    """No tokens, and only holes: the part alone; without one, zeros."""
    for heads, n, holes in ((33, 0, 0.0), (33, 300, 1.0), (400, 0, 0.0), (400, 1000, 1.0)):
        for part in (True, False):
            q, rows, table, out, lse, p, pl = call(4, heads, n, seed=n, holes=holes, part=part)
            if part:
                keep = [0, 1, 3]                # (request 2's part has no weight)
                assert torch.equal(out[keep], p[keep])
                assert torch.allclose(lse[keep], pl[keep], rtol=4 * U32, atol=0)
                assert (out[2] == 0).all() and (lse[2] == -float("inf")).all()
            else:
                assert (out == 0).all() and (lse == -float("inf")).all()


def test_a_single_row():
    """The output is that row, exactly."""
    for row in ROWS:
        q, rows, table, out, lse, _, _ = call(2, 70, 1, row, seed=5, part=False)
        lat, _ = M.values_of_rows(named(rows, table, 16, 1), "bf16")
        assert np.array_equal(out.double().cpu().numpy(), np.broadcast_to(lat[0], (2, 70, 512)))


@pytest.mark.parametrize("spread", [0.0, 1e-6, 30.0, 300.0])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_flat_and_sharp_scores(spread, dtype):
    call(2, 40, 700, M.ROW4, dtype, seed=8, spread=spread)


@pytest.mark.parametrize("scale", [-576 ** -0.5, 0.0, 1e-30])
def test_scales(scale):
    call(3, 40, 500, M.ROW16, seed=3, scale=scale)


def test_a_nan_scale_gives_nan_where_a_token_is_named():
    q, rows, table, out, lse, p, pl = call(2, 20, 200, seed=1)
    H.attend_prefix(q, rows, table, 16, 200, out, float("nan"), lse=lse, part=p, part_lse=pl)
    assert torch.isnan(out).all() and torch.isnan(lse).all()
    H.attend_prefix(q, rows, torch.full_like(table, -1), 16, 200, out, float("nan"), lse=lse)
    assert (out == 0).all() and (lse == -float("inf")).all()


def test_scores_rise_from_tile_to_tile():
    """Each later row outweighs all earlier ones: the running reference moves with
    every tile, up to the last row, and back, in any order."""
    n = 700
    rng = np.random.default_rng(0)
    base = rng.standard_normal(576)
    x = torch.from_numpy(np.outer(np.linspace(0.02, 4.0, n), base)).to(torch.bfloat16).cuda()
    rows = torch.empty((n, M.ROW16), dtype=torch.uint8, device="cuda")
    H.norm_rows(x, rows)
    q = torch.from_numpy(np.stack([base * s for s in (1, 3, -1, -3, 0.1)] * 30)[None]).to(torch.bfloat16).cuda()
    for order in (np.arange(n), np.arange(n)[::-1].copy(), rng.permutation(n)):
        table = torch.from_numpy(order.astype(np.int32)).cuda()
        out = torch.empty((1, 150, 512), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((1, 150), device="cuda")
        H.attend_prefix(q, rows, table, 1, n, out, 0.2, lse=lse)
        check(q, named(rows, table, 1, n), out, lse, float(np.float32(0.2)), "bf16")


def test_rows_that_are_not_named_do_not_matter():
    """NaN in the other rows of the pool: pages that no entry names, and behind the
    last token in its page."""
    q, rows, table, out, lse, p, pl = call(3, 50, 333, M.ROW16, seed=2, holes=0.2)
    t = np.arange(333)
    page = table.cpu().numpy()[t // 16].astype(np.int64)
    used = torch.zeros(rows.shape[0], dtype=torch.bool, device="cuda")
    used[torch.from_numpy((page * 16 + t % 16)[page >= 0]).cuda()] = True
    rows[~used] = 0xFF
    again, sums = torch.empty_like(out), torch.empty_like(lse)
    H.attend_prefix(q, rows, table, 16, 333, again, 576 ** -0.5, lse=sums, part=p, part_lse=pl)
    assert torch.equal(again, out) and torch.equal(sums, lse)


def test_bad_pages_are_left_out_and_reported():
    q, rows, table, out, lse, p, pl = call(3, 20, 400, seed=4, extra=0)
    for bad in (-2, -2 ** 31, rows.shape[0] // 16, 2 ** 31 - 1):
        t2 = table.clone()
        t2[3] = bad
        status = torch.zeros(3, dtype=torch.int32, device="cuda")
        H.attend_prefix(q, rows, t2, 16, 400, out, 576 ** -0.5, lse=lse, part=p, part_lse=pl, status=status)
        assert (status == 1 << M.BAD_RESIDENT).all()
        hole = table.clone()
        hole[3] = -1
        check(q, named(rows, hole, 16, 400), out, lse, float(np.float32(576 ** -0.5)), "bf16", p, pl)
    # a page of which only the first rows are there
    status.zero_()
    H.attend_prefix(q, rows[:-5], table, 16, 400, out, 576 ** -0.5, lse=lse, part=p, part_lse=pl, status=status)
    assert (status == 1 << M.BAD_RESIDENT).all()
    check(q, named(rows[:-5], table, 16, 400), out, lse, float(np.float32(576 ** -0.5)), "bf16", p, pl)
    H.attend_prefix(q, rows, torch.full_like(table, -7), 16, 400, out, 576 ** -0.5)      # no status: none kept
    assert (out == 0).all()


@pytest.mark.parametrize("R,heads,n", [(3, 50, 100), (3, 50, 4000), (40, 128, 200)])
def test_in_place(R, heads, n):
    """part and part_lse as out and lse: what attend() left."""
    q, rows, table, out, lse, p, pl = call(R, heads, n, seed=9, requests=[0])
    H.attend_prefix(q, rows, table, 16, n, p, 576 ** -0.5, lse=pl, part=p, part_lse=pl)
    assert torch.equal(p, out) and torch.equal(pl, lse)


def test_strides():
    R, heads, n = 5, 30, 300
    q, rows, table, out, lse, p, pl = call(R, heads, n, M.ROW4, seed=6)
    wide_q = torch.zeros((heads, R, 640), dtype=torch.bfloat16, device="cuda")
    wide_q[:, :, :576] = q.transpose(0, 1)
    pool = torch.zeros((rows.shape[0], 480), dtype=torch.uint8, device="cuda")
    pool[:, :416] = rows
    wide_out = torch.full((R, 2 * heads, 520), 3.0, dtype=torch.bfloat16, device="cuda")
    wide_part = torch.zeros((heads, R, 512), dtype=torch.bfloat16, device="cuda")
    wide_part.copy_(p.transpose(0, 1))
    view = wide_out[:, ::2, :512]
    H.attend_prefix(wide_q.transpose(0, 1)[:, :, :576], pool[:, :416], table, 16, n, view, 576 ** -0.5, part=wide_part.transpose(0, 1),
                    part_lse=pl)
    assert torch.equal(view, out)
    assert (wide_out[:, 1::2] == 3.0).all() and (wide_out[:, :, 512:] == 3.0).all()


def test_a_request_of_its_own_or_in_a_batch():
    """Results do not depend on the other requests' values."""
    q, rows, table, out, lse, p, pl = call(6, 128, 1500, seed=7)
    q2, p2, pl2 = q.clone(), p.clone(), pl.clone()
    q2[0], q2[5], p2[0], pl2[5] = 50.0, float("nan"), 7.0, 80.0
    again, sums = torch.empty_like(out), torch.empty_like(lse)
    H.attend_prefix(q2, rows, table, 16, 1500, again, 576 ** -0.5, lse=sums, part=p2, part_lse=pl2)
    assert torch.equal(again[1:5], out[1:5]) and torch.equal(sums[1:5], lse[1:5])


def test_repeats_bit_for_bit():
    q, rows, table, out, lse, p, pl = call(30, 64, 3000, seed=11, requests=[0])
    for _ in range(5):
        again, sums = torch.empty_like(out), torch.empty_like(lse)
        H.attend_prefix(q, rows, table, 16, 3000, again, 576 ** -0.5, lse=sums, part=p, part_lse=pl)
        assert torch.equal(again, out) and torch.equal(sums, lse)


def test_two_streams_at_once():
    """Each with a workspace of its own."""
    a = call(20, 64, 2500, M.ROW4, seed=1, requests=[0])
    b = call(7, 128, 4000, M.ROW8, seed=2, requests=[0])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    torch.cuda.synchronize()
    for _ in range(4):
        for s, (q, rows, table, out, lse, p, pl), n in zip(streams, (a, b), (2500, 4000)):
            o, l = torch.empty_like(out), torch.empty_like(lse)
            H.attend_prefix(q, rows, table, 16, n, o, 576 ** -0.5, lse=l, part=p, part_lse=pl, stream=s)
            outs.append((o, l, out, lse))
    torch.cuda.synchronize()
    for o, l, out, lse in outs:
        assert torch.equal(o, out) and torch.equal(l, lse)


def test_captured_and_replayed():
    """Inputs changed between replays, one workspace in the graph; small and large."""
    for R, heads, n in ((3, 20, 150), (20, 100, 3000)):
        q, rows, table, out, lse, p, pl = call(R, heads, n, seed=12, requests=[0])
        space = torch.empty(H.attend_prefix_workspace_bytes(R, heads, n), dtype=torch.uint8, device="cuda")
        o, l = torch.empty_like(out), torch.empty_like(lse)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(2):      # (the second on the first's heels, in the same workspace)
                H.attend_prefix(q, rows, table, 16, n, o, 576 ** -0.5, lse=l, part=p, part_lse=pl, workspace=space)
        for k in range(3):
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, out) and torch.equal(l, lse)
            q.copy_(-q)
            H.attend_prefix(q, rows, table, 16, n, out, 576 ** -0.5, lse=lse, part=p, part_lse=pl)
            space.fill_(0xFF)


def test_the_workspace_may_hold_anything_before():
    q, rows, table, out, lse, p, pl = call(9, 70, 1000, seed=13, requests=[0])
    space = torch.full((H.attend_prefix_workspace_bytes(9, 70, 1000),), 0xFF, dtype=torch.uint8, device="cuda")
    o = torch.empty_like(out)
    H.attend_prefix(q, rows, table, 16, 1000, o, 576 ** -0.5, part=p, part_lse=pl, workspace=space)
    assert torch.equal(o, out)


def test_a_table_in_pinned_memory():
    q, rows, table, out, lse, p, pl = call(3, 20, 300, seed=14)
    o = torch.empty_like(out)
    H.attend_prefix(q, rows, table.cpu().pin_memory(), 16, 300, o, 576 ** -0.5, part=p, part_lse=pl)
    assert torch.equal(o, out)


@pytest.mark.slow
def test_the_longest_prefix():
    """2^20 tokens, rows beyond 32 bits of offset, the last pages first."""
    n, bs = 1 << 20, 1024
    count = 4 * n
    rows = torch.empty((count, M.ROW16), dtype=torch.uint8, device="cuda")
    some = make_rows(4096, "bf16", M.ROW16, 1)
    rows.view(count // 4096, 4096, M.ROW16).copy_(some)
    table = torch.arange(count // bs - 1, count // bs - 1 - n // bs, -1, dtype=torch.int32, device="cuda")
    q = make_q(1, 16, "bf16", 2)
    out = torch.empty((1, 16, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((1, 16), device="cuda")
    H.attend_prefix(q, rows, table, bs, n, out, 576 ** -0.5, lse=lse)
    # every row as often as every other: the same as once each, and ln(256) in the sum
    lat, rope = M.values_of_rows(some.cpu().numpy(), "bf16")
    want, w_lse, sp = M.attend_prefix(q[0].double().cpu().numpy(), lat, rope, float(np.float32(576 ** -0.5)))
    ds = 580 * U32 * sp["dot"]
    # sums: a tile of 128 rows at a time (8,192 tiles over 76 pairs), a step each
    tol = HALF["bf16"] * np.abs(want) + (np.expm1(2 * ds) + HALF["bf16"] + 20000 * U32)[:, None] * sp["abs"]
    assert (np.abs(out[0].double().cpu().numpy() - want) <= tol).all()
    assert (np.abs(lse[0].double().cpu().numpy() - w_lse - np.log(256.0)) <= ds + 20000 * U32).all()


def test_pages_past_two_gigabytes():
    """2.4 GB of rows, the prefix's pages the last of them."""
    n, bs, dtype = 300, 64, "bf16"
    count = 2 ** 31 // M.ROW16 + 40 * bs
    count -= count % bs
    rows = torch.zeros((count, M.ROW16), dtype=torch.uint8, device="cuda")
    last = make_rows(8 * bs, dtype, M.ROW16, 3)
    rows[-8 * bs:] = last
    table = torch.tensor([count // bs - 1 - k for k in range(5)], dtype=torch.int32, device="cuda")
    q = make_q(2, 20, dtype, 4)
    out, lse = torch.empty((2, 20, 512), dtype=TYPES[dtype], device="cuda"), torch.empty((2, 20), device="cuda")
    H.attend_prefix(q, rows, table, bs, n, out, 576 ** -0.5, lse=lse)
    near = torch.tensor([7 - k for k in range(5)], dtype=torch.int32, device="cuda")
    check(q, named(last, near, bs, n), out, lse, float(np.float32(576 ** -0.5)), dtype)
