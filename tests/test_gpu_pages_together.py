"""The resident pages' calls in a decode step, as they are used: pages for each
request's new tokens behind a shared prefix, the tokens' rows stored at their slots,
a swap-in that finds them resident, attention over what it names, and attention over
the prefix joined with it.  Compared with attention over all those rows in 64 bits;
tolerances as in test_gpu_attend_prefix.py, with attend()'s own rounding of its output
(its probabilities enter as f16) before the join."""

import numpy as np
import pytest
import torch

import pages_model as M
import rows4_model as M4
from hierarchical_sparse_kv_request_gb300 import hisparse as H

pytestmark = pytest.mark.gpu
HALF, U32 = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("captured", [False, True])
def test_a_decode_loop_behind_a_shared_prefix(captured):
    R, heads, k, D, bs, steps = 3, 40, 48, 96, 16, 5
    prefix_len, first = 200, [300, 260, 411]          # tokens shared, and of each request at first
    shared = -(-prefix_len // bs)                      # the prefix's last page is part full: requests begin behind it
    own = shared * bs
    cap, blocks, pages = 512, 40, 160
    rng = np.random.default_rng(0)
    g = torch.Generator(device="cuda").manual_seed(0)
    scale = 576 ** -0.5
    hs = H.HiSparse(R, 1, H.ROW4_BYTES, k, D, host_to_device_ratio=6, host_capacity=[cap] * R)
    kv = torch.randn((R, cap, 576), generator=g, device="cuda").to(torch.bfloat16)
    kv[:, :own] = kv[0, :own]                          # the prefix is the same for all
    weight = (1 + 0.1 * torch.randn(512, generator=g, device="cuda")).to(torch.bfloat16)
    pool = torch.zeros(((pages + shared) * bs, H.ROW4_BYTES), dtype=torch.uint8, device="cuda")
    ids = torch.from_numpy(rng.permutation(pages + shared).astype(np.int32)).cuda()
    prefix_table, free_list = ids[:shared].clone(), ids[shared:].clone()
    held = torch.zeros(R, dtype=torch.int32, device="cuda")
    tables = torch.full((R, blocks), -1, dtype=torch.int32, device="cuda")
    free_count = torch.tensor([pages], dtype=torch.int32, device="cuda")
    status = torch.zeros(R, dtype=torch.int32, device="cuda")

    # the prefix's rows, once, and all rows into the pinned pool
    at = torch.arange(own, device="cuda")
    prefix_slots = (prefix_table[at // bs] * bs + at % bs).to(torch.int32)
    H.norm_rows(kv[0, :own], pool, slots=prefix_slots, weight=weight)
    for r in range(R):
        H.norm_rows(kv[r], torch.from_numpy(hs.host_rows(0, r)), weight=weight)

    def place(lens, new, tokens):
        offsets = torch.empty(R + 1, dtype=torch.int32, device="cuda")
        slots, positions = (torch.empty(tokens, dtype=torch.int32, device="cuda") for _ in range(2))
        H.page_tables(lens, tables, held, free_list, free_count, bs, shared=prefix_table, new_tokens=new, offsets=offsets,
                      slots=slots, positions=positions, status=status)
        return offsets, slots, positions

    # admission: the prompts behind the prefix
    lens = torch.tensor(first, dtype=torch.int32, device="cuda")
    new = lens - own
    total = int(new.sum())
    offsets, slots, positions = place(lens, new, total + 9)
    assert (slots[total:] == -1).all() and (slots[:total] >= 0).all()
    packed = torch.cat([kv[r, own:first[r]] for r in range(R)] + [torch.zeros((9, 576), dtype=torch.bfloat16, device="cuda")])
    H.norm_rows(packed, pool, slots=slots, weight=weight)
    hs.prefill(lens)

    out_ids = torch.empty((R, k), dtype=torch.int32, device="cuda")
    out = torch.empty((R, heads, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((R, heads), device="cuda")
    plan = torch.empty((R, k, 2), dtype=torch.int32, device="cuda")
    misses = torch.empty(R, dtype=torch.int32, device="cuda")
    one = torch.ones(R, dtype=torch.int32, device="cuda")
    q = torch.empty((R, heads, 576), dtype=torch.bfloat16, device="cuda")
    topk = torch.empty((R, k), dtype=torch.int32, device="cuda")
    row = torch.empty((R, 576), dtype=torch.bfloat16, device="cuda")
    backup = torch.empty((1, R, H.ROW4_BYTES), dtype=torch.uint8, device="cuda")
    resident = torch.empty_like(tables)
    spaces = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in
              (H.attend_workspace_bytes(R, heads, k), H.attend_prefix_workspace_bytes(R, heads, own))]
    slot_buf, offset_buf = torch.empty(R, dtype=torch.int32, device="cuda"), torch.empty(R + 1, dtype=torch.int32, device="cuda")

    def step():
        # the step's token: a page if it needs one, its row there and to the host
        lens.add_(1)
        H.page_tables(lens, tables, held, free_list, free_count, bs, shared=prefix_table, new_tokens=one,
                      offsets=offset_buf, slots=slot_buf, status=status)
        H.norm_rows(row, pool, slots=slot_buf, weight=weight)
        H.norm_rows(row, backup[0], weight=weight)
        hs.backup(0, backup[0], lens - 1)
        # every other page counts as resident, so that all tiers are met
        resident.copy_(tables)
        resident[:, 1::2] = -1
        hs.swap_in_resident(0, topk, lens, resident, bs, out_ids, plan, misses)
        hs.attend(0, q, out_ids, out, scale, lse=lse, resident_rows=pool, workspace=spaces[0])
        H.attend_prefix(q, pool, prefix_table, bs, own, out, scale, lse=lse, part=out, part_lse=lse, status=status,
                        workspace=spaces[1])

    graph = None
    for s in range(steps):
        now = lens.cpu().numpy()
        q.copy_(2 * torch.randn((R, heads, 576), generator=g, device="cuda"))
        row.copy_(torch.stack([kv[r, int(now[r])] for r in range(R)]))
        chosen = [rng.permutation(np.arange(own, now[r] + 1))[:k] for r in range(R)]
        topk.copy_(torch.from_numpy(np.stack(chosen).astype(np.int32)))
        torch.cuda.synchronize()
        if captured and s == 1:
            keep = lens.clone()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            assert torch.equal(lens, keep)
        graph.replay() if graph is not None else step()
        torch.cuda.synchronize()
        assert (status == 0).all() and (hs.status() == 0).all()
        ids_now = out_ids.cpu().numpy()
        assert (ids_now >= 0).all() and (ids_now & H.RESIDENT_FLAG != 0).any() and (ids_now & H.RESIDENT_FLAG == 0).any()
        for r in range(R):
            tokens = np.concatenate([np.arange(own), chosen[r]])
            rows = hs.host_rows(0, r)[tokens]
            lat, rope = M4.unpack(np.ascontiguousarray(rows), "bf16")
            want, w_lse, sp = M.attend_prefix(q[r].double().cpu().numpy(), lat, rope, float(np.float32(scale)))
            ds = 580 * U32 * sp["dot"] + 16 * U32 * np.abs(w_lse)
            rel = np.expm1(2 * ds) + HALF + 1000 * U32
            # attend()'s output is rounded to bf16 before the join: HALF of at most the spread
            tol = HALF * np.abs(want) + (1 + HALF) * (rel[:, None] + HALF) * sp["abs"] + 2.0 ** -25 * (1 + np.abs(lat).sum(0))
            got = out[r].double().cpu().numpy()
            assert (np.abs(got - want) <= tol).all(), (s, r, np.abs(got - want).max())
            assert (np.abs(lse[r].double().cpu().numpy() - w_lse) <= ds + 2000 * U32).all()
    hs.close()


@pytest.mark.parametrize("new_tokens", [False, True])
def test_tables_changed_between_programmatic_swap_ins(new_tokens):
    """A swap-in that reads ahead of its wait, its handle's last launch having been on
    another layer: the resident tables that page_tables has written in between are those
    it finds."""
    R, k, D, bs, blocks, cap = 64, 64, 128, 16, 60, 1024
    rng = np.random.default_rng(5)
    hs = H.HiSparse(R, 2, H.ROW4_BYTES, k, D, host_to_device_ratio=8, host_capacity=[cap] * R)
    hs.set_programmatic_launch(True)
    lens = torch.full((R,), 800, dtype=torch.int32, device="cuda")
    hs.prefill(lens)
    tables = torch.full((R, blocks), -1, dtype=torch.int32, device="cuda")
    held = torch.zeros(R, dtype=torch.int32, device="cuda")
    pages = torch.from_numpy(rng.permutation(R * blocks).astype(np.int32)).cuda()
    count = torch.tensor([R * blocks], dtype=torch.int32, device="cuda")
    topk = torch.from_numpy(np.stack([rng.permutation(800)[:k] for _ in range(R)]).astype(np.int32)).cuda()
    outs = [torch.empty((R, k), dtype=torch.int32, device="cuda") for _ in range(40)]
    covered = [torch.full((R,), int(n), dtype=torch.int32, device="cuda") for n in rng.integers(1, 800, 40)]
    new = torch.ones(R, dtype=torch.int32, device="cuda")
    more = dict(new_tokens=new, offsets=torch.empty(R + 1, dtype=torch.int32, device="cuda"),
                slots=torch.empty(1 << 15, dtype=torch.int32, device="cuda")) if new_tokens else {}
    seen = []
    for n in range(40):
        H.page_tables(covered[n], tables, held, pages, count, bs, **more)
        seen.append(tables.clone() if n % 2 else None)      # (half of them with no other kernel in between)
        hs.swap_in_resident(n & 1, topk, lens, tables, bs, outs[n])
    torch.cuda.synchronize()
    assert (hs.status() == 0).all()
    t = topk.cpu().numpy()
    for n in range(40):
        ids, resident = outs[n].cpu().numpy(), t < -(-int(covered[n][0]) // bs) * bs
        assert np.array_equal((ids & H.RESIDENT_FLAG) != 0, resident), n
        if seen[n] is not None:
            page = np.take_along_axis(seen[n].cpu().numpy(), t // bs, 1)
            assert np.array_equal(ids[resident], (H.RESIDENT_FLAG | (page * bs + t % bs))[resident])
    hs.close()
