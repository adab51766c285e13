"""Eviction by accumulated weight: the chosen slots equal the definition's
(tests/rows4_model.py), and freeing them leaves a hot state that the resolver
goes on from exactly as from one written by hand."""

import numpy as np
import pytest
import torch

import rows4_model as M
from hierarchical_sparse_kv_request_gb300 import hisparse as H
from hierarchical_sparse_kv_request_gb300 import workload as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def select(w, tok, seq, n, recent, want=None):
    R = tok.shape[0]
    slots = torch.full((R, n), 77, dtype=torch.int32, device="cuda")
    counts = torch.full((R,), 77, dtype=torch.int32, device="cuda")
    H.evict_select(torch.from_numpy(w).cuda(), torch.from_numpy(tok).cuda(),
                   torch.from_numpy(seq).cuda(), slots, counts, recent,
                   None if want is None else torch.from_numpy(want).cuda())
    return slots.cpu().numpy(), counts.cpu().numpy()


def check(w, tok, seq, n, recent, want=None):
    slots, counts = select(w, tok, seq, n, recent, want)
    for r in range(tok.shape[0]):
        m = n if want is None else min(max(int(want[r]), 0), n)
        at = M.evict(w[r], tok[r], int(seq[r]), recent, m)
        assert counts[r] == at.size, r
        assert np.array_equal(slots[r, :at.size], at), r
        assert (slots[r, at.size:] == -1).all(), r


def state(R, D, tokens, seed, kind="random"):
    rng = np.random.default_rng(seed)
    tok = np.stack([rng.permutation(tokens)[:D] for _ in range(R)]).astype(np.int32)
    tok[rng.random((R, D)) < 0.05] = -1
    seq = rng.integers(D + 1, tokens + 1, R).astype(np.int32)
    tok = np.where(tok < seq[:, None], tok, -1).astype(np.int32)
    w = (rng.random((R, tokens)) ** 6 * 40).astype(np.float32)
    if kind == "ties":
        w = rng.integers(0, 3, (R, tokens)).astype(np.float32)
    elif kind == "equal":
        w[:] = 0.25
    elif kind == "zero":
        w[:] = 0
        w[:, ::2] = -0.0
    elif kind == "odd":
        w = rng.standard_normal((R, tokens)).astype(np.float32)
        w[rng.random((R, tokens)) < 0.1] = np.nan
        w[rng.random((R, tokens)) < 0.1] = np.inf
        w[rng.random((R, tokens)) < 0.1] = -np.inf
        w[rng.random((R, tokens)) < 0.1] = np.float32(1e-45)
    elif kind == "last digit":     # keys that differ in the lowest bits only
        w = (np.uint32(0x3F800000) + rng.integers(0, 700, (R, tokens)).astype(np.uint32)).view(np.float32)
    return w, tok, seq


@pytest.mark.parametrize("kind", ["random", "ties", "equal", "zero", "odd", "last digit"])
@pytest.mark.parametrize("D", [1, 2, 31, 33, 512, 1023, 1024, 1025, 2050, 6144])
def test_select(D, kind):
    w, tok, seq = state(3, D, 2 * D + 50, D, kind)
    for n in sorted({1, max(1, D // 5), max(1, D - 1), D}):
        check(w, tok, seq, n, D // 10)


@pytest.mark.parametrize("D", [9000, 32768])
def test_select_large(D):
    w, tok, seq = state(2, D, 3 * D, D, "random")
    check(w, tok, seq, D // 4, 100)
    w, tok, seq = state(2, D, 3 * D, D, "ties")
    check(w, tok, seq, D // 2, 100)


@pytest.mark.parametrize("kind", ["random", "ties", "equal", "zero", "odd", "last digit"])
@pytest.mark.parametrize("D", [8193, 16384, 16385, 24000])
def test_select_where_two_ctas_share_a_request(D, kind):
    w, tok, seq = state(2, D, 2 * D + 50, D, kind)
    seq[1] = D if kind == "odd" else seq[1]      # nothing to choose there
    for n in (1, D // 5, D):
        check(w, tok, seq, n, D // 10)


def test_select_large_in_more_requests_than_pairs():
    w, tok, seq = state(100, 9000, 20000, 3, "ties")
    check(w, tok, seq, 2000, 50)


def test_evict_frees_in_a_large_buffer():
    test_evict_frees_and_the_resolver_goes_on(9000, 700, [20000, 9500], 0)


def test_short_requests_recent_tokens_and_want():
    D, tokens = 300, 900
    w, tok, seq = state(8, D, tokens, 1)
    seq[0], seq[1], seq[2] = D, D - 5, 0          # short: none
    seq[3] = D + 1
    seq[4] = -7
    tok = np.where(tok < np.maximum(seq, 0)[:, None], tok, -1).astype(np.int32)
    for recent in (0, 1, 250, 899, 5000, 2 ** 31 - 1):
        check(w, tok, seq, 50, recent)
    check(w, tok, seq, 50, 10, np.array([50, 0, 3, -4, 9, 1, 60, 50], dtype=np.int32))
    # no accumulator for the later tokens: they are kept
    check(np.ascontiguousarray(w[:, :200]), tok, seq, 50, 10)
    check(np.ascontiguousarray(w[:, :0]), tok, seq, 50, 10)


def test_select_in_a_graph_on_strided_weights():
    D, tokens, R, n = 400, 1000, 4, 60
    w, tok, seq = state(R, D, tokens, 3)
    wide = torch.zeros((R, tokens + 7), device="cuda")
    wide[:, :tokens] = torch.from_numpy(w).cuda()
    slots = torch.empty((R, n), dtype=torch.int32, device="cuda")
    counts = torch.empty((R,), dtype=torch.int32, device="cuda")
    tok_d, seq_d = torch.from_numpy(tok).cuda(), torch.from_numpy(seq).cuda()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        H.evict_select(wide[:, :tokens], tok_d, seq_d, slots, counts, 5)
    g.replay()
    for r in range(R):
        at = M.evict(w[r], tok[r], int(seq[r]), 5, n)
        assert np.array_equal(slots[r, :at.size].cpu().numpy(), at)


# -- freeing in a handle's hot state ---------------------------------------------

def handle(w):
    g = H.HiSparse.for_workload(w)
    for l in range(w.num_layers):
        for r in range(w.num_requests):
            W.fill_host_rows(w, l, r, g.host_rows(l, r), int(w.seq_lens0[r]))
    g.prefill(torch.from_numpy(w.seq_lens0).cuda())
    return g


def freed_state(before, cap_off, chosen):
    """The state after freeing chosen[r] of `before` (read_state's arrays)."""
    s2t, lu, t2s, _, ticks = [x.copy() for x in before]
    R, D = s2t.shape
    lru = np.empty((R, D), dtype=np.int32)
    for r in range(R):
        for s in chosen[r]:
            t2s[cap_off[r] + s2t[r, s]] = -1
            s2t[r, s] = -1
            lu[r, s] = 0
        lru[r] = np.lexsort((np.arange(D), lu[r]))
    return s2t, lu, t2s, lru, ticks


@pytest.mark.parametrize("protect", [0, 1, 2])
@pytest.mark.parametrize("D,k,lens", [(64, 24, [300, 64, 517, 70]), (1500, 700, [4000, 1400, 9000]),
                                      (2048, 512, [2049, 6000])])
def test_evict_frees_and_the_resolver_goes_on(D, k, lens, protect):
    R = len(lens)
    w = W.custom(R, k, D, lens, row_bytes=32, layers=2, anchor_of_layer=[-1, 0], seed=D)
    a, b = handle(w), handle(w)
    a.set_protected_calls(protect)
    b.set_protected_calls(protect)
    off = np.concatenate([[0], np.cumsum(a.cap)])[:-1]
    seq = torch.from_numpy(w.seq_lens0).cuda()
    rng = np.random.default_rng(D)
    out_a, out_b = (torch.empty((R, k), dtype=torch.int32, device="cuda") for _ in range(2))
    plan_a, plan_b = (torch.zeros((R, k, 2), dtype=torch.int32, device="cuda") for _ in range(2))
    cnt_a, cnt_b = (torch.empty(R, dtype=torch.int32, device="cuda") for _ in range(2))
    tokens = int(max(lens))
    for step in range(5):
        topk = torch.from_numpy(np.stack([rng.permutation(s)[:k] for s in lens]).astype(np.int32)).cuda()
        a.swap_in(0, topk, seq, out_a, plan_a, cnt_a)
        b.swap_in(0, topk, seq, out_b, plan_b, cnt_b)
        torch.cuda.synchronize()
        assert torch.equal(out_a, out_b) and torch.equal(cnt_a, cnt_b), step
        for r in range(R):
            assert torch.equal(plan_a[r, :int(cnt_a[r])], plan_b[r, :int(cnt_b[r])]), step
        for x, y in zip(a.read_state(0), b.read_state(0)):
            assert np.array_equal(x, y), step
        before = a.read_state(0)
        wt = (rng.random((R, tokens)) ** 3).astype(np.float32)
        wt[:, ::7] = 0
        n = [D // 3, 1, D, 5, D // 2][step]
        slots = torch.empty((R, n), dtype=torch.int32, device="cuda")
        counts = torch.empty((R,), dtype=torch.int32, device="cuda")
        wt_d = torch.from_numpy(wt).cuda()
        if step == 3:       # outputs are optional
            a.evict(0, wt_d, seq, n, keep_recent=9)
        else:
            a.evict(0, wt_d, seq, n, keep_recent=9, out_slots=slots, out_counts=counts)
        chosen = []
        for r in range(R):
            tok = before[0][r].copy()
            if protect:
                # slots that the last `protect` calls selected stay
                thr = max(1, int(before[4][r]) + 1 - protect)
                tok[before[1][r] >= thr] = -1
            at = M.evict(wt[r], tok, lens[r], 9, n)
            chosen.append(at)
            if step != 3:
                assert int(counts[r]) == at.size
                assert np.array_equal(slots[r, :at.size].cpu().numpy(), at)
        want = freed_state(before, off, chosen)
        for x, y, name in zip(a.read_state(0), want, ("slot2tok", "last_used", "tok2slot", "lru", "ticks")):
            assert np.array_equal(x, y), (step, name)
        b.write_state(0, want[0], want[1], want[4], rebuild_rows=False)
    # with two protected calls of 24 rows in 64 slots a third may not fit
    # (CAPACITY): then on both
    assert torch.equal(a.status(), b.status())
    assert 3 * k <= D or protect == 2 or (a.status() == 0).all()
    a.close()
    b.close()


def test_evict_refuses_bad_layers_and_counts():
    w = W.custom(2, 8, 32, [100, 60], row_bytes=32, layers=2, anchor_of_layer=[-1, 0])
    g = handle(w)
    seq = torch.from_numpy(w.seq_lens0).cuda()
    wt = torch.zeros((2, 100), device="cuda")
    for layer, n, recent, code in [(1, 4, 0, H.ERR_LAYER), (2, 4, 0, H.ERR_LAYER), (-1, 4, 0, H.ERR_LAYER),
                                   (0, 0, 0, H.ERR_INVALID_ARG), (0, 33, 0, H.ERR_INVALID_ARG),
                                   (0, 4, -1, H.ERR_INVALID_ARG)]:
        with pytest.raises(H.HiSparseError) as e:
            g.evict(layer, wt, seq, n, keep_recent=recent)
        assert e.value.code == code
    with pytest.raises(ValueError):
        g.evict(0, wt[:1], seq, 4)
    with pytest.raises(ValueError):     # 32-byte rows are not 4-bit rows
        g.attend(0, torch.zeros((2, 1, 576), dtype=torch.bfloat16, device="cuda"),
                 torch.zeros((2, 8), dtype=torch.int32, device="cuda"),
                 torch.zeros((2, 1, 512), dtype=torch.bfloat16, device="cuda"), 1.0)
    g.close()


@pytest.mark.parametrize("guards", ["1"])
def test_evict_writes_inside_its_arrays(guards, monkeypatch):
    monkeypatch.setenv("HISPARSE_DEBUG_GUARDS", guards)
    w = W.custom(3, 50, 1100, [3000, 2000, 1200], row_bytes=32)
    g = handle(w)
    seq = torch.from_numpy(w.seq_lens0).cuda()
    g.evict(0, torch.rand((3, 3000), device="cuda"), seq, 1100)
    assert g.check_guards() == 0
    s2t = g.read_state(0)[0]
    assert (s2t == -1).all()
    g.close()
