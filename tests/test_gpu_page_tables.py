"""Block tables and slot maps on the GPU against the definition on lists
(pages_model.Tables): equal, entry by entry."""

import numpy as np
import pytest
import torch

import pages_model as M
from hierarchical_sparse_kv_request_gb300 import hisparse as H

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def gpu(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


class Both:
    """The same state on the GPU and in the model."""

    def __init__(self, R, W, bs, pages, shared=0, free=None, rng=None, stride=0):
        rng = rng or np.random.default_rng(0)
        ids = rng.permutation(pages + shared)
        self.bs, self.R, self.W = bs, R, W
        free = pages if free is None else free
        listed = np.full(pages, -7)
        listed[:free] = ids[shared:shared + free]
        self.model = M.Tables(np.full((R, W), -1), np.zeros(R), listed, free, ids[:shared], bs)
        whole = torch.full((R, W + stride), -1, dtype=torch.int32, device="cuda")
        self.tables, self.beside = whole[:, :W], whole[:, W:]
        self.held, self.free_list, self.free_count = gpu(np.zeros(R)), gpu(listed), gpu([free])
        self.shared = gpu(ids[:shared]) if shared else None
        self.status = gpu(np.zeros(R))

    def call(self, lens, new=None, tokens=0, positions=True, stream=None):
        out = {}
        if new is not None:
            out = dict(new_tokens=gpu(new), offsets=gpu(np.full(self.R + 1, 99)), slots=gpu(np.full(tokens, 99)),
                       positions=gpu(np.full(tokens, 99)) if positions else None)
        H.page_tables(gpu(lens), self.tables, self.held, self.free_list, self.free_count, self.bs, shared=self.shared,
                      status=self.status, stream=stream, **out)
        torch.cuda.synchronize()
        want = self.model.call(lens, new, tokens)
        self.same()
        if new is not None:
            assert np.array_equal(out["offsets"].cpu().numpy(), want[0])
            assert np.array_equal(out["slots"].cpu().numpy(), want[1])
            if positions:
                assert np.array_equal(out["positions"].cpu().numpy(), want[2])
        return out

    def same(self):
        m = self.model
        assert np.array_equal(self.tables.cpu().numpy(), m.tables)
        assert np.array_equal(self.held.cpu().numpy(), m.held)
        assert int(self.free_count) == m.count
        assert np.array_equal(self.free_list.cpu().numpy(), m.list)
        assert np.array_equal(self.status.cpu().numpy(), m.status)
        assert (self.beside == -1).all()


@pytest.mark.parametrize("R", [1, 2, 31, 32, 33, 257, 1025])
@pytest.mark.parametrize("bs", [1, 7, 64])
def test_requests_come_grow_shrink_and_go(R, bs):
    rng = np.random.default_rng(R * 100 + bs)
    W = 40
    b = Both(R, W, bs, R * W // 2 + 5, shared=3 if R % 2 else 0, rng=rng, stride=5)
    lens = np.zeros(R, dtype=np.int64)
    for step in range(12):
        kind = rng.integers(0, 5, R)
        lens = np.where(kind == 0, 0, np.where(kind == 1, rng.integers(0, W * bs + 1, R),
                        np.minimum(lens + rng.integers(0, 2 * bs + 1, R), W * bs)))
        asked = np.where(kind == 4, -1 - rng.integers(0, 3, R), lens)
        new = np.minimum(rng.integers(0, 6, R), np.maximum(asked, 0))
        if step % 3 == 2:
            b.call(asked)
        else:
            b.call(asked, new, int(new.sum()) + int(rng.integers(0, 70)), positions=step % 2 == 0)
        lens = np.array(b.model.held) * bs


@pytest.mark.parametrize("tokens", [0, 1, 4095, 4096, 4097, 16384, 16385, 20000])
def test_slots_in_one_launch_and_in_two(tokens):
    """On both sides of where the slots get a launch of their own, and with
    places behind the last token."""
    rng = np.random.default_rng(tokens)
    R, bs, W = 5, 16, 400
    b = Both(R, W, bs, R * W, rng=rng)
    new = np.sort(rng.integers(0, tokens + 1, R - 1)) if tokens else np.zeros(R - 1, dtype=np.int64)
    new = np.diff(np.concatenate([[0], new, [tokens]]))
    lens = new + rng.integers(0, 30, R)
    fits = lens <= W * bs
    lens, new = np.where(fits, lens, 3), np.where(fits, new, 3)
    b.call(lens, new, tokens)
    b.call(lens, new, max(int(new.sum()), 1))


@pytest.mark.parametrize("R", [3, 40, 300])
def test_too_few_pages(R):
    """Requests are served in their order until one does not fit; those that need
    nothing, or only shared pages, still are."""
    rng = np.random.default_rng(R)
    b = Both(R, 30, 4, R * 6, shared=5, rng=rng)
    lens = rng.integers(0, 121, R)
    b.call(lens, np.minimum(lens, 3), 4 * R)
    assert (b.model.status != 0).any()
    b.call(np.where(rng.random(R) < 0.5, 0, lens), np.zeros(R, dtype=int), 8)
    b.call(lens)


def test_there_and_back_again():
    """A call with other lengths and one with the old ones: as it was."""
    rng = np.random.default_rng(3)
    b = Both(60, 50, 8, 4000, shared=2, rng=rng)
    first, second = rng.integers(0, 401, 60), rng.integers(0, 401, 60)
    b.call(first)
    # (what the list holds past its count is left over from pages taken)
    state = lambda: (b.tables, b.held, b.free_count, b.free_list[:int(b.free_count)])  # noqa: E731
    before = [x.clone() for x in state()]
    b.call(second, np.minimum(second, 5), 300)
    b.call(first)
    assert all(torch.equal(x, y) for x, y in zip(before, state()))


def test_data_errors():
    b = Both(8, 10, 4, 200)
    b.call([9, 40, 17, 5, 0, 33, 12, 8])
    b.held[3], b.model.held[3] = 11, 11              # beyond the table
    b.held[5], b.model.held[5] = -1, -1
    lens = [9, 41, 17, 5, 2, 33, -1, 7]               # 1: longer than a table
    new = [10, 1, -3, 2, 2, 4, 2, 8]                  # 0: more than there are; 2: fewer than none; 6: left alone; 7: too many
    b.call(lens, new, 40)
    bits = b.model.status
    assert bits[1] == 1 << M.BAD_SEQ_LEN and bits[3] == 1 << M.BAD_INDEX and bits[5] == 1 << M.BAD_INDEX
    assert bits[0] == bits[2] == bits[6] == bits[7] == 1 << M.BAD_POSITION and bits[4] == 0
    b.call([9, 9, 9, 9, 9, 9, 9, 9], [1] * 8, 5)      # places for five of eight tokens


def test_a_free_count_that_is_none():
    """Too large or too small: taken as the nearest there is."""
    for count in (-5, 999):
        b = Both(3, 6, 4, 12)
        b.free_count[0] = count
        b.model.count = 0 if count < 0 else 12
        b.call([9, 8, 4], [1, 2, 3], 10)


def test_pages_past_the_flag_bit_have_no_slots():
    b = Both(2, 2, 1 << 20, 4)
    b.free_list.copy_(gpu([1022, 1023, 1024, 5]))
    b.model.list[:] = [1022, 1023, 1024, 5]
    b.call([1 << 20, 1 << 21], [2, (1 << 20) + 5], (1 << 20) + 7)
    assert b.model.status[1] == 1 << M.BAD_RESIDENT


@pytest.mark.parametrize("bs", [1, 2, 3, 5, 63, 65, 1000, 65535, 65537, (1 << 20) - 1, 1 << 30])
def test_block_sizes(bs):
    """Positions on both sides of pages' ends; the last of a length near 2^31 / 1024."""
    top = min(1024 * bs, (1 << 21) + 11)
    W = -(-top // bs)
    b = Both(2, W, bs, 2 * W)
    if bs == 1 << 30:
        b.free_list.zero_()              # page 0: the only one below the flag bit
        b.model.list[:] = 0
    for n in (1, bs, bs + 1, 2 * bs - 1, top):
        n = min(n, top)
        b.call([n, max(n - 1, 0)], [min(n, 50), min(n - 1, 50)], 128)
        b.call([0, 0])


@pytest.mark.parametrize("R", [8192])
def test_the_most_requests(R):
    rng = np.random.default_rng(1)
    b = Both(R, 4, 16, 2 * R, rng=rng)
    lens = rng.integers(0, 65, R)
    b.call(lens, np.minimum(lens, 2), 2 * R)
    b.call(lens, np.minimum(lens, 3), 3 * R + 5)
    b.call(np.zeros(R, dtype=int))


def test_captured_and_replayed():
    """A step of one more token each, captured once and replayed: the lengths, and
    all that the call keeps, are on the GPU."""
    R, bs = 6, 4
    b = Both(R, 30, bs, 200)
    b.call([10, 11, 12, 13, 14, 15])
    lens, new = gpu([10, 11, 12, 13, 14, 15]), gpu([1] * R)
    offsets, slots, positions = gpu(np.zeros(R + 1)), gpu(np.zeros(8)), gpu(np.zeros(8))

    def step():
        lens.add_(1)
        H.page_tables(lens, b.tables, b.held, b.free_list, b.free_count, bs, new_tokens=new, offsets=offsets, slots=slots,
                      positions=positions, status=b.status)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for n in range(1, 30):
        graph.replay()
        torch.cuda.synchronize()
        want = b.model.call([10 + n + r for r in range(R)], [1] * R, 8)
        b.same()
        assert np.array_equal(slots.cpu().numpy(), want[1]) and np.array_equal(positions.cpu().numpy(), want[2])


def test_another_stream_and_pinned_inputs():
    R, bs = 5, 8
    b = Both(R, 20, bs, 100)
    side = torch.cuda.Stream()
    b.call([30, 1, 0, 8, 9], [3, 1, 0, 2, 9], 20, stream=side)
    lens = torch.tensor([31, 9, 0, 100, 2], dtype=torch.int32).pin_memory()
    new = torch.tensor([1, 8, 0, 5, 0], dtype=torch.int32).pin_memory()
    offsets, slots = gpu(np.zeros(R + 1)), gpu(np.zeros(20))
    H.page_tables(lens, b.tables, b.held, b.free_list, b.free_count, bs, new_tokens=new, offsets=offsets, slots=slots,
                  stream=side.cuda_stream)
    torch.cuda.synchronize()
    want = b.model.call(lens.numpy(), new.numpy(), 20)
    b.same()
    assert np.array_equal(slots.cpu().numpy(), want[1]) and np.array_equal(offsets.cpu().numpy(), want[0])


@pytest.mark.slow
def test_long_tables():
    """Whole prompts come and go: every page of a large pool."""
    rng = np.random.default_rng(9)
    R, bs, W = 128, 64, 1280
    b = Both(R, W, bs, R * W, rng=rng)
    lens = rng.integers(2048, W * bs + 1, R)
    b.call(lens)
    b.call(np.zeros(R, dtype=int))
