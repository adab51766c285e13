"""What the binding of the resident pages' calls checks before a launch, with the
GPU's part played by fakes (CPU only)."""

import types

import pytest
import torch

from hierarchical_sparse_kv_request_gb300 import hisparse as H
from test_rows4_binding import Elsewhere, Stream, Gpu, lib  # noqa: F401

R, HEADS, BLOCKS, PAGES, TOKENS, BS, LEN = 2, 3, 6, 10, 9, 4, 23


@pytest.fixture
def gpu(lib, monkeypatch):  # noqa: F811
    g = Gpu(lib)
    g.calls = []

    def record(name):
        def call(*args):
            g.calls.append((name, args))
            return H.OK
        return call

    g.lib = types.SimpleNamespace(
        hisparse_error_string=lib.hisparse_error_string,
        hisparse_attend_prefix_workspace=lib.hisparse_attend_prefix_workspace,
        **{n: record(n) for n in ("hisparse_page_tables", "hisparse_norm_rows", "hisparse_gather_rows",
                                  "hisparse_attend_prefix")})
    monkeypatch.setattr(H, "_torch", g.torch)
    monkeypatch.setattr(H, "_lib", g.lib)
    monkeypatch.setattr(H, "_raw_stream", lambda device: g.now.cuda_stream)
    monkeypatch.setattr(H, "_device", lambda: -1)     # the tensors' (the CPU's) number
    return g


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def tables():
    t = dict(lens=ints(R), tables=ints(R, BLOCKS), held=ints(R), free_list=ints(PAGES), free_count=ints(1),
             block_size=BS)
    more = dict(shared=ints(2), new_tokens=ints(R), offsets=ints(R + 1), slots=ints(TOKENS), positions=ints(TOKENS),
                status=ints(R))
    return t, more


def prefix():
    return dict(q=torch.zeros((R, HEADS, 576), dtype=torch.bfloat16), rows=torch.zeros((40, 656), dtype=torch.uint8),
                table=ints(6), block_size=BS, prefix_len=LEN, out=torch.zeros((R, HEADS, 512), dtype=torch.bfloat16),
                scale=1.0), dict(
        lse=torch.zeros((R, HEADS)), part=torch.zeros((R, HEADS, 512), dtype=torch.bfloat16),
        part_lse=torch.zeros((R, HEADS)), status=ints(R),
        workspace=torch.zeros(H.attend_prefix_workspace_bytes(R, HEADS, LEN), dtype=torch.uint8))


# -- page_tables --------------------------------------------------------------------

def test_page_tables_passes_what_it_got(gpu):
    t, more = tables()
    H.page_tables(**t)
    H.page_tables(**t, **more)
    a = H.PageTablesArgs.from_buffer_copy(gpu.calls[1][1][0])
    assert (a.num_requests, a.max_blocks, a.block_size, a.num_shared) == (R, BLOCKS, BS, 2)
    assert (a.free_capacity, a.num_tokens, a.tables_stride) == (PAGES, TOKENS, BLOCKS)
    for name in ("lens", "tables", "held", "free_list", "free_count", "shared", "new_tokens", "offsets", "slots",
                 "positions", "status"):
        x = t[name] if name in t else more[name]
        assert getattr(a, name) == x.data_ptr(), name
    a = H.PageTablesArgs.from_buffer_copy(gpu.calls[0][1][0])
    assert not (a.shared or a.new_tokens or a.offsets or a.slots or a.positions or a.status or a.num_tokens)


@pytest.mark.parametrize("name,bad", [
    ("lens", ints(R, 1)), ("lens", torch.zeros(R, dtype=torch.int64)), ("lens", ints(2 * R)[::2]),
    ("tables", ints(R + 1, BLOCKS)), ("tables", ints(BLOCKS, R).T), ("tables", torch.zeros((R, BLOCKS))),
    ("held", ints(R + 1)), ("held", torch.zeros(R)), ("free_count", ints(2)), ("free_list", ints(PAGES, 1)),
    ("free_list", ints(2 * PAGES)[::2]), ("shared", torch.zeros(2)), ("shared", ints(4)[::2]),
    ("new_tokens", ints(R + 1)), ("offsets", ints(R)), ("offsets", torch.zeros(R + 1)), ("slots", ints(3, 3)),
    ("slots", torch.zeros(TOKENS, dtype=torch.int64)), ("positions", ints(TOKENS - 1)), ("status", ints(R - 1)),
    ("status", torch.zeros(R))])
def test_page_tables_refuses_shapes_and_types(gpu, name, bad):
    t, more = tables()
    for d in (t, more):
        if name in d:
            d[name] = bad
    with pytest.raises(ValueError):
        H.page_tables(**t, **more)
    assert gpu.calls == []


@pytest.mark.parametrize("drop", [["offsets"], ["slots"], ["new_tokens"], ["offsets", "slots", "new_tokens"]])
def test_a_slot_map_is_asked_for_as_a_whole(gpu, drop):
    t, more = tables()
    for name in drop:
        del more[name]
    with pytest.raises(ValueError):
        H.page_tables(**t, **more)
    assert gpu.calls == []


@pytest.mark.parametrize("name", ["lens", "tables", "held", "free_list", "free_count", "shared", "new_tokens",
                                  "offsets", "slots", "positions", "status"])
def test_page_tables_refuses_tensors_of_another_device(gpu, name):
    t, more = tables()
    for d in (t, more):
        if name in d:
            d[name] = d[name].as_subclass(Elsewhere)
    with pytest.raises(ValueError):
        H.page_tables(**t, **more)
    assert gpu.calls == []


class Pinned(torch.Tensor):
    """A tensor in pinned host memory."""

    def get_device(self):
        return -1

    def is_pinned(self):
        return True


def test_only_inputs_may_be_pinned(gpu, monkeypatch):
    monkeypatch.setattr(H, "_device", lambda: 1)
    t, more = tables()
    everything = {k: (v.as_subclass(Elsewhere) if isinstance(v, torch.Tensor) else v) for k, v in {**t, **more}.items()}
    H.page_tables(**everything)
    for name in ("lens", "new_tokens", "shared"):
        pinned = everything[name].as_subclass(Pinned)
        H.page_tables(**{**everything, name: pinned})
        with pytest.raises(ValueError):       # pageable
            H.page_tables(**{**everything, name: ints(*everything[name].shape)})
    assert len(gpu.calls) == 4
    for name in ("tables", "held", "free_list", "free_count", "offsets", "slots", "positions", "status"):
        with pytest.raises(ValueError):
            H.page_tables(**{**everything, name: everything[name].as_subclass(Pinned)})
    assert len(gpu.calls) == 4


# -- rows ----------------------------------------------------------------------------

def rows():
    return dict(values=torch.zeros((5, 576), dtype=torch.float16), rows=torch.zeros((8, 656), dtype=torch.uint8),
                slots=ints(5))


@pytest.mark.parametrize("name,bad", [
    ("values", torch.zeros((5, 576))), ("values", torch.zeros((5, 575), dtype=torch.float16)),
    ("values", torch.zeros((576, 5), dtype=torch.float16).T), ("rows", torch.zeros((8, 657), dtype=torch.uint8)),
    ("rows", torch.zeros((8, 656), dtype=torch.int8)), ("rows", torch.zeros((2, 4, 656), dtype=torch.uint8)),
    ("rows", torch.zeros((656, 8), dtype=torch.uint8).T), ("slots", ints(4)), ("slots", torch.zeros(5, dtype=torch.int64)),
    ("slots", ints(10)[::2]), ("rows", rows()["rows"].as_subclass(Elsewhere)),
    ("values", rows()["values"].as_subclass(Elsewhere)), ("slots", ints(5).as_subclass(Elsewhere))])
def test_rows_are_refused(gpu, name, bad):
    a = rows()
    a[name] = bad
    for call in (H.norm_rows, H.gather_rows):
        with pytest.raises(ValueError):
            call(**a)
    assert gpu.calls == []


def test_rows_without_slots_need_as_many(gpu):
    a = rows()
    del a["slots"]
    H.norm_rows(**a)
    H.gather_rows(**a)
    a["rows"] = a["rows"][:4]
    for call in (H.norm_rows, H.gather_rows):
        with pytest.raises(ValueError):
            call(**a)
    assert len(gpu.calls) == 2


@pytest.mark.parametrize("weight", [torch.zeros(512), torch.zeros(511, dtype=torch.float16),
                                    torch.zeros(512, dtype=torch.bfloat16), torch.zeros(1024, dtype=torch.float16)[::2],
                                    torch.zeros(512, dtype=torch.float16).as_subclass(Elsewhere)])
def test_weights_are_refused(gpu, weight):
    with pytest.raises(ValueError):
        H.norm_rows(**rows(), weight=weight)
    assert gpu.calls == []
    H.norm_rows(**rows(), weight=torch.zeros(512, dtype=torch.float16))
    assert len(gpu.calls) == 1


# -- attend_prefix ---------------------------------------------------------------------

@pytest.mark.parametrize("stream,address", [(None, 0x111), (Stream(0x222), 0x222), (0x333, 0x333), (0, 0)])
def test_a_workspace_of_the_call_belongs_to_the_launch_stream(gpu, stream, address):
    t, _ = prefix()
    H.attend_prefix(**t, stream=stream)
    assert gpu.calls[0][1][1] == address
    assert gpu.allocations == [(address, H.attend_prefix_workspace_bytes(R, HEADS, LEN))]


def test_attend_prefix_passes_what_it_got(gpu):
    t, more = prefix()
    H.attend_prefix(**t, **more)
    a = H.AttendPrefixArgs.from_buffer_copy(gpu.calls[0][1][0])
    assert (a.num_requests, a.num_heads, a.dtype, a.row_bytes) == (R, HEADS, H.BF16, 656)
    assert (a.q_request_stride, a.q_head_stride, a.row_stride, a.num_rows) == (HEADS * 576, 576, 656, 40)
    assert (a.part_request_stride, a.part_head_stride) == (HEADS * 512, 512)
    assert (a.out_request_stride, a.out_head_stride) == (HEADS * 512, 512)
    assert (a.block_size, a.prefix_len, a.scale, a.workspace_bytes) == (BS, LEN, 1.0, more["workspace"].nbytes)
    for name in ("q", "rows", "table", "part", "part_lse", "out", "lse", "status", "workspace"):
        x = t[name] if name in t else more[name]
        assert getattr(a, name) == x.data_ptr(), name


B16 = torch.bfloat16


@pytest.mark.parametrize("name,bad", [
    ("q", torch.zeros((R, HEADS, 512), dtype=B16)), ("q", torch.zeros((R, HEADS, 576))),
    ("q", torch.zeros((R, HEADS, 576), dtype=torch.float16)), ("q", torch.zeros((HEADS, 576), dtype=B16)),
    ("out", torch.zeros((R, HEADS, 576), dtype=B16)), ("out", torch.zeros((R + 1, HEADS, 512), dtype=B16)),
    ("out", torch.zeros((R, HEADS, 512))), ("out", torch.zeros((R, 512, HEADS), dtype=B16).transpose(1, 2)),
    ("part", torch.zeros((R, HEADS, 511), dtype=B16)), ("part", torch.zeros((R, HEADS, 512), dtype=torch.float16)),
    ("part", None), ("part_lse", None), ("part_lse", torch.zeros((R, HEADS), dtype=torch.float64)),
    ("part_lse", torch.zeros((HEADS, R)).T), ("lse", torch.zeros((R, HEADS + 1))), ("lse", torch.zeros((HEADS, R)).T),
    ("rows", torch.zeros((40, 640), dtype=torch.uint8)), ("table", ints(5)), ("table", ints(6, 1)),
    ("table", torch.zeros(6, dtype=torch.int64)), ("block_size", 3), ("block_size", 0), ("prefix_len", 25),
    ("status", ints(R + 1)), ("workspace", torch.zeros(1 << 26, dtype=torch.uint8)[::2])])
def test_attend_prefix_refuses_shapes_and_types(gpu, name, bad):
    t, more = prefix()
    for d in (t, more):
        if name in d:
            d[name] = bad
    with pytest.raises(ValueError):
        H.attend_prefix(**t, **more)
    assert gpu.calls == []


@pytest.mark.parametrize("name", ["q", "rows", "table", "out", "lse", "part", "part_lse", "status", "workspace"])
def test_attend_prefix_refuses_tensors_of_another_device(gpu, name):
    t, more = prefix()
    for d in (t, more):
        if name in d:
            d[name] = d[name].as_subclass(Elsewhere)
    with pytest.raises(ValueError):
        H.attend_prefix(**t, **more)
    assert gpu.calls == []


def test_sizes_beyond_the_limits(gpu):
    t, _ = prefix()
    t["table"] = ints((1 << 20) // BS + 1)
    with pytest.raises(H.HiSparseError) as e:
        H.attend_prefix(**{**t, "prefix_len": (1 << 20) + 1})
    assert e.value.code == H.ERR_UNSUPPORTED
    with pytest.raises(H.HiSparseError) as e:
        H.attend_prefix(**{**t, "prefix_len": -1})
    assert e.value.code == H.ERR_INVALID_ARG
    assert gpu.calls == []
