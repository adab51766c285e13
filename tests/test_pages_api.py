"""Refusals of the resident pages' calls: host checks that run before any GPU work
(CPU only)."""

import ctypes
import os
import re

import pytest

from hierarchical_sparse_kv_request_gb300 import build as B
from hierarchical_sparse_kv_request_gb300 import hisparse as H

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20      # a 16-byte aligned address that is never read
ROWS = [H.ROW4_BYTES, H.ROW8_BYTES, H.ROW16_BYTES]


@pytest.fixture(scope="module")
def lib():
    B.build_library()
    return H.load_library()


def test_constants_match_the_header():
    text = open(os.path.join(ROOT, "include", "hisparse_pages.h")).read()
    assert int(re.search(r"#define HISPARSE_ROW8_BYTES (\d+)", text).group(1)) == H.ROW8_BYTES
    assert int(re.search(r"#define HISPARSE_ROW16_BYTES (\d+)", text).group(1)) == H.ROW16_BYTES
    assert "#define HISPARSE_MAX_PREFIX (1 << 20)" in text and H.MAX_PREFIX == 1 << 20


# -- page_tables ----------------------------------------------------------------

def tables_args(**change):
    a = H.PageTablesArgs()
    a.num_requests, a.max_blocks, a.block_size, a.num_shared = 2, 8, 16, 0
    a.lens = a.tables = a.held = a.free_list = a.free_count = A
    a.tables_stride, a.free_capacity = 8, 20
    for name, v in change.items():
        setattr(a, name, v)
    return a


WITH_TOKENS = dict(new_tokens=A, offsets=A, slots=A, positions=A, num_tokens=10)


@pytest.mark.parametrize("change,code", [
    (dict(num_requests=0), H.ERR_INVALID_ARG), (dict(num_requests=-1), H.ERR_INVALID_ARG),
    (dict(max_blocks=0), H.ERR_INVALID_ARG), (dict(block_size=0), H.ERR_INVALID_ARG),
    (dict(block_size=-4), H.ERR_INVALID_ARG), (dict(free_capacity=0), H.ERR_INVALID_ARG),
    (dict(lens=None), H.ERR_INVALID_ARG), (dict(tables=None), H.ERR_INVALID_ARG),
    (dict(held=None), H.ERR_INVALID_ARG), (dict(free_list=None), H.ERR_INVALID_ARG),
    (dict(free_count=None), H.ERR_INVALID_ARG),
    (dict(num_shared=-1), H.ERR_INVALID_ARG), (dict(num_shared=9, shared=A), H.ERR_INVALID_ARG),
    (dict(num_shared=3), H.ERR_INVALID_ARG), (dict(tables_stride=7), H.ERR_INVALID_ARG),
    (dict(WITH_TOKENS, offsets=None), H.ERR_INVALID_ARG), (dict(WITH_TOKENS, slots=None), H.ERR_INVALID_ARG),
    (dict(WITH_TOKENS, num_tokens=-1), H.ERR_INVALID_ARG),
    (dict(num_requests=8193), H.ERR_UNSUPPORTED),
    (dict(max_blocks=(1 << 20) + 1, tables_stride=1 << 21), H.ERR_UNSUPPORTED),
    (dict(num_requests=4096, max_blocks=1 << 20, tables_stride=1 << 20), H.ERR_UNSUPPORTED),
    (dict(block_size=(1 << 30) + 1), H.ERR_UNSUPPORTED),
    (dict(WITH_TOKENS, num_tokens=(1 << 30) + 1), H.ERR_UNSUPPORTED),
])
def test_page_tables_refuses(lib, change, code):
    a = tables_args(**change)
    assert lib.hisparse_page_tables(ctypes.byref(a), None) == code


def test_null_arguments(lib):
    assert lib.hisparse_page_tables(None, None) == H.ERR_INVALID_ARG
    assert lib.hisparse_attend_prefix(None, None) == H.ERR_INVALID_ARG
    assert lib.hisparse_attend_prefix_workspace(1, 1, 1, None) == H.ERR_INVALID_ARG


# -- rows -------------------------------------------------------------------------

@pytest.mark.parametrize("row", ROWS)
@pytest.mark.parametrize("change,code", [
    (dict(values=None), H.ERR_INVALID_ARG), (dict(rows=None), H.ERR_INVALID_ARG),
    (dict(dtype=2), H.ERR_INVALID_ARG), (dict(dtype=-1), H.ERR_INVALID_ARG), (dict(n=-1), H.ERR_INVALID_ARG),
    (dict(vstride=568), H.ERR_INVALID_ARG), (dict(vstride=580), H.ERR_INVALID_ARG),
    (dict(rstride=-16), H.ERR_INVALID_ARG), (dict(rstride=8), H.ERR_INVALID_ARG),
    (dict(row=400), H.ERR_INVALID_ARG), (dict(count=-1), H.ERR_INVALID_ARG),
    (dict(slots=None, count=3), H.ERR_INVALID_ARG),
    (dict(values=A + 2), H.ERR_ALIGNMENT), (dict(rows=A + 8), H.ERR_ALIGNMENT),
    (dict(n=4 * 0x7FFFFFFF + 1), H.ERR_UNSUPPORTED),
])
def test_rows_refuse(lib, row, change, code):
    a = dict(values=A, vstride=576, dtype=0, n=4, rows=A, rstride=0, row=row, count=100, slots=A)
    a.update(change)
    stride = a["row"] + a["rstride"]
    assert lib.hisparse_norm_rows(a["values"], a["vstride"], a["dtype"], a["n"], A, 1e-6, a["rows"], stride,
                                  a["row"], a["count"], a["slots"], None) == code
    assert lib.hisparse_gather_rows(a["rows"], stride, a["row"], a["count"], a["slots"], a["n"], a["values"],
                                    a["vstride"], a["dtype"], None) == code


@pytest.mark.parametrize("weight,eps,code", [(A + 8, 1e-6, H.ERR_ALIGNMENT), (A, -1e-6, H.ERR_INVALID_ARG),
                                             (A, float("nan"), H.ERR_INVALID_ARG)])
def test_norm_rows_refuses_weights_and_eps(lib, weight, eps, code):
    assert lib.hisparse_norm_rows(A, 576, 0, 4, weight, eps, A, 656, 656, 100, A, None) == code


def test_nothing_to_move_is_ok(lib):
    for row in ROWS:
        assert lib.hisparse_norm_rows(None, 576, 0, 0, None, 0.0, None, row, row, 0, None, None) == H.OK
        assert lib.hisparse_gather_rows(None, row, row, 0, None, 0, None, 576, 1, None) == H.OK
        # no rows: nothing has a slot
        assert lib.hisparse_norm_rows(A, 576, 0, 5, None, 0.0, None, row, row, 0, A, None) == H.OK
        assert lib.hisparse_gather_rows(None, row, row, 0, A, 5, A, 576, 1, None) == H.OK


# -- attend_prefix --------------------------------------------------------------------

def prefix_args(lib, **change):
    a = H.AttendPrefixArgs()
    a.num_requests, a.num_heads, a.dtype, a.row_bytes = 2, 3, H.BF16, H.ROW8_BYTES
    a.q, a.q_request_stride, a.q_head_stride = A, 3 * 576, 576
    a.rows, a.row_stride, a.num_rows = A, 656, 640
    a.table, a.block_size, a.prefix_len, a.scale = A, 64, 500, 1.0
    a.part, a.part_request_stride, a.part_head_stride, a.part_lse = A, 3 * 512, 512, A
    a.out, a.out_request_stride, a.out_head_stride, a.lse = A, 3 * 512, 512, A
    a.workspace, a.workspace_bytes = A, 1 << 40
    for name, v in change.items():
        setattr(a, name, v)
    return a


@pytest.mark.parametrize("change,code", [
    (dict(num_requests=0), H.ERR_INVALID_ARG), (dict(num_heads=0), H.ERR_INVALID_ARG),
    (dict(prefix_len=-1), H.ERR_INVALID_ARG), (dict(dtype=3), H.ERR_INVALID_ARG),
    (dict(row_bytes=657), H.ERR_INVALID_ARG), (dict(row_bytes=H.ROW16_BYTES), H.ERR_INVALID_ARG),   # stride 656
    (dict(q=None), H.ERR_INVALID_ARG), (dict(out=None), H.ERR_INVALID_ARG), (dict(workspace=None), H.ERR_INVALID_ARG),
    (dict(rows=None), H.ERR_INVALID_ARG), (dict(num_rows=-1), H.ERR_INVALID_ARG), (dict(table=None), H.ERR_INVALID_ARG),
    (dict(block_size=0), H.ERR_INVALID_ARG), (dict(part=None), H.ERR_INVALID_ARG), (dict(part_lse=None), H.ERR_INVALID_ARG),
    (dict(row_stride=648), H.ERR_INVALID_ARG), (dict(row_stride=664), H.ERR_INVALID_ARG),
    (dict(q_request_stride=1732), H.ERR_INVALID_ARG), (dict(q_head_stride=580), H.ERR_INVALID_ARG),
    (dict(part_head_stride=516), H.ERR_INVALID_ARG), (dict(part_request_stride=1540), H.ERR_INVALID_ARG),
    (dict(out_head_stride=0), H.ERR_INVALID_ARG), (dict(out_head_stride=504), H.ERR_INVALID_ARG),
    (dict(out_request_stride=8), H.ERR_INVALID_ARG), (dict(out_head_stride=-504), H.ERR_INVALID_ARG),
    (dict(num_requests=8193), H.ERR_UNSUPPORTED), (dict(num_heads=1025), H.ERR_UNSUPPORTED),
    (dict(prefix_len=(1 << 20) + 1), H.ERR_UNSUPPORTED),
    (dict(q=A + 8), H.ERR_ALIGNMENT), (dict(rows=A + 8), H.ERR_ALIGNMENT), (dict(part=A + 2), H.ERR_ALIGNMENT),
    (dict(out=A + 4), H.ERR_ALIGNMENT), (dict(workspace=A + 8), H.ERR_ALIGNMENT),
    (dict(workspace_bytes=0), H.ERR_CAPACITY), (dict(workspace_bytes=-1), H.ERR_CAPACITY),
])
def test_attend_prefix_refuses(lib, change, code):
    a = prefix_args(lib, **change)
    assert lib.hisparse_attend_prefix(ctypes.byref(a), None) == code


def test_the_workspace_is_what_is_asked_for(lib):
    for sizes in ((1, 1, 0), (1, 1, 1), (32, 128, 8192), (8192, 1024, 1), (1, 1, 1 << 20), (37, 40, 5003)):
        n = H.attend_prefix_workspace_bytes(*sizes)
        assert n >= 16
        a = prefix_args(lib, num_requests=sizes[0], num_heads=sizes[1], prefix_len=sizes[2], workspace_bytes=n - 1,
                        q_request_stride=sizes[1] * 576, out_request_stride=sizes[1] * 512,
                        part_request_stride=sizes[1] * 512)
        assert lib.hisparse_attend_prefix(ctypes.byref(a), None) == H.ERR_CAPACITY
    # the expanded rows are 1,152 bytes each, in tiles of 128
    assert H.attend_prefix_workspace_bytes(1, 1, 1 << 20) >= (1 << 20) * 1152


@pytest.mark.parametrize("sizes,code", [((0, 1, 1), H.ERR_INVALID_ARG), ((1, 0, 1), H.ERR_INVALID_ARG),
                                        ((1, 1, -1), H.ERR_INVALID_ARG), ((8193, 1, 1), H.ERR_UNSUPPORTED),
                                        ((1, 1025, 1), H.ERR_UNSUPPORTED), ((1, 1, (1 << 20) + 1), H.ERR_UNSUPPORTED)])
def test_the_workspace_refuses(lib, sizes, code):
    n = ctypes.c_int64(7)
    assert lib.hisparse_attend_prefix_workspace(*sizes, ctypes.byref(n)) == code
    assert n.value == 0
