"""Refusals of the 4-bit row calls: host checks that run before any GPU work
(CPU only), and the binding's own checks of tensors."""

import ctypes
import os
import re

import pytest
import torch

from hierarchical_sparse_kv_request_gb300 import build as B
from hierarchical_sparse_kv_request_gb300 import hisparse as H

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20      # a 16-byte aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    B.build_library()
    return H.load_library()


@pytest.mark.parametrize("args,code", [
    ((None, 576, 0, 4, A, 416), H.ERR_INVALID_ARG),
    ((A, 576, 0, 4, None, 416), H.ERR_INVALID_ARG),
    ((A, 576, 2, 4, A, 416), H.ERR_INVALID_ARG),       # no such type
    ((A, 576, -1, 4, A, 416), H.ERR_INVALID_ARG),
    ((A, 576, 0, -1, A, 416), H.ERR_INVALID_ARG),
    ((A, 568, 0, 4, A, 416), H.ERR_INVALID_ARG),       # stride below the row
    ((A, 580, 0, 4, A, 416), H.ERR_INVALID_ARG),       # stride off 16 bytes
    ((A, 576, 0, 4, A, 400), H.ERR_INVALID_ARG),
    ((A, 576, 0, 4, A, 424), H.ERR_INVALID_ARG),
    ((A + 2, 576, 0, 4, A, 416), H.ERR_ALIGNMENT),
    ((A, 576, 1, 4, A + 8, 416), H.ERR_ALIGNMENT),
])
def test_pack_and_unpack_refuse(lib, args, code):
    v, vs, dt, n, r, rs = args
    assert lib.hisparse_pack_rows(v, vs, dt, n, r, rs, None) == code
    assert lib.hisparse_unpack_rows(r, rs, n, v, vs, dt, None) == code


def test_more_rows_than_a_launch_takes(lib):
    n = 4 * 0x7FFFFFFF + 1
    assert lib.hisparse_pack_rows(A, 576, 0, n, A, 416, None) == H.ERR_UNSUPPORTED
    assert lib.hisparse_unpack_rows(A, 416, n, A, 576, 0, None) == H.ERR_UNSUPPORTED


def test_nothing_to_pack_is_ok(lib):
    assert lib.hisparse_pack_rows(None, 576, 0, 0, None, 416, None) == H.OK
    assert lib.hisparse_unpack_rows(None, 416, 0, None, 576, 1, None) == H.OK


def good_args():
    a = H.AttendArgs()
    a.num_requests, a.num_heads, a.top_k, a.dtype = 2, 3, 5, H.BF16
    a.q, a.q_request_stride, a.q_head_stride = A, 3 * 576, 576
    a.rows, a.row_stride, a.request_stride, a.rows_per_request = A, 416, 416 * 8, 8
    a.scale = 1.0
    a.slot_ids, a.ids_stride = A, 5
    a.out, a.out_request_stride, a.out_head_stride = A, 3 * 512, 512
    a.workspace, a.workspace_bytes = A, 0     # too small: nothing here may launch
    return a


@pytest.mark.parametrize("change,code", [
    (dict(num_requests=0), H.ERR_INVALID_ARG),
    (dict(num_heads=0), H.ERR_INVALID_ARG),
    (dict(top_k=0), H.ERR_INVALID_ARG),
    (dict(num_requests=8193), H.ERR_UNSUPPORTED),
    (dict(num_heads=H.MAX_HEADS + 1), H.ERR_UNSUPPORTED),
    (dict(top_k=8193), H.ERR_UNSUPPORTED),
    (dict(dtype=2), H.ERR_INVALID_ARG),
    (dict(q=None), H.ERR_INVALID_ARG),
    (dict(rows=None), H.ERR_INVALID_ARG),
    (dict(slot_ids=None), H.ERR_INVALID_ARG),
    (dict(out=None), H.ERR_INVALID_ARG),
    (dict(workspace=None), H.ERR_INVALID_ARG),
    (dict(rows_per_request=0), H.ERR_INVALID_ARG),
    (dict(ids_stride=4), H.ERR_INVALID_ARG),
    (dict(q_head_stride=580), H.ERR_INVALID_ARG),
    (dict(q_request_stride=3 * 576 + 4), H.ERR_INVALID_ARG),
    (dict(out_head_stride=516), H.ERR_INVALID_ARG),
    (dict(out_request_stride=1540), H.ERR_INVALID_ARG),
    (dict(row_stride=400), H.ERR_INVALID_ARG),
    (dict(row_stride=420), H.ERR_INVALID_ARG),
    (dict(request_stride=8), H.ERR_INVALID_ARG),
    (dict(resident_count=4), H.ERR_INVALID_ARG),
    (dict(resident_count=-1), H.ERR_INVALID_ARG),
    (dict(resident_count=4, resident_rows=A, resident_stride=400), H.ERR_INVALID_ARG),
    (dict(weights=A, weights_stride=10, weights_tokens=10), H.ERR_INVALID_ARG),   # no positions
    (dict(weights=A, weights_stride=10, weights_tokens=11, positions=A, positions_stride=5), H.ERR_INVALID_ARG),
    (dict(weights=A, weights_stride=10, weights_tokens=10, positions=A, positions_stride=4), H.ERR_INVALID_ARG),
    (dict(q=A + 8), H.ERR_ALIGNMENT),
    (dict(rows=A + 4), H.ERR_ALIGNMENT),
    (dict(out=A + 2), H.ERR_ALIGNMENT),
    (dict(workspace=A + 8), H.ERR_ALIGNMENT),
    (dict(resident_count=4, resident_rows=A + 8, resident_stride=416), H.ERR_ALIGNMENT),
])
def test_attend_refuses(lib, change, code):
    a = good_args()
    for name, v in change.items():
        setattr(a, name, v)
    assert lib.hisparse_attend(ctypes.byref(a), None) == code


def test_attend_workspace_refuses(lib):
    n = ctypes.c_int64()
    assert lib.hisparse_attend(None, None) == H.ERR_INVALID_ARG
    assert lib.hisparse_attend_workspace(1, 1, 1, 0, None) == H.ERR_INVALID_ARG
    assert lib.hisparse_attend_workspace(0, 1, 1, 0, ctypes.byref(n)) == H.ERR_INVALID_ARG
    assert lib.hisparse_attend_workspace(1, 1025, 1, 0, ctypes.byref(n)) == H.ERR_UNSUPPORTED
    assert lib.hisparse_attend_workspace(1, 1, 8193, 0, ctypes.byref(n)) == H.ERR_UNSUPPORTED


@pytest.mark.parametrize("change,code", [
    (dict(weights=None), H.ERR_INVALID_ARG),
    (dict(slot2tok=None), H.ERR_INVALID_ARG),
    (dict(seq=None), H.ERR_INVALID_ARG),
    (dict(out=None), H.ERR_INVALID_ARG),
    (dict(counts=None), H.ERR_INVALID_ARG),
    (dict(R=0), H.ERR_INVALID_ARG),
    (dict(D=0), H.ERR_INVALID_ARG),
    (dict(n=0), H.ERR_INVALID_ARG),
    (dict(n=17), H.ERR_INVALID_ARG),
    (dict(recent=-1), H.ERR_INVALID_ARG),
    (dict(tokens=-1), H.ERR_INVALID_ARG),
    (dict(tokens=101), H.ERR_INVALID_ARG),
    (dict(D=32769), H.ERR_UNSUPPORTED),
    (dict(R=8193), H.ERR_UNSUPPORTED),
])
def test_evict_select_refuses(lib, change, code):
    v = dict(R=2, D=16, weights=A, stride=100, tokens=100, slot2tok=A, seq=A, recent=0, n=4, want=None,
             out=A, counts=A)
    v.update(change)
    assert lib.hisparse_evict_select(*[v[x] for x in (
        "R", "D", "weights", "stride", "tokens", "slot2tok", "seq", "recent", "n", "want", "out",
        "counts")], None) == code


def test_evict_refuses_a_null_handle(lib):
    assert lib.hisparse_evict(None, 0, A, 10, 10, A, 0, 1, None, None, None, None) == H.ERR_INVALID_ARG


def test_binding_constants_match_the_header():
    text = open(os.path.join(ROOT, "include", "hisparse_rows4.h")).read()
    defs = dict(re.findall(r"#define\s+HISPARSE_(\w+)\s+(\d+)", text))
    for name, value in {"ROW4_LATENT": H.ROW4_LATENT, "ROW4_ROPE": H.ROW4_ROPE,
                        "ROW4_VALUES": H.ROW4_VALUES, "ROW4_BYTES": H.ROW4_BYTES, "BF16": H.BF16,
                        "F16": H.F16, "MAX_HEADS": H.MAX_HEADS,
                        "STATUS_ATTEND_TIMEOUT": H.STATUS_ATTEND_TIMEOUT}.items():
        assert int(defs[name]) == value, name


def test_binding_struct_matches_the_header():
    """Field names and order of hisparse_attend_args."""
    text = open(os.path.join(ROOT, "include", "hisparse_rows4.h")).read()
    body = re.search(r"typedef struct hisparse_attend_args \{(.*?)\}", text, re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    names = re.findall(r"(\w+)\s*;", body)
    assert names == [f[0] for f in H.AttendArgs._fields_]


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("call", [
    lambda: H.pack_rows(t(4, 576, dtype=torch.float32), t(4, 416, dtype=torch.uint8)),
    lambda: H.pack_rows(t(4, 575), t(4, 416, dtype=torch.uint8)),
    lambda: H.pack_rows(t(4, 576), t(3, 416, dtype=torch.uint8)),
    lambda: H.pack_rows(t(4, 576), t(4, 432, dtype=torch.uint8)),
    lambda: H.pack_rows(t(576, 4).T, t(4, 416, dtype=torch.uint8)),
    lambda: H.unpack_rows(t(4, 416), t(4, 576)),
    lambda: H.attend(t(2, 3, 512), t(2, 8, 416, dtype=torch.uint8), t(2, 5, dtype=torch.int32),
                     t(2, 3, 512), 1.0),
    lambda: H.attend(t(2, 3, 576), t(2, 8, 416, dtype=torch.uint8), t(2, 5, dtype=torch.int64),
                     t(2, 3, 512), 1.0),
    lambda: H.attend(t(2, 3, 576), t(2, 8, 416, dtype=torch.uint8), t(2, 5, dtype=torch.int32),
                     t(2, 3, 512, dtype=torch.float16), 1.0),
    lambda: H.attend(t(2, 3, 576), t(2, 8, 416, dtype=torch.uint8), t(2, 5, dtype=torch.int32),
                     t(2, 3, 512), 1.0, lse=t(2, 2, dtype=torch.float32)),
    lambda: H.attend(t(2, 3, 576), t(2, 8, 416, dtype=torch.uint8), t(2, 5, dtype=torch.int32),
                     t(2, 3, 512), 1.0, weights=t(2, 9, dtype=torch.float32)),
    lambda: H.attend(t(2, 3, 576), t(2, 8, 416, dtype=torch.uint8), t(2, 5, dtype=torch.int32),
                     t(2, 3, 512), 1.0, weights=t(2, 9, dtype=torch.float32),
                     positions=t(2, 6, dtype=torch.int32)),
    lambda: H.evict_select(t(2, 9, dtype=torch.float64), t(2, 4, dtype=torch.int32),
                           t(2, dtype=torch.int32), t(2, 2, dtype=torch.int32), t(2, dtype=torch.int32)),
    lambda: H.evict_select(t(2, 9, dtype=torch.float32), t(2, 4, dtype=torch.int32),
                           t(3, dtype=torch.int32), t(2, 2, dtype=torch.int32), t(2, dtype=torch.int32)),
])
def test_binding_refuses(lib, call):
    with pytest.raises(ValueError):
        call()
