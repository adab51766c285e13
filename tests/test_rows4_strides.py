"""Strides that hisparse_attend takes and refuses: host checks before any GPU work
(CPU only).  The workspace is too small in every call here, which is checked
last: CAPACITY says that nothing else was wrong."""

import ctypes

import pytest
import torch

from hierarchical_sparse_kv_request_gb300 import build as B
from hierarchical_sparse_kv_request_gb300 import hisparse as H
from test_rows4_api import good_args


@pytest.fixture(scope="module")
def lib():
    B.build_library()
    return H.load_library()


def call(lib, **change):
    a = good_args()
    for name, v in change.items():
        setattr(a, name, v)
    return lib.hisparse_attend(ctypes.byref(a), None)


@pytest.mark.parametrize("change", [
    dict(),
    dict(num_heads=1, q_head_stride=1), dict(num_heads=1, q_head_stride=580), dict(num_heads=1, out_head_stride=3),
    dict(num_heads=1, out_head_stride=0), dict(num_requests=1, q_request_stride=7),
    dict(num_requests=1, out_request_stride=1), dict(num_requests=1, request_stride=5),
    dict(num_requests=1, num_heads=1, q_request_stride=1, q_head_stride=1, out_request_stride=1, out_head_stride=1)])
def test_strides_of_a_single_head_or_request_mean_nothing(lib, change):
    assert call(lib, **change) == H.ERR_CAPACITY


@pytest.mark.parametrize("change", [
    dict(num_requests=1, q_head_stride=580), dict(num_requests=1, out_head_stride=516),
    dict(num_heads=1, q_request_stride=580), dict(num_heads=1, out_request_stride=516),
    dict(num_heads=1, request_stride=8)])
def test_strides_of_the_other_dimension_still_count(lib, change):
    assert call(lib, **change) == H.ERR_INVALID_ARG


@pytest.mark.parametrize("change,code", [
    (dict(out_head_stride=0), H.ERR_INVALID_ARG),            # one head's row for all
    (dict(out_request_stride=0), H.ERR_INVALID_ARG),
    (dict(out_head_stride=504), H.ERR_INVALID_ARG),
    (dict(out_head_stride=-8), H.ERR_INVALID_ARG),
    (dict(out_request_stride=-(1 << 63) + 16), H.ERR_CAPACITY),
    (dict(out_request_stride=512, out_head_stride=1024), H.ERR_CAPACITY),     # [H][R][512]
    (dict(out_request_stride=-1536, out_head_stride=-512), H.ERR_CAPACITY),
    (dict(q_request_stride=0, q_head_stride=0), H.ERR_CAPACITY)])             # read only: one query for all
def test_heads_of_out_may_not_overlap(lib, change, code):
    assert call(lib, **change) == code
