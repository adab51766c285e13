"""Thin ctypes binding of libhisparse.so (include/hisparse.h).

Argument marshalling only: every step of the swap-in path runs in the CUDA
library.  Device arrays may be passed as torch CUDA tensors or raw integer
addresses; streams as torch streams, raw ``cudaStream_t`` integers or None
(torch's current stream).  There is no CPU fallback: if the library is not
built, loading it raises.
"""

from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional, Sequence

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libhisparse.so")

OK = 0
ERR_INVALID_ARG, ERR_LAYOUT, ERR_CAPACITY, ERR_LAYER = -1, -2, -3, -4
ERR_CUDA, ERR_NO_MEMORY, ERR_UNSUPPORTED, ERR_ALIGNMENT = -5, -6, -7, -8
STATUS_OK, STATUS_BAD_INDEX, STATUS_DUPLICATE, STATUS_BAD_SEQ_LEN, STATUS_BAD_POSITION = 0, 1, 2, 3, 4
STATUS_BAD_RESIDENT, STATUS_NO_HOST_ROW, STATUS_CAPACITY, STATUS_COPY_TIMEOUT = 5, 6, 7, 8
STATUS_ATTEND_TIMEOUT = 9


def STATUS_BIT(code: int) -> int:
    """The bit a status code sets in a request's status word."""
    return 1 << code


RESIDENT_FLAG = 1 << 30
COPY_FUSED, COPY_SPLIT, COPY_AUTO = 1, 2, 3
NOALLOC_SCRATCH_BYTES = 8 << 20   # HISPARSE_NOALLOC_SCRATCH_BYTES

# 4-bit rows (include/hisparse_rows4.h)
ROW4_LATENT, ROW4_ROPE, ROW4_VALUES, ROW4_BYTES = 512, 64, 576, 416
BF16, F16 = 0, 1
MAX_HEADS = 1024

# resident pages (include/hisparse_pages.h)
ROW8_BYTES, ROW16_BYTES = 656, 1152
MAX_PREFIX = 1 << 20


class HiSparseError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {error_string(code)} ({code})")
        self.code = code


class Layout(ctypes.Structure):
    _fields_ = [("num_requests", ctypes.c_int32), ("num_layers", ctypes.c_int32),
                ("row_bytes", ctypes.c_int64), ("top_k", ctypes.c_int32),
                ("device_buffer_size", ctypes.c_int32),
                ("host_to_device_ratio", ctypes.c_int32),
                ("swap_in_block_size", ctypes.c_int32),
                ("anchor_of_layer", ctypes.c_void_p), ("host_capacity", ctypes.c_void_p)]


class Plan(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_void_p), ("counts", ctypes.c_void_p)]


class AttendArgs(ctypes.Structure):
    """hisparse_attend_args (attend() fills it in with struct: 0.9 -> 0.3 us)."""
    _fields_ = [("num_requests", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("q", ctypes.c_void_p), ("q_request_stride", ctypes.c_int64),
                ("q_head_stride", ctypes.c_int64),
                ("rows", ctypes.c_void_p), ("row_stride", ctypes.c_int64),
                ("request_stride", ctypes.c_int64), ("rows_per_request", ctypes.c_int32),
                ("scale", ctypes.c_float),
                ("slot_ids", ctypes.c_void_p), ("ids_stride", ctypes.c_int64),
                ("resident_rows", ctypes.c_void_p), ("resident_stride", ctypes.c_int64),
                ("resident_count", ctypes.c_int64),
                ("out", ctypes.c_void_p), ("out_request_stride", ctypes.c_int64),
                ("out_head_stride", ctypes.c_int64),
                ("lse", ctypes.c_void_p),
                ("weights", ctypes.c_void_p), ("weights_stride", ctypes.c_int64),
                ("weights_tokens", ctypes.c_int64),
                ("positions", ctypes.c_void_p), ("positions_stride", ctypes.c_int64),
                ("status", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64)]


class PageTablesArgs(ctypes.Structure):
    """hisparse_page_tables_args."""
    _fields_ = [("num_requests", ctypes.c_int32), ("max_blocks", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("num_shared", ctypes.c_int32),
                ("lens", ctypes.c_void_p), ("tables", ctypes.c_void_p),
                ("tables_stride", ctypes.c_int64), ("held", ctypes.c_void_p),
                ("free_list", ctypes.c_void_p), ("free_capacity", ctypes.c_int32),
                ("free_count", ctypes.c_void_p), ("shared", ctypes.c_void_p),
                ("new_tokens", ctypes.c_void_p), ("offsets", ctypes.c_void_p),
                ("slots", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("num_tokens", ctypes.c_int32), ("status", ctypes.c_void_p)]


class AttendPrefixArgs(ctypes.Structure):
    """hisparse_attend_prefix_args."""
    _fields_ = [("num_requests", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("row_bytes", ctypes.c_int32),
                ("q", ctypes.c_void_p), ("q_request_stride", ctypes.c_int64),
                ("q_head_stride", ctypes.c_int64),
                ("rows", ctypes.c_void_p), ("row_stride", ctypes.c_int64),
                ("num_rows", ctypes.c_int64), ("table", ctypes.c_void_p),
                ("block_size", ctypes.c_int32), ("prefix_len", ctypes.c_int32),
                ("scale", ctypes.c_float),
                ("part", ctypes.c_void_p), ("part_request_stride", ctypes.c_int64),
                ("part_head_stride", ctypes.c_int64), ("part_lse", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("out_request_stride", ctypes.c_int64),
                ("out_head_stride", ctypes.c_int64), ("lse", ctypes.c_void_p),
                ("status", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64)]


def _packer(args):
    """struct.pack with the layout of a ctypes structure."""
    return struct.Struct("@" + "".join(
        {ctypes.c_int32: "i", ctypes.c_int64: "q", ctypes.c_float: "f", ctypes.c_void_p: "P"}[t]
        for _, t in args._fields_)).pack


_pack_attend_args = _packer(AttendArgs)
_pack_page_tables_args = _packer(PageTablesArgs)
_pack_attend_prefix_args = _packer(AttendPrefixArgs)
_lib: Optional[ctypes.CDLL] = None


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libhisparse.so (built in-tree by ``__graft_entry__.build()``)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is missing: build the CUDA library first "
                           "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(p)
    P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    sig = {
        "hisparse_create": [P, P],
        "hisparse_create_paged": [P, I32, P],
        "hisparse_host_reserve": [P, I32, P, P, P],
        "hisparse_host_release": [P, I32, P, P],
        "hisparse_host_block_table": [P, I32, P, I32, P],
        "hisparse_host_pool_info": [P, P, P, P],
        "hisparse_host_block_rows": [P, I32, I32, P],
        "hisparse_destroy": [P],
        "hisparse_host_rows": [P, I32, I32, P],
        "hisparse_device_buffer": [P, I32, P],
        "hisparse_prefill": [P, P, P],
        "hisparse_swap_in": [P, I32, P, P, P, P, P],
        "hisparse_swap_in_noalloc": [P, I32, P, P, P, P],
        "hisparse_swap_in_resident": [P, I32, P, P, P, I32, I32, P, P, P],
        "hisparse_replay_plan": [P, P, I32, I32, P],
        "hisparse_replay_plan_layers": [P, P, P, I32, I32, P],
        "hisparse_backup": [P, I32, P, P, P],
        "hisparse_backup_layers": [P, P, I32, P, P, P],
        "hisparse_status": [P, P],
        "hisparse_status_clear": [P, P],
        "hisparse_read_state": [P, I32, P, P, P, P, P, P],
        "hisparse_write_state": [P, I32, P, P, P, I32, P],
        "hisparse_set_copy_mode": [P, I32],
        "hisparse_set_protected_calls": [P, I32],
        "hisparse_set_stage_rows": [P, I32],
        "hisparse_set_programmatic_launch": [P, I32],
        "hisparse_set_copy_ctas": [P, I32],
        "hisparse_get_copy_ctas": [P, P],
        "hisparse_get_device": [P, P],
        "hisparse_check_guards": [P, P],
        "hisparse_version": [],
        "hisparse_synthetic_compute": [P, I64, I32, I32, P],
        "hisparse_link_probe": [P, P, I64, I32, P],
        "hisparse_link_gather": [P, I64, P, I64, P, I32, P],
        "hisparse_pack_rows": [P, I64, I32, I64, P, I64, P],
        "hisparse_unpack_rows": [P, I64, I64, P, I64, I32, P],
        "hisparse_attend": [P, P],
        "hisparse_attend_workspace": [I32, I32, I32, I32, P],
        "hisparse_evict_select": [I32, I32, P, I64, I64, P, P, I32, I32, P, P, P, P],
        "hisparse_evict": [P, I32, P, I64, I64, P, I32, I32, P, P, P, P],
        "hisparse_page_tables": [P, P],
        "hisparse_norm_rows": [P, I64, I32, I64, P, ctypes.c_float, P, I64, I32, I64, P, P],
        "hisparse_gather_rows": [P, I64, I32, I64, P, I64, P, I64, I32, P],
        "hisparse_attend_prefix": [P, P],
        "hisparse_attend_prefix_workspace": [I32, I32, I32, P],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    lib.hisparse_error_string.argtypes = [ctypes.c_int]
    lib.hisparse_error_string.restype = ctypes.c_char_p
    if path is None:
        _lib = lib
    return lib


def error_string(code: int) -> str:
    try:
        return load_library().hisparse_error_string(code).decode()
    except RuntimeError:
        return "unknown"


def _addr(x) -> Optional[int]:
    """Device/host address of a torch tensor, numpy array or raw integer."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if isinstance(x, np.ndarray):
        return x.ctypes.data
    return x.data_ptr()


_torch = _raw_stream = _device = None


def _current_device() -> int:
    return _device() if _device is not None else (_torch or _load_torch()).cuda.current_device()


def _load_torch():
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _current_stream() -> int:
    """Initialises CUDA, and leaves behind the same call without Stream and
    Device objects where torch has it (2.9 -> 0.3 us)."""
    global _raw_stream, _device
    t = _torch or _load_torch()
    stream = t.cuda.current_stream().cuda_stream
    _device = getattr(t._C, "_cuda_getDevice", None)
    _raw_stream = _device and getattr(t._C, "_cuda_getCurrentRawStream", None)
    return stream


def _stream(s) -> Optional[int]:
    if s is None:
        return _raw_stream(_device()) if _raw_stream is not None else _current_stream()
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(rc: int, what: str) -> None:
    if rc != OK:
        raise HiSparseError(rc, what)


class HiSparse:
    """One handle of the swap-in resolver (see include/hisparse.h).

    host_block_tokens > 0 creates a paged host pool (hisparse_create_paged):
    host_capacity then only bounds each request's length, and rows come from
    blocks that host_reserve hands out."""

    def __init__(self, num_requests: int, num_layers: int, row_bytes: int, top_k: int,
                 device_buffer_size: int, host_to_device_ratio: int,
                 host_capacity: Sequence[int], anchor_of_layer: Optional[Sequence[int]] = None,
                 swap_in_block_size: int = 960, host_block_tokens: int = 0):
        self.lib = load_library()
        self.R, self.L, self.B = num_requests, num_layers, row_bytes
        self.k, self.D = top_k, device_buffer_size
        self.cap = np.ascontiguousarray(host_capacity, dtype=np.int64)
        self.anchor = np.ascontiguousarray(
            anchor_of_layer if anchor_of_layer is not None else [-1] * num_layers, dtype=np.int32)
        self.total_cap = int(self.cap.sum())
        lay = Layout(num_requests, num_layers, row_bytes, top_k, device_buffer_size,
                     host_to_device_ratio, swap_in_block_size,
                     self.anchor.ctypes.data, self.cap.ctypes.data)
        h = ctypes.c_void_p()
        self.hb = int(host_block_tokens)
        if self.hb:
            _check(self.lib.hisparse_create_paged(ctypes.byref(lay), self.hb, ctypes.byref(h)),
                   "hisparse_create_paged")
        else:
            _check(self.lib.hisparse_create(ctypes.byref(lay), ctypes.byref(h)), "hisparse_create")
        self.h = h
        device = ctypes.c_int32(-1)
        _check(self.lib.hisparse_get_device(self.h, ctypes.byref(device)), "hisparse_get_device")
        self.device = device.value

    @classmethod
    def for_workload(cls, w, host_block_tokens: int = 0) -> "HiSparse":
        return cls(w.num_requests, w.num_layers, w.row_bytes, w.top_k, w.device_buffer_size,
                   w.host_to_device_ratio, w.host_capacity, w.anchor_of_layer,
                   host_block_tokens=host_block_tokens)

    def close(self) -> None:
        if getattr(self, "h", None) and self.h.value:
            self.lib.hisparse_destroy(self.h)
            self.h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- storage ------------------------------------------------------------
    def host_rows_ptr(self, layer: int, request: int) -> int:
        p = ctypes.c_void_p()
        _check(self.lib.hisparse_host_rows(self.h, layer, request, ctypes.byref(p)),
               "hisparse_host_rows")
        return p.value

    def host_rows(self, layer: int, request: int) -> np.ndarray:
        """Writable numpy view [host_capacity[request]][B] of pinned host rows."""
        n = int(self.cap[request]) * self.B
        buf = (ctypes.c_uint8 * n).from_address(self.host_rows_ptr(layer, request))
        return np.frombuffer(buf, dtype=np.uint8).reshape(int(self.cap[request]), self.B)

    # -- paged host pool ----------------------------------------------------
    def host_reserve(self, requests, num_tokens, stream=None) -> None:
        """Grow the block tables so request requests[i] covers tokens
        [0, num_tokens[i]); raises HiSparseError (code ERR_CAPACITY when the
        pool is short, nothing reserved)."""
        q = np.ascontiguousarray(requests, dtype=np.int32)
        n = np.ascontiguousarray(num_tokens, dtype=np.int64)
        if q.shape != n.shape:
            raise ValueError("requests and num_tokens differ in length")
        _check(self.lib.hisparse_host_reserve(self.h, q.size, q.ctypes.data, n.ctypes.data,
                                              _stream(stream)), "hisparse_host_reserve")

    def host_release(self, requests, stream=None) -> None:
        q = np.ascontiguousarray(requests, dtype=np.int32)
        _check(self.lib.hisparse_host_release(self.h, q.size, q.ctypes.data, _stream(stream)),
               "hisparse_host_release")

    def host_block_table(self, request: int) -> np.ndarray:
        cnt = ctypes.c_int32()
        _check(self.lib.hisparse_host_block_table(self.h, request, None, 0, ctypes.byref(cnt)),
               "hisparse_host_block_table")
        ids = np.empty(max(cnt.value, 1), dtype=np.int32)
        _check(self.lib.hisparse_host_block_table(self.h, request, ids.ctypes.data, cnt.value,
                                                  ctypes.byref(cnt)), "hisparse_host_block_table")
        return ids[: cnt.value].copy()

    def host_pool_info(self):
        """(host_block_tokens, pool_blocks, free_blocks)."""
        v = [ctypes.c_int32() for _ in range(3)]
        _check(self.lib.hisparse_host_pool_info(self.h, *[ctypes.byref(x) for x in v]),
               "hisparse_host_pool_info")
        return tuple(x.value for x in v)

    def host_block_rows(self, layer: int, block: int) -> np.ndarray:
        """Writable numpy view [host_block_tokens][B] of a pinned pool block."""
        p = ctypes.c_void_p()
        _check(self.lib.hisparse_host_block_rows(self.h, layer, block, ctypes.byref(p)),
               "hisparse_host_block_rows")
        buf = (ctypes.c_uint8 * (self.hb * self.B)).from_address(p.value)
        return np.frombuffer(buf, dtype=np.uint8).reshape(self.hb, self.B)

    def write_host_rows(self, layer: int, request: int, t0: int, rows: np.ndarray) -> None:
        """Copy rows ([n][B] uint8) into the pinned host rows of tokens
        [t0, t0 + n) of (layer, request): the request's region, or, with a
        paged pool, the blocks its table names (which must be reserved)."""
        n = rows.shape[0]
        if not self.hb:
            self.host_rows(layer, request)[t0:t0 + n] = rows
            return
        hb = self.hb
        table = self.host_block_table(request)
        t1 = t0 + n
        if n and (t1 - 1) // hb >= table.size:
            raise ValueError("rows beyond the request's reserved host blocks")
        for b in range(t0 // hb, (t1 + hb - 1) // hb):
            a, e = max(b * hb, t0), min((b + 1) * hb, t1)
            self.host_block_rows(layer, int(table[b]))[a - b * hb:e - b * hb] = rows[a - t0:e - t0]

    def device_buffer_ptr(self, layer: int) -> int:
        p = ctypes.c_void_p()
        _check(self.lib.hisparse_device_buffer(self.h, layer, ctypes.byref(p)),
               "hisparse_device_buffer")
        return p.value

    def device_buffer(self, layer: int):
        """torch uint8 CUDA tensor [R][D][B] aliasing the layer's hot buffer."""
        import torch

        class _View:
            __cuda_array_interface__ = {
                "shape": (self.R, self.D, self.B), "typestr": "|u1",
                "data": (self.device_buffer_ptr(layer), False), "version": 3,
                "strides": None}
        return torch.as_tensor(_View(), device="cuda")

    def status_ptr(self) -> int:
        p = ctypes.c_void_p()
        _check(self.lib.hisparse_status(self.h, ctypes.byref(p)), "hisparse_status")
        return p.value

    def status_clear(self, stream=None) -> None:
        """hisparse_status_clear: zero every request's status word (stream-ordered)."""
        _check(self.lib.hisparse_status_clear(self.h, _stream(stream)), "hisparse_status_clear")

    def status(self):
        """torch int32 CUDA tensor [R] aliasing the status words: bit
        STATUS_BIT(code) of entry r is set for every error code request r met
        since the handle was created or the words were last cleared."""
        import torch

        class _View:
            __cuda_array_interface__ = {
                "shape": (self.R,), "typestr": "<i4", "data": (self.status_ptr(), False),
                "version": 3, "strides": None}
        return torch.as_tensor(_View(), device="cuda")

    # -- decode path --------------------------------------------------------
    def prefill(self, seq_lens, stream=None) -> None:
        _check(self.lib.hisparse_prefill(self.h, _addr(seq_lens), _stream(stream)),
               "hisparse_prefill")

    def swap_in(self, layer: int, topk, seq_lens, out_slot_ids, plan_rows=None,
                plan_counts=None, stream=None) -> None:
        plan = None
        if plan_rows is not None or plan_counts is not None:
            plan = ctypes.byref(Plan(_addr(plan_rows), _addr(plan_counts)))
        _check(self.lib.hisparse_swap_in(self.h, layer, _addr(topk), _addr(seq_lens),
                                         _addr(out_slot_ids), plan, _stream(stream)),
               "hisparse_swap_in")

    def swap_in_resident(self, layer: int, topk, seq_lens, resident_blocks, block_size: int,
                         out_slot_ids, plan_rows=None, plan_counts=None, stream=None) -> None:
        """hisparse_swap_in_resident; resident_blocks is a [R][max_blocks]
        int32 device tensor of resident page ids (-1 = not resident)."""
        plan = None
        if plan_rows is not None or plan_counts is not None:
            plan = ctypes.byref(Plan(_addr(plan_rows), _addr(plan_counts)))
        max_blocks = int(resident_blocks.shape[1])
        _check(self.lib.hisparse_swap_in_resident(self.h, layer, _addr(topk), _addr(seq_lens),
                                                  _addr(resident_blocks), max_blocks, block_size,
                                                  _addr(out_slot_ids), plan, _stream(stream)),
               "hisparse_swap_in_resident")

    def swap_in_noalloc(self, layer: int, topk, seq_lens, out_slot_ids, stream=None) -> None:
        """hisparse_swap_in_noalloc: the split-copy swap-in whose internal
        miss plan lives in the library's fixed per-GPU array, so the call
        causes no device allocation (for callers that may not allocate)."""
        _check(self.lib.hisparse_swap_in_noalloc(self.h, layer, _addr(topk), _addr(seq_lens),
                                                 _addr(out_slot_ids), _stream(stream)),
               "hisparse_swap_in_noalloc")

    def replay_plan(self, plan_rows, plan_counts, layer: int, num_ctas: int = 0,
                    stream=None) -> None:
        plan = Plan(_addr(plan_rows), _addr(plan_counts))
        _check(self.lib.hisparse_replay_plan(self.h, ctypes.byref(plan), layer, num_ctas,
                                             _stream(stream)), "hisparse_replay_plan")

    def replay_plan_layers(self, plan_rows, plan_counts, layers, num_ctas: int = 0,
                           stream=None) -> None:
        plan = Plan(_addr(plan_rows), _addr(plan_counts))
        lay = np.ascontiguousarray(layers, dtype=np.int32)
        _check(self.lib.hisparse_replay_plan_layers(self.h, ctypes.byref(plan), lay.ctypes.data,
                                                    len(lay), num_ctas, _stream(stream)),
               "hisparse_replay_plan_layers")

    def backup(self, layer: int, rows, positions, stream=None) -> None:
        _check(self.lib.hisparse_backup(self.h, layer, _addr(rows), _addr(positions),
                                        _stream(stream)), "hisparse_backup")

    def backup_layers(self, layers, rows, positions, stream=None) -> None:
        """hisparse_backup_layers: rows is a [len(layers)][R][B] uint8 device tensor."""
        lay = np.ascontiguousarray(layers, dtype=np.int32)
        _check(self.lib.hisparse_backup_layers(self.h, lay.ctypes.data, len(lay), _addr(rows),
                                               _addr(positions), _stream(stream)),
               "hisparse_backup_layers")

    def write_state(self, layer: int, slot2tok, last_used, ticks, rebuild_rows: bool = True,
                    stream=None) -> None:
        """hisparse_write_state from numpy arrays (slot2tok [R][D] int32,
        last_used [R][D] uint32, ticks [R] uint32)."""
        s2t = np.ascontiguousarray(slot2tok, dtype=np.int32).reshape(self.R, self.D)
        lu = np.ascontiguousarray(last_used, dtype=np.uint32).reshape(self.R, self.D)
        tk = np.ascontiguousarray(ticks, dtype=np.uint32).reshape(self.R)
        _check(self.lib.hisparse_write_state(self.h, layer, s2t.ctypes.data, lu.ctypes.data,
                                             tk.ctypes.data, 1 if rebuild_rows else 0,
                                             _stream(stream)), "hisparse_write_state")

    def check_guards(self) -> int:
        """Overwritten guard bands (handle created with HISPARSE_DEBUG_GUARDS=1)."""
        n = ctypes.c_int32()
        _check(self.lib.hisparse_check_guards(self.h, ctypes.byref(n)), "hisparse_check_guards")
        return n.value

    def set_protected_calls(self, calls: int) -> None:
        """Keep the hot rows of each request's last `calls` calls (0: off)."""
        _check(self.lib.hisparse_set_protected_calls(self.h, calls),
               "hisparse_set_protected_calls")

    def set_stage_rows(self, rows: int) -> None:
        """Miss rows per request the fused copy stages through shared memory
        with the bulk-copy engine (0: none, the default; -1: as many as fit)."""
        _check(self.lib.hisparse_set_stage_rows(self.h, rows), "hisparse_set_stage_rows")

    def set_copy_ctas(self, ctas: int) -> None:
        """CTAs per request of a fused-copy swap-in: 1 resolves and copies in
        one CTA; 2-4 form a cluster whose rank 0 resolves and whose other
        CTAs copy (hisparse_set_copy_ctas)."""
        _check(self.lib.hisparse_set_copy_ctas(self.h, ctas), "hisparse_set_copy_ctas")

    def copy_ctas(self) -> int:
        """CTAs per request that fused-copy swap-ins use now."""
        v = ctypes.c_int32(0)
        _check(self.lib.hisparse_get_copy_ctas(self.h, ctypes.byref(v)), "hisparse_get_copy_ctas")
        return int(v.value)

    def set_programmatic_launch(self, on: bool) -> None:
        """Launch swap-ins and backups with a programmatic dependency on the
        stream's previous kernel (off by default)."""
        _check(self.lib.hisparse_set_programmatic_launch(self.h, 1 if on else 0),
               "hisparse_set_programmatic_launch")

    # -- 4-bit rows ---------------------------------------------------------
    def attend(self, layer: int, q, slot_ids, out, scale: float, lse=None, positions=None,
               weights=None, resident_rows=None, workspace=None, stream=None) -> None:
        """attend() over the layer's hot buffer (row_bytes must be
        ROW4_BYTES); data errors go to this handle's status words.
        INVALID_ARG unless the handle's device is current."""
        if self.B != ROW4_BYTES:
            raise ValueError(f"row_bytes is {self.B}: attention reads {ROW4_BYTES}-byte rows")
        if _current_device() != self.device:
            raise HiSparseError(ERR_INVALID_ARG, f"attend of a handle of device {self.device}")
        _attend(q, None, self.device_buffer_ptr(layer), self.B, self.D * self.B, self.R, self.D,
                slot_ids, out, scale, lse, positions, weights, resident_rows, self.status_ptr(),
                workspace, stream)

    def evict(self, layer: int, weights, seq_lens, n: int, keep_recent: int = 0, want=None,
              out_slots=None, out_counts=None, stream=None) -> None:
        """hisparse_evict: free, per request, up to n (or want[r]) hot slots
        of the least accumulated weight (weights: float32 [R][tokens])."""
        tokens, stride = _rows_of(weights, "weights", "float32", self.R)
        _ints(seq_lens, "seq_lens", (self.R,))
        _ints(want, "want", (self.R,))
        _ints(out_slots, "out_slots", (self.R, n))
        _ints(out_counts, "out_counts", (self.R,))
        _check(self.lib.hisparse_evict(self.h, layer, _addr(weights), stride,
                                       tokens, _addr(seq_lens), keep_recent, n,
                                       _addr(want), _addr(out_slots), _addr(out_counts),
                                       _stream(stream)), "hisparse_evict")

    def set_copy_mode(self, mode: int) -> None:
        _check(self.lib.hisparse_set_copy_mode(self.h, mode), "hisparse_set_copy_mode")

    def read_state(self, layer: int, stream=None):
        """(slot2tok [R][D], last_used [R][D], tok2slot [total_cap], lru [R][D], ticks [R])."""
        s2t = np.empty((self.R, self.D), dtype=np.int32)
        lu = np.empty((self.R, self.D), dtype=np.uint32)
        t2s = np.empty(self.total_cap, dtype=np.int32)
        lru = np.empty((self.R, self.D), dtype=np.int32)
        ticks = np.empty(self.R, dtype=np.uint32)
        _check(self.lib.hisparse_read_state(self.h, layer, s2t.ctypes.data, lu.ctypes.data,
                                            t2s.ctypes.data, lru.ctypes.data, ticks.ctypes.data,
                                            _stream(stream)), "hisparse_read_state")
        return s2t, lu, t2s, lru, ticks


# -- 4-bit rows (include/hisparse_rows4.h) ----------------------------------

def _dtype16(x, what: str) -> int:
    t = _torch or _load_torch()
    if x.dtype is t.bfloat16:
        return BF16
    if x.dtype is t.float16:
        return F16
    raise ValueError(f"{what} must be bfloat16 or float16, not {x.dtype}")


def _rows_of(x, what: str, dtype: str, n: int):
    """Columns and row stride of x, which is [n][...] of dtype with contiguous
    rows (a single row has no stride to go by)."""
    shape = x.shape
    if x.dtype is getattr(_torch or _load_torch(), dtype) and len(shape) == 2 and shape[0] == n:
        stride, one = x.stride()
        if one == 1 or shape[1] <= 1:
            return shape[1], stride if n > 1 else shape[1]
    raise ValueError(f"{what} must be {dtype} [{n}][...] with contiguous rows")


def _ints(x, what: str, shape) -> None:
    """x is None or a contiguous int32 tensor of this shape."""
    if x is not None and (x.dtype is not (_torch or _load_torch()).int32 or x.shape != shape
                          or not x.is_contiguous()):
        raise ValueError(f"{what} must be a contiguous int32 tensor of shape {shape}")


def _words(status, R: int) -> int:
    """Address of status: None, an address, or a contiguous int32 tensor [R]."""
    if status is None or isinstance(status, int):
        return status or 0
    _ints(status, "status", (R,))
    return status.data_ptr()


def _packed(rows, what: str, dims: int):
    """Shape and strides of packed rows."""
    shape, strides = rows.shape, rows.stride()
    if (rows.dtype is not (_torch or _load_torch()).uint8 or len(shape) != dims
            or shape[-1] != ROW4_BYTES or strides[-1] != 1):
        raise ValueError(f"{what} must be uint8 [...][{ROW4_BYTES}] with contiguous rows")
    return shape, strides


def _pack_args(values, rows):
    dt = _dtype16(values, "values")
    shape, strides = values.shape, values.stride()
    if len(shape) != 2 or shape[1] != ROW4_VALUES or strides[1] != 1:
        raise ValueError(f"values must be [n][{ROW4_VALUES}] with contiguous rows")
    row_shape, row_strides = _packed(rows, "rows", 2)
    n = shape[0]
    if row_shape[0] != n:
        raise ValueError("values and rows differ in length")
    return (dt, n, strides[0], row_strides[0]) if n > 1 else (dt, n, ROW4_VALUES, ROW4_BYTES)


def pack_rows(values, rows, stream=None) -> None:
    """rows (uint8 [n][416], device or pinned) <- values (bf16 or f16
    [n][576]: 512 latent and 64 rope values) in 4 bits."""
    dt, n, vs, rs = _pack_args(values, rows)
    _check((_lib or load_library()).hisparse_pack_rows(values.data_ptr(), vs, dt, n,
                                                       rows.data_ptr(), rs, _stream(stream)),
           "hisparse_pack_rows")


def unpack_rows(rows, values, stream=None) -> None:
    """values (bf16 or f16 [n][576]) <- what rows (uint8 [n][416]) stand for."""
    dt, n, vs, rs = _pack_args(values, rows)
    _check((_lib or load_library()).hisparse_unpack_rows(rows.data_ptr(), rs, n, values.data_ptr(),
                                                         vs, dt, _stream(stream)),
           "hisparse_unpack_rows")


def _allocate(size: int, device, stream, handle: int):
    """uint8 tensor for work on `stream` (None, a Stream or an address;
    handle: its address) that may be dropped once that work is launched: its
    memory is the allocator's for that stream, so what gets it next runs
    behind the work."""
    t = _torch
    if stream is None:
        return t.empty(size, dtype=t.uint8, device=device)
    if not isinstance(stream, t.cuda.Stream):
        stream = t.cuda.ExternalStream(handle, device=device)
    with t.cuda.stream(stream):
        return t.empty(size, dtype=t.uint8, device=device)


def attend_workspace_bytes(num_requests: int, num_heads: int, top_k: int,
                           weights: bool = False) -> int:
    """Bytes of workspace that attend() needs for these sizes."""
    n = ctypes.c_int64()
    _check(load_library().hisparse_attend_workspace(num_requests, num_heads, top_k,
                                                    1 if weights else 0, ctypes.byref(n)),
           "hisparse_attend_workspace")
    return n.value


def attend(q, rows, slot_ids, out, scale: float, lse=None, positions=None, weights=None,
           resident_rows=None, status=None, workspace=None, stream=None) -> None:
    """hisparse_attend: one step's sparse attention over 4-bit rows, on the
    current device.

    q [R][H][576] and out [R][H][512] in bf16 or f16; rows uint8 [R][D][416];
    slot_ids int32 [R][k] as swap_in writes them; lse float32 [R][H] or None;
    weights float32 [R][tokens] (accumulated into at positions, int32 [R][k])
    or None; resident_rows uint8 [n][416] for flagged ids; status int32 [R]
    or None; workspace a uint8 tensor of attend_workspace_bytes (None:
    allocated for this call, on its stream).  All of them on that device;
    slot_ids and positions also in pinned host memory."""
    (R, D, _), (request_stride, row_stride, _) = _packed(rows, "rows", 3)
    _attend(q, rows, rows.data_ptr(), row_stride if D > 1 else ROW4_BYTES,
            request_stride if R > 1 else 0, R, D, slot_ids, out, scale, lse, positions, weights,
            resident_rows, status, workspace, stream)


def _attend(q, rows, rows_at, row_stride, request_stride, R, D, slot_ids, out, scale, lse, positions,
            weights, resident_rows, status, workspace, stream) -> None:
    dt = _dtype16(q, "q")
    shape, strides = q.shape, q.stride()
    if len(shape) != 3 or shape[0] != R or shape[2] != ROW4_VALUES or strides[2] != 1:
        raise ValueError(f"q must be [{R}][H][{ROW4_VALUES}] with contiguous heads")
    H = shape[1]
    out_strides = out.stride()
    if out.dtype is not q.dtype or out.shape != (R, H, ROW4_LATENT) or out_strides[2] != 1:
        raise ValueError(f"out must be [{R}][{H}][{ROW4_LATENT}] of q's type with contiguous heads")
    k, ids_stride = _rows_of(slot_ids, "slot_ids", "int32", R)
    if lse is not None and (lse.dtype is not _torch.float32 or lse.shape != (R, H)
                            or not lse.is_contiguous()):
        raise ValueError(f"lse must be a contiguous float32 tensor of shape ({R}, {H})")
    resident = (0, 0, 0)
    if resident_rows is not None:
        (count, _), (stride, _) = _packed(resident_rows, "resident_rows", 2)
        resident = (resident_rows.data_ptr(), stride if count > 1 else ROW4_BYTES, count)
    acc, where = (0, 0, 0), (0, 0)
    if weights is not None:
        tokens, stride = _rows_of(weights, "weights", "float32", R)
        if positions is None:
            raise ValueError("weights need positions")
        columns, positions_stride = _rows_of(positions, "positions", "int32", R)
        if columns != k:
            raise ValueError("positions and slot_ids differ in length")
        acc, where = (weights.data_ptr(), stride, tokens), (positions.data_ptr(), positions_stride)
    words = _words(status, R)
    device = _current_device()
    if (q.get_device() != device or out.get_device() != device
            or rows is not None and rows.get_device() != device
            or lse is not None and lse.get_device() != device
            or weights is not None and weights.get_device() != device
            or resident_rows is not None and resident_rows.get_device() != device
            or workspace is not None and workspace.get_device() != device
            or words and status is not words and status.get_device() != device):
        raise ValueError(f"only slot_ids and positions may be outside the current device, {device}")
    if (slot_ids.get_device() not in (device, -1)
            or positions is not None and positions.get_device() not in (device, -1)):
        raise ValueError(f"slot_ids and positions must be on device {device} or pinned")
    launch_stream = _stream(stream)
    if workspace is None:
        workspace = _allocate(attend_workspace_bytes(R, H, k, weights is not None), q.device,
                              stream, launch_stream)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    args = _pack_attend_args(
        R, H, k, dt, q.data_ptr(), strides[0], strides[1], rows_at, row_stride, request_stride, D, scale,
        slot_ids.data_ptr(), ids_stride, *resident, out.data_ptr(), out_strides[0], out_strides[1],
        0 if lse is None else lse.data_ptr(), *acc, *where, words, workspace.data_ptr(),
        workspace.nbytes)
    _check((_lib or load_library()).hisparse_attend(args, launch_stream), "hisparse_attend")


def evict_select(weights, slot2tok, seq_lens, out_slots, out_counts, keep_recent: int = 0,
                 want=None, stream=None) -> None:
    """hisparse_evict_select: the slots of the least accumulated weight
    (out_slots int32 [R][n], ascending, -1 behind them; out_counts int32 [R])
    of slot2tok int32 [R][D]; weights float32 [R][tokens]."""
    R, D = slot2tok.shape
    tokens, stride = _rows_of(weights, "weights", "float32", R)
    _ints(slot2tok, "slot2tok", (R, D))
    _ints(seq_lens, "seq_lens", (R,))
    n = out_slots.shape[1]
    _ints(out_slots, "out_slots", (R, n))
    _ints(out_counts, "out_counts", (R,))
    _ints(want, "want", (R,))
    _check((_lib or load_library()).hisparse_evict_select(
        R, D, weights.data_ptr(), stride, tokens, slot2tok.data_ptr(),
        seq_lens.data_ptr(), keep_recent, n, _addr(want), out_slots.data_ptr(),
        out_counts.data_ptr(), _stream(stream)), "hisparse_evict_select")


# -- resident pages (include/hisparse_pages.h) ------------------------------

def _reachable(x, device: int, what: str) -> None:
    """x (None: not there) is on the current device or in pinned memory."""
    if x is not None and x.get_device() != device and not (x.get_device() == -1 and x.is_pinned()):
        raise ValueError(f"{what} is neither on the current device, {device}, nor pinned")


def _line(x, what: str) -> int:
    """Length of x, a contiguous int32 tensor of one dimension."""
    shape = x.shape
    if x.dtype is not (_torch or _load_torch()).int32 or len(shape) != 1 or not x.is_contiguous():
        raise ValueError(f"{what} must be a contiguous int32 tensor of one dimension")
    return shape[0]


def page_tables(lens, tables, held, free_list, free_count, block_size: int, shared=None,
                new_tokens=None, offsets=None, slots=None, positions=None, status=None,
                stream=None) -> None:
    """hisparse_page_tables: brings the block tables (int32 [R][blocks], held
    int32 [R] entries of each in use) to the lengths lens (int32 [R]; negative:
    left alone), with free pages from and back to free_list (int32 [pages],
    free_count int32 [1]); shared: int32 page ids of a common prefix.  With
    new_tokens (int32 [R]) also offsets (int32 [R + 1]), slots and positions
    (int32 [tokens]; positions may be None) of the last new_tokens[r] tokens of
    each request.  status int32 [R] or None.  On the current device; lens,
    new_tokens and shared also in pinned host memory."""
    R = _line(lens, "lens")
    blocks, stride = _rows_of(tables, "tables", "int32", R)
    if _line(held, "held") != R or _line(free_count, "free_count") != 1:
        raise ValueError(f"held must have {R} entries and free_count one")
    capacity = _line(free_list, "free_list")
    prefix = tokens = 0
    prefix_at = new_at = offsets_at = slots_at = positions_at = 0
    device = _current_device()
    here = (tables.get_device() == device and held.get_device() == device and free_list.get_device() == device
            and free_count.get_device() == device)
    _reachable(lens, device, "lens")
    if shared is not None:
        prefix, prefix_at = _line(shared, "shared"), shared.data_ptr()
        _reachable(shared, device, "shared")
    if new_tokens is not None:
        if offsets is None or slots is None:
            raise ValueError("new_tokens need offsets and slots")
        tokens = _line(slots, "slots")
        if _line(new_tokens, "new_tokens") != R or _line(offsets, "offsets") != R + 1:
            raise ValueError(f"new_tokens must have {R} entries and offsets {R + 1}")
        new_at, offsets_at, slots_at = new_tokens.data_ptr(), offsets.data_ptr(), slots.data_ptr()
        _reachable(new_tokens, device, "new_tokens")
        here = here and offsets.get_device() == device and slots.get_device() == device
        if positions is not None:
            if _line(positions, "positions") != tokens:
                raise ValueError("positions and slots differ in length")
            positions_at = positions.data_ptr()
            here = here and positions.get_device() == device
    elif offsets is not None or slots is not None or positions is not None:
        raise ValueError("offsets, slots and positions need new_tokens")
    words = _words(status, R)
    if not here or words and status is not words and status.get_device() != device:
        raise ValueError(f"only lens, new_tokens and shared may be outside the current device, {device}")
    _check((_lib or load_library()).hisparse_page_tables(_pack_page_tables_args(
        R, blocks, block_size, prefix, lens.data_ptr(), tables.data_ptr(), stride, held.data_ptr(),
        free_list.data_ptr(), capacity, free_count.data_ptr(), prefix_at, new_at, offsets_at, slots_at,
        positions_at, tokens, words), _stream(stream)), "hisparse_page_tables")


def _format_rows(rows, what: str):
    """Count, stride and format of rows, uint8 [count][416, 656 or 1152]."""
    shape = rows.shape
    if rows.dtype is (_torch or _load_torch()).uint8 and len(shape) == 2 and shape[1] in (
            ROW4_BYTES, ROW8_BYTES, ROW16_BYTES):
        stride, one = rows.stride()
        if one == 1:
            return shape[0], stride if shape[0] > 1 else shape[1], shape[1]
    raise ValueError(f"{what} must be uint8 [...][{ROW4_BYTES}, {ROW8_BYTES} or {ROW16_BYTES}] with contiguous rows")


def _row_values(values, rows, slots):
    dt = _dtype16(values, "values")
    shape, strides = values.shape, values.stride()
    if len(shape) != 2 or shape[1] != ROW4_VALUES or strides[1] != 1:
        raise ValueError(f"values must be [n][{ROW4_VALUES}] with contiguous rows")
    n = shape[0]
    count, stride, row_bytes = _format_rows(rows, "rows")
    if slots is not None:
        if _line(slots, "slots") != n:
            raise ValueError(f"slots must have {n} entries")
    elif count < n:
        raise ValueError("more values than rows")
    device = _current_device()
    _reachable(values, device, "values")
    _reachable(rows, device, "rows")
    _reachable(slots, device, "slots")
    return dt, n, strides[0] if n > 1 else ROW4_VALUES, count, stride, row_bytes


def norm_rows(values, rows, slots=None, weight=None, eps: float = 1e-6, stream=None) -> None:
    """hisparse_norm_rows: rows[slots[i]] (uint8 [count][416, 656 or 1152]) <-
    values[i] (bf16 or f16 [n][576]), the 512 latent values divided by their root
    mean square and times weight ([512] of that type; None: stored as they are),
    in the rows' format.  slots int32 [n] (negative: not stored) or None: row i.
    On the current device or in pinned host memory."""
    dt, n, vs, count, rs, row_bytes = _row_values(values, rows, slots)
    weight_at = None
    if weight is not None:
        if weight.dtype is not values.dtype or weight.shape != (ROW4_LATENT,) or not weight.is_contiguous():
            raise ValueError(f"weight must be a contiguous [{ROW4_LATENT}] of the values' type")
        _reachable(weight, _current_device(), "weight")
        weight_at = weight.data_ptr()
    _check((_lib or load_library()).hisparse_norm_rows(
        values.data_ptr(), vs, dt, n, weight_at, eps, rows.data_ptr(), rs, row_bytes, count,
        None if slots is None else slots.data_ptr(), _stream(stream)), "hisparse_norm_rows")


def gather_rows(rows, values, slots=None, stream=None) -> None:
    """hisparse_gather_rows: values[i] (bf16 or f16 [n][576]) <- what
    rows[slots[i]] stands for; arguments as norm_rows()."""
    dt, n, vs, count, rs, row_bytes = _row_values(values, rows, slots)
    _check((_lib or load_library()).hisparse_gather_rows(
        rows.data_ptr(), rs, row_bytes, count, None if slots is None else slots.data_ptr(), n,
        values.data_ptr(), vs, dt, _stream(stream)), "hisparse_gather_rows")


def _sums(x, what: str, R: int, H: int) -> None:
    if x.dtype is not _torch.float32 or x.shape != (R, H) or not x.is_contiguous():
        raise ValueError(f"{what} must be a contiguous float32 tensor of shape ({R}, {H})")


def attend_prefix_workspace_bytes(num_requests: int, num_heads: int, prefix_len: int) -> int:
    """Bytes of workspace that attend_prefix() needs for these sizes."""
    n = ctypes.c_int64()
    _check(load_library().hisparse_attend_prefix_workspace(num_requests, num_heads, prefix_len,
                                                           ctypes.byref(n)),
           "hisparse_attend_prefix_workspace")
    return n.value


def attend_prefix(q, rows, table, block_size: int, prefix_len: int, out, scale: float, lse=None,
                  part=None, part_lse=None, status=None, workspace=None, stream=None) -> None:
    """hisparse_attend_prefix: attention of all requests over the prefix_len
    tokens whose pages table (int32 [blocks]) names, joined with `part`.

    q [R][H][576], out and part (or None) [R][H][512] in bf16 or f16; rows uint8
    [count][416, 656 or 1152], the pool of pages of block_size rows; lse and
    part_lse float32 [R][H] (lse may be None, part_lse goes with part; part and
    part_lse may be out and lse); status int32 [R] or None; workspace a uint8
    tensor of attend_prefix_workspace_bytes (None: allocated for this call, on
    its stream).  All of them on the current device, table also in pinned host
    memory."""
    dt = _dtype16(q, "q")
    shape, strides = q.shape, q.stride()
    if len(shape) != 3 or shape[2] != ROW4_VALUES or strides[2] != 1:
        raise ValueError(f"q must be [R][H][{ROW4_VALUES}] with contiguous heads")
    R, H = shape[0], shape[1]
    out_strides = out.stride()
    if out.dtype is not q.dtype or out.shape != (R, H, ROW4_LATENT) or out_strides[2] != 1:
        raise ValueError(f"out must be [{R}][{H}][{ROW4_LATENT}] of q's type with contiguous heads")
    count, row_stride, row_bytes = _format_rows(rows, "rows")
    if block_size < 1 or _line(table, "table") * block_size < prefix_len:
        raise ValueError(f"table names fewer than {prefix_len} tokens")
    words = _words(status, R)
    device = _current_device()
    here = q.get_device() == device and rows.get_device() == device and out.get_device() == device
    lse_at = part_at = part_lse_at = 0
    part_strides = (0, 0)
    if lse is not None:
        _sums(lse, "lse", R, H)
        lse_at = lse.data_ptr()
        here = here and lse.get_device() == device
    if part is not None:
        part_strides = part.stride()
        if part.dtype is not q.dtype or part.shape != (R, H, ROW4_LATENT) or part_strides[2] != 1:
            raise ValueError(f"part must be [{R}][{H}][{ROW4_LATENT}] of q's type with contiguous heads")
        if part_lse is None:
            raise ValueError("part needs part_lse")
        _sums(part_lse, "part_lse", R, H)
        part_at, part_lse_at = part.data_ptr(), part_lse.data_ptr()
        here = here and part.get_device() == device and part_lse.get_device() == device
    elif part_lse is not None:
        raise ValueError("part_lse needs part")
    if (not here or workspace is not None and workspace.get_device() != device
            or words and status is not words and status.get_device() != device):
        raise ValueError(f"only table may be outside the current device, {device}")
    _reachable(table, device, "table")
    launch_stream = _stream(stream)
    if workspace is None:
        workspace = _allocate(attend_prefix_workspace_bytes(R, H, prefix_len), q.device, stream, launch_stream)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _check((_lib or load_library()).hisparse_attend_prefix(_pack_attend_prefix_args(
        R, H, dt, row_bytes, q.data_ptr(), strides[0], strides[1], rows.data_ptr(), row_stride, count,
        table.data_ptr(), block_size, prefix_len, scale, part_at, part_strides[0], part_strides[1], part_lse_at,
        out.data_ptr(), out_strides[0], out_strides[1], lse_at, words, workspace.data_ptr(),
        workspace.nbytes), launch_stream), "hisparse_attend_prefix")


# -- measurement kernels (include/hisparse_measure.h) -----------------------

def synthetic_compute(buf, passes: int, ctas_per_sm: int = 2, stream=None) -> None:
    """The memory-bound bf16 stand-in compute over torch tensor `buf`."""
    lib = load_library()
    _check(lib.hisparse_synthetic_compute(_addr(buf), buf.numel() * buf.element_size(), passes,
                                          ctas_per_sm, _stream(stream)),
           "hisparse_synthetic_compute")


def link_gather(src, row_bytes: int, rows, dst, num_ctas: int = 0, stream=None) -> None:
    """hisparse_link_gather: dst row i <- src row rows[i] (rows: device int64
    tensor, every entry in range -- the kernel does not check)."""
    lib = load_library()
    _check(lib.hisparse_link_gather(_addr(src), row_bytes, _addr(rows), int(rows.numel()),
                                    _addr(dst), num_ctas, _stream(stream)),
           "hisparse_link_gather")


def link_probe(src, dst, nbytes: int, num_ctas: int = 0, stream=None) -> None:
    lib = load_library()
    _check(lib.hisparse_link_probe(_addr(src), _addr(dst), nbytes, num_ctas, _stream(stream)),
           "hisparse_link_probe")
