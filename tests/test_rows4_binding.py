"""What the binding of the 4-bit row calls does before a launch, with the GPU's
part played by fakes (CPU only): the library's calls are recorded instead of
made, and torch's allocator and streams by what they were asked for."""

import ctypes
import types

import pytest
import torch

from hierarchical_sparse_kv_request_gb300 import build as B
from hierarchical_sparse_kv_request_gb300 import hisparse as H

R, HEADS, K, D, TOKENS = 2, 3, 5, 8, 20


@pytest.fixture(scope="module")
def lib():
    B.build_library()
    return H.load_library()


class Stream:
    """Stands for torch.cuda.Stream."""

    def __init__(self, address):
        self.cuda_stream = address


class Gpu:
    """torch as the binding sees it: `empty` notes the stream that is current
    while it allocates; and the library: hisparse_attend notes its stream."""

    def __init__(self, lib):
        self.now, self.allocations, self.launches = Stream(0x111), [], []
        gpu = self

        class scope:
            def __init__(self, s):
                self.s = s

            def __enter__(self):
                self.s, gpu.now = gpu.now, self.s

            def __exit__(self, *e):
                gpu.now = self.s

        def empty(size, dtype, device):
            gpu.allocations.append((gpu.now.cuda_stream, size))
            return torch.empty(size, dtype=dtype, device=device)

        self.torch = types.SimpleNamespace(
            bfloat16=torch.bfloat16, float16=torch.float16, float32=torch.float32, int32=torch.int32,
            uint8=torch.uint8, empty=empty,
            cuda=types.SimpleNamespace(Stream=Stream, stream=scope, current_stream=lambda: gpu.now,
                                       ExternalStream=lambda a, device: Stream(a)))
        self.lib = types.SimpleNamespace(hisparse_attend=self.launch, hisparse_destroy=lambda h: H.OK,
                                         hisparse_error_string=lib.hisparse_error_string,
                                         hisparse_attend_workspace=lib.hisparse_attend_workspace)

    def launch(self, args, stream):
        self.launches.append(stream)
        return H.OK


@pytest.fixture
def gpu(lib, monkeypatch):
    g = Gpu(lib)
    monkeypatch.setattr(H, "_torch", g.torch)
    monkeypatch.setattr(H, "_lib", g.lib)
    monkeypatch.setattr(H, "_raw_stream", lambda device: g.now.cuda_stream)
    monkeypatch.setattr(H, "_device", lambda: -1)     # the tensors' (the CPU's) number
    return g


def tensors():
    t = dict(q=torch.zeros((R, HEADS, 576), dtype=torch.bfloat16),
             rows=torch.zeros((R, D, 416), dtype=torch.uint8),
             slot_ids=torch.zeros((R, K), dtype=torch.int32),
             out=torch.zeros((R, HEADS, 512), dtype=torch.bfloat16))
    more = dict(weights=torch.zeros((R, TOKENS)), positions=torch.zeros((R, K), dtype=torch.int32))
    return t, more


@pytest.mark.parametrize("stream,address", [(None, 0x111), (Stream(0x222), 0x222), (0x333, 0x333), (0, 0)])
@pytest.mark.parametrize("weights", [False, True])
def test_a_workspace_of_the_call_belongs_to_the_launch_stream(gpu, stream, address, weights):
    """Freed when the call returns, its memory may go only to work that the
    launch stream runs behind the call's own."""
    t, more = tensors()
    H.attend(**t, scale=1.0, **(more if weights else {}), stream=stream)
    assert gpu.launches == [address]
    assert gpu.allocations == [(address, H.attend_workspace_bytes(R, HEADS, K, weights))]
    assert gpu.now.cuda_stream == 0x111      # the current stream is as it was


def handle(gpu, device):
    """A handle of this device, without the library's side of one."""
    h = object.__new__(H.HiSparse)
    h.lib, h.h, h.device = gpu.lib, None, device
    h.R, h.D, h.B = R, D, H.ROW4_BYTES
    h.device_buffer_ptr, h.status_ptr = lambda layer: 1 << 20, lambda: 1 << 21
    return h


def test_a_handle_refuses_to_attend_on_another_device(gpu):
    """As its other launching calls do."""
    t, _ = tensors()
    del t["rows"]
    handle(gpu, -1).attend(0, **t, scale=1.0)
    assert len(gpu.launches) == 1
    with pytest.raises(H.HiSparseError) as e:
        handle(gpu, 1).attend(0, **t, scale=1.0)
    assert e.value.code == H.ERR_INVALID_ARG
    assert len(gpu.launches) == 1 and len(gpu.allocations) == 1


@pytest.mark.parametrize("status", [
    torch.zeros(R - 1, dtype=torch.int32), torch.zeros(R + 1, dtype=torch.int32), torch.zeros((R, 1), dtype=torch.int32),
    torch.zeros(R, dtype=torch.int64), torch.zeros(R), torch.zeros(2 * R, dtype=torch.int32)[::2]])
def test_attend_refuses_status_words_of_another_shape_or_type(gpu, status):
    """A word past the end would be written at the first bad id there."""
    t, _ = tensors()
    with pytest.raises(ValueError):
        H.attend(**t, scale=1.0, status=status)
    assert gpu.launches == []
    for good in (torch.zeros(R, dtype=torch.int32), 1 << 20, None):
        H.attend(**t, scale=1.0, status=good)
    assert len(gpu.launches) == 3


def test_attend_refuses_a_workspace_that_is_not_contiguous(gpu):
    """Its size says nothing about the memory that it has."""
    t, _ = tensors()
    size = H.attend_workspace_bytes(R, HEADS, K)
    one = torch.zeros(16, dtype=torch.uint8)
    for bad in (one[:1].expand(size), torch.zeros(2 * size, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError):
            H.attend(**t, scale=1.0, workspace=bad)
    assert gpu.launches == []
    H.attend(**t, scale=1.0, workspace=torch.zeros(size // 4, dtype=torch.int32))
    assert len(gpu.launches) == 1


class Elsewhere(torch.Tensor):
    """A tensor of another GPU."""

    def get_device(self):
        return 1


@pytest.mark.parametrize("name", ["q", "rows", "slot_ids", "out", "lse", "positions", "weights", "resident_rows",
                                  "status", "workspace"])
def test_attend_refuses_tensors_of_another_device(gpu, name):
    t, more = tensors()
    t.update(more, lse=torch.zeros((R, HEADS)), resident_rows=torch.zeros((4, 416), dtype=torch.uint8),
             status=torch.zeros(R, dtype=torch.int32),
             workspace=torch.zeros(H.attend_workspace_bytes(R, HEADS, K, True), dtype=torch.uint8))
    H.attend(**t, scale=1.0)
    assert len(gpu.launches) == 1
    t[name] = t[name].as_subclass(Elsewhere)
    with pytest.raises(ValueError):
        H.attend(**t, scale=1.0)
    if name != "rows":
        del t["rows"], t["status"]
        if name != "status":
            with pytest.raises(ValueError):
                handle(gpu, -1).attend(0, **t, scale=1.0)
    assert len(gpu.launches) == 1


def test_only_ids_and_positions_may_be_host_tensors(gpu, monkeypatch):
    t, more = tensors()
    t.update(more)
    monkeypatch.setattr(H, "_device", lambda: 1)       # now the CPU's tensors are the host's
    with pytest.raises(ValueError):
        H.attend(**t, scale=1.0)
    for name in ("q", "rows", "out", "weights"):
        t[name] = t[name].as_subclass(Elsewhere)
    H.attend(**t, scale=1.0, workspace=torch.zeros(1 << 16, dtype=torch.uint8).as_subclass(Elsewhere))
    assert len(gpu.launches) == 1


def test_a_handle_is_made_without_torch(monkeypatch):
    """Its device is the library's to say; torch is loaded by calls that need it."""
    def get_device(h, device):
        device._obj.value = 3
        return H.OK

    def load():
        raise AssertionError("torch is not needed here")

    monkeypatch.setattr(H, "_torch", None)
    monkeypatch.setattr(H, "_device", None)
    monkeypatch.setattr(H, "_load_torch", load)
    monkeypatch.setattr(H, "_lib", types.SimpleNamespace(hisparse_create=lambda layout, h: H.OK,
                                                         hisparse_get_device=get_device))
    assert H.HiSparse(2, 1, H.ROW4_BYTES, 4, 8, 1, [16, 16]).device == 3


def test_get_device_refuses_null(lib):
    assert lib.hisparse_get_device(None, ctypes.byref(ctypes.c_int32())) == H.ERR_INVALID_ARG
