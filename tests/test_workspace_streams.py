"""A workspace that the binding allocates comes out of the memory of the stream that the call launches on.

The caching allocator hands a freed block on in the order of its own stream only.  A block of the current stream's,
used on another one, could still be read or written there by what had it before.
"""
import contextlib

import numpy as np
import pytest
import torch

from gated_deltanet_recurrence_gdn_amd import binding as gb


class Stream:
    cuda_stream, device_index = 0x1230, 0


@pytest.fixture
def allocations(monkeypatch):
    """(stream made current, bytes) of every torch.empty, on the host: streams are only recorded."""
    current, got, empty = [None], [], torch.empty

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    def record(*a, **kw):
        t = empty(*a, **kw)
        got.append((current[-1], t.numel()))
        return t

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: ("external", handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    monkeypatch.setattr(torch, "empty", record)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None)
    return got


def test_the_workspace_is_allocated_on_the_launching_stream(allocations):
    s, cpu = Stream(), torch.device("cpu")
    gb._workspace(100, cpu, s)
    gb._workspace(0, cpu, 0x55)
    gb._workspace(7, cpu, None)
    assert allocations == [(s, 100), (("external", 0x55), 16), (None, 16)]


CU = np.array([0, 2, 6], np.int32)


def scan_args(device, tape=None):
    z = lambda *n, t=torch.float32: torch.zeros(*n, dtype=t, device=device)  # noqa: E731
    return [z(6, 2, 32), z(6, 2, 32), z(6, 4, 16), z(6, 4), z(6, 4)]


def call(name, device, **kw):
    """One call of an entry point that allocates its workspace, of the smallest sizes."""
    x = scan_args(device)
    out = torch.zeros_like(x[2])
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device=device)  # noqa: E731
    pool = torch.zeros(2, 4, 8, device=device)
    if name.startswith("prefill"):
        state = torch.zeros(2, 4, 32, 32, device=device)
        v = torch.zeros(6, 4, 32, device=device)
        if name == "prefill_varlen":
            return gb.gdn_prefill_varlen(CU, x[0], x[1], v, x[3], x[4], state, torch.zeros_like(v), **kw)
        b = [t.view(2, 3, *t.shape[1:]) for t in (x[0], x[1], v, x[3], x[4])]
        return gb.gdn_prefill_chunked(*b, state, torch.zeros_like(b[2]), **kw)
    if name == "scan_forward":
        return gb.gdn_scan_forward(CU, *x, out, **kw)
    if name == "scan_backward":
        tape = torch.zeros(gb.gdn_scan_tape_bytes(CU, x[0], x[2]), dtype=torch.uint8, device=device)
        return gb.gdn_scan_backward(CU, *x, tape, out, *[torch.zeros_like(t) for t in x], **kw)
    if name == "pool_fork":
        return gb.gdn_pool_fork(pool, ints(2, -1), ints(0), ints(1), **kw)
    return gb.gdn_pool_compact(pool, ints(2, -1), **kw)


@pytest.mark.parametrize("name", ["scan_forward", "scan_backward", "prefill_chunked", "prefill_varlen"])
def test_entry_points_on_the_host(name, allocations):
    s = Stream()
    with pytest.raises(TypeError, match="device tensor"):
        call(name, "cpu", stream=s)
    assert [a for a in allocations if a[0] is not None] == [(s, allocations[-1][1])]


def segment_stream(t):
    """The stream whose memory a tensor's block is part of."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("no such segment")


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", ["scan_forward", "scan_backward", "pool_fork", "pool_compact",
                                  "prefill_chunked", "prefill_varlen"])
def test_entry_points_on_the_gpu(name, handle):
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    prepared = call(name, "cuda:0", stream=side.cuda_stream if handle else side, prepare=True)
    workspace = [t for t in prepared._keep if isinstance(t, torch.Tensor) and t.dtype == torch.uint8][-1]
    assert segment_stream(workspace) == side.cuda_stream
    assert segment_stream(torch.empty(64, device="cuda:0")) == torch.cuda.current_stream().cuda_stream
    side.wait_stream(torch.cuda.current_stream())  # the inputs were made on the current stream
    prepared()
    torch.cuda.synchronize()


def test_the_handle_of_the_default_stream(allocations):
    """torch takes a handle of 0 for no handle at all: an ExternalStream of it is some other stream."""
    gb._workspace(7, torch.device("cpu"), 0)
    assert allocations == [("default", 16)]


@pytest.mark.gpu
def test_the_handle_of_the_default_stream_on_the_gpu():
    with torch.cuda.stream(torch.cuda.Stream()):
        workspace = gb._workspace(7, torch.device("cuda:0"), 0)
    assert segment_stream(workspace) == torch.cuda.default_stream().cuda_stream == 0


def test_a_stream_of_another_device_is_refused(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    other = Stream()
    other.device_index = 1
    with pytest.raises(ValueError, match="the stream is on cuda:1, the current device is cuda:0"):
        gb._on_current_device("gdn_scan_forward", other)
    for s in (None, 0x1230, Stream()):
        gb._on_current_device("gdn_scan_forward", s, None)
