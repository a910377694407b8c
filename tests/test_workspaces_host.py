"""Buffers that the binding keeps in a workspace dict, without a GPU: an outgrown buffer stays (a captured graph may hold its
address), and a use on another stream is recorded."""
import contextlib
import gc
import weakref

import pytest
import torch

import paged_split_kv_gb300 as sk

CPU = torch.device("cpu")


def test_outgrown_buffers_stay_and_sizes_double():
    ws, seen = {}, []
    for need in (100, 100, 101, 150, 199, 202, 203, 5000, 5001, 64):
        at = sk._buffer(ws, "prefill", need, CPU, None)
        assert ws["prefill"].data_ptr() == at and ws["prefill"].numel() >= need
        if not seen or seen[-1]() is not ws["prefill"]:
            seen.append(weakref.ref(ws["prefill"]))
    gc.collect()
    assert len(seen) == 5 and all(r() is not None for r in seen)
    sizes = [r().numel() for r in seen]
    assert sum(sizes) <= 2 * sizes[-1]
    other = sk._buffer(ws, "accum", 10, CPU, None)
    assert other == ws["accum"].data_ptr() != ws["prefill"].data_ptr()


class Memory:
    """Stands for a device buffer."""

    def __init__(self, n, device):
        self.n, self.device, self.used_on = n, device, []

    def numel(self):
        return self.n

    def data_ptr(self):
        return id(self)

    def record_stream(self, stream):
        self.used_on.append(stream)


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def streams(monkeypatch):
    """Device memory and streams without a device; the current stream's handle is the list's only entry."""
    now = [7]
    monkeypatch.setattr(torch, "empty", lambda n, dtype, device: Memory(n, device))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: now[0], raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(now[0]))
    monkeypatch.setattr(torch.cuda, "stream", lambda stream: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: Stream(handle))
    return now


def test_uses_on_other_streams_are_recorded(streams):
    dev, ws = torch.device("cuda", 0), {}

    def use(need, stream=None):
        sk._buffer(ws, "accum", need, dev, stream)
        return [s.cuda_stream for s in ws["accum"].used_on]

    assert use(10) == [] and use(10) == [] and use(10, Stream(7)) == [] and use(10, 7) == []
    assert use(10, Stream(8)) == [8] and use(10, 9) == [8, 9]
    streams[0] = 11
    assert use(10) == [8, 9, 11]
    assert use(50, Stream(12)) == [] and use(50, 12) == [] and use(50) == [11]    # a new buffer, taken on 12
    assert [s.cuda_stream for s in ws["outgrown"][0].used_on] == [8, 9, 11]
