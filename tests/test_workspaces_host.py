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


def test_eviction_lists_follow_the_call(monkeypatch):
    """One dict through calls with growing lengths and changing batches: lists of the call's shape and capacity, with the memory
    of earlier ones kept; lists that the caller put there serve while they fit."""
    got = []

    def select(acc, pos, bt, lens, nxt, src, dst, counts, new, *, budget, recent, max_seq_len, stream):
        got.append((src, dst, counts))
        assert src.shape == dst.shape and src.shape[:2] == counts.shape == (lens.numel(), acc.shape[1])
        assert src.shape[2] >= sk.sk_evict_capacity(budget, max_seq_len)
        for t in (src, dst, counts):
            assert t.dtype == torch.int32 and t.is_contiguous()
        spans = sorted((t.data_ptr(), t.data_ptr() + 4 * t.numel()) for t in (src, dst, counts))
        assert spans[0][1] <= spans[1][0] and spans[1][1] <= spans[2][0]

    monkeypatch.setattr(sk, "sk_evict_select", select)
    monkeypatch.setattr(sk, "sk_evict_move", lambda *a, **kw: None)

    def evict(ws, bs, longest, budget=100, hkv=2):
        i32 = torch.int32
        sk.evict_rows(torch.zeros(4, hkv, 16, 256, dtype=torch.bfloat16), torch.zeros(4, hkv, 16),
                      torch.zeros(4, hkv, 16, dtype=i32), torch.zeros(bs, 40, dtype=i32), torch.zeros(bs, dtype=i32),
                      torch.zeros(bs, dtype=i32), budget=budget, max_seq_len=longest, workspace=ws)
        return got[-1][0]

    ws = {}
    for bs, longest, budget, hkv in ((3, 90, 100, 2), (3, 101, 100, 2), (3, 160, 100, 2), (3, 110, 100, 2), (5, 640, 100, 2),
                                     (1, 640, 300, 2), (4, 500, 100, 4), (3, 90, 100, 2)):
        evict(ws, bs, longest, budget, hkv)
        assert ws["src_rows"].shape[:2] == (bs, hkv)
    at = evict(ws, 5, 640).data_ptr()
    for _ in range(3):                               # batches in turn take no more memory
        assert evict(ws, 5, 640).data_ptr() == at and evict(ws, 2, 90).data_ptr() == at
    kept = [ws["evict"]] + ws["outgrown"]
    assert sum(t.numel() for t in kept) <= 2 * ws["evict"].numel() and len(kept) < 6

    mine = dict(src_rows=torch.zeros(3, 2, 50, dtype=torch.int32), dst_rows=torch.zeros(3, 2, 50, dtype=torch.int32),
                counts=torch.zeros(3, 2, dtype=torch.int32))
    ws = dict(mine)
    assert evict(ws, 3, 150) is mine["src_rows"] and ws["src_rows"] is mine["src_rows"]
    assert evict(ws, 3, 151) is not mine["src_rows"] and any(t is mine["src_rows"] for t in ws["outgrown"])


def test_a_stream_is_recorded_once(streams):
    dev, ws = torch.device("cuda", 0), {}
    for handle in (7, 8, 7, 8, 9, 8, 9):
        sk._buffer(ws, "prefill", 10, dev, Stream(handle))
    assert [s.cuda_stream for s in ws["prefill"].used_on] == [8, 9]
