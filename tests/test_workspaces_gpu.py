"""Workspaces that captured calls and other streams still use when a later call needs more of them."""
import numpy as np
import pytest
import torch

import paged_split_kv_gb300 as sk
from test_evict_gpu import PAGE, cache, dev, reference as evicted
from test_prefill_gpu import batch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def calls(b, ws, acc):
    w = b["w"]
    out, lse = sk.paged_prefill_attention(b["q"], b["kv"], b["bt"], b["lens"], b["cu"], max_q_len=w.max_q_len,
                                          sm_scale=w.sm_scale, k_scale=w.k_scale, v_scale=w.v_scale, workspace=ws)
    sk.sk_accum_attn_weights(b["q"], b["kv"], b["bt"], b["lens"], b["cu"], lse, acc, max_q_len=w.max_q_len,
                             sm_scale=w.sm_scale, k_scale=w.k_scale, workspace=ws)
    return out, lse


def test_a_captured_call_after_its_workspace_was_outgrown():
    """Warmed up, captured, then a larger call with the same dict: what is allocated after that stays as it is under
    replays, and they give the results of the small call."""
    small, large = batch([3000, 2500], [40, 10], 8, 1, True, 81), batch([9000, 4000], [2000, 1500], 16, 2, True, 82)
    ws = {}
    acc = torch.zeros(small["kv"].shape[:3], device=DEV)
    want = [t.clone() for t in calls(small, ws, acc)] + [acc.clone()]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out, lse = calls(small, ws, acc)
    before = ws["prefill"].numel(), ws["accum"].numel()
    more = torch.zeros(large["kv"].shape[:3], device=DEV)
    calls(large, ws, more)
    assert ws["prefill"].numel() > before[0] and ws["accum"].numel() > before[1]
    held = [torch.full((n,), 0xA5, dtype=torch.uint8, device=DEV) for n in 4 * before]
    for _ in range(3):
        acc.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and torch.equal(acc, want[2])
    assert all(bool((t == 0xA5).all()) for t in held)
    assert sk.sk_get_device_status() == 0


def test_a_workspace_used_on_another_stream_and_dropped():
    """A dict whose buffers were taken on one stream, last used by calls that wait on another: what is allocated after the
    dict is gone is not written by them."""
    b = batch([3000, 2500], [40, 10], 8, 1, True, 83)
    ws = {}
    acc = torch.zeros(b["kv"].shape[:3], device=DEV)
    want = [t.clone() for t in calls(b, ws, acc)] + [acc.clone()]
    acc.zero_()
    sizes = ws["prefill"].numel(), ws["accum"].numel()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
        out, lse = calls(b, ws, acc)
    ws.clear()
    held = [torch.full((n,), 0xA5, dtype=torch.uint8, device=DEV) for n in 4 * sizes]
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and torch.equal(acc, want[2])
    assert all(bool((t == 0xA5).all()) for t in held)
    assert sk.sk_get_device_status() == 0


def test_evictions_of_growing_lengths_and_other_batches_with_one_workspace():
    """What a server does that passes its longest length of the moment: the lists follow."""
    ws = {}
    for lens, hkv, longest in (([30, 20, 32], 2, 32), ([33, 30, 36], 2, 36), ([33, 64, 100], 2, 100), ([300] * 5, 2, 300),
                               ([64], 2, 64), ([70, 40], 4, 70)):
        bt, acc, pos, pages = cache(lens, hkv, 31 + longest)
        want = evicted(bt, acc, pos, lens, lens, hkv, 32, 4)
        pg, a, p = dev(pages).view(torch.bfloat16), dev(acc), dev(pos)
        n = dev(lens, torch.int32)
        new = sk.evict_rows(pg, a, p, dev(bt), n, n, budget=32, recent=4, max_seq_len=longest, workspace=ws)
        assert sk.sk_get_device_status() == 0
        assert new.tolist() == [min(x, 32) for x in lens]
        for (s, h), (x, y) in want.items():
            assert ws["counts"][s, h] == len(x)
            assert ws["src_rows"][s, h, :len(x)].tolist() == x.tolist() and ws["dst_rows"][s, h, :len(x)].tolist() == y.tolist()
            for t in (pages, acc, pos):
                t[bt[s, y // PAGE], h, y % PAGE] = t[bt[s, x // PAGE], h, x % PAGE]
        np.testing.assert_array_equal(pg.view(torch.uint8).cpu().numpy(), pages)
        np.testing.assert_array_equal(a.cpu().numpy(), acc)
        np.testing.assert_array_equal(p.cpu().numpy(), pos)
