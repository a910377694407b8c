"""Attention with a sliding window and sinks against the definition in 64 bits (bounds: window_helpers)."""
import pytest
import torch

import paged_split_kv_gb300 as sk
import sk_inputs as si
from window_helpers import DEV, batch, check, reference, run

pytestmark = pytest.mark.gpu

SHAPES = [
    # steps: one to a few tokens a sequence
    ([1], [1], 1, 1), ([40], [1], 8, 1), ([300, 17, 0, 1], [1, 1, 0, 1], 16, 2), ([700, 128, 129], [4, 2, 3], 32, 2),
    ([2, 5], [4, 5], 5, 1), ([600], [5], 40, 1), ([1025] * 3, [1] * 3, 4, 4), ([260, 90], [2, 3], 300, 1),
    # chunks
    ([300], [300], 4, 2), ([127, 128, 129, 255, 256, 257], [127, 1, 129, 100, 256, 2], 2, 1),
    ([700, 64, 3], [133, 64, 60], 5, 1), ([1000, 1500], [140, 60], 12, 4), ([513], [300], 128, 1),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (17, 4), (128, 16), (129, 33), (500, 130),
                                          (5000, 0), (64, 5000), (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("lens,qs,hq,hkv", SHAPES)
def test_against_64_bits(lens, qs, hq, hkv, window, sinks, fp8):
    b = batch(lens, qs, hq, hkv, fp8, 31 + len(lens), window, sinks)
    out, lse = run(b)
    assert sk.sk_get_device_status() == 0
    check(b, out, lse)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("q,sinks,first", [(1, 20, d) for d in (19, 20, 21, 31, 32, 33, 47, 48, 49, 64, 160)] +
                         [(9, 0, d) for d in (0, 1, 15, 16, 17, 127, 128, 129)] + [(70, 3, 16), (70, 3, 144)])
def test_window_that_starts_near_the_sinks(q, sinks, first, fp8):
    """The first row of the window lies before, on and past the pages of the sinks, and of tiles."""
    n = 400 + q
    b = batch([n, n - 3], [q, q], 8, 2, fp8, 11, n - q + 1 - first, sinks)
    out, lse = run(b)
    assert sk.sk_get_device_status() == 0
    check(b, out, lse)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window", [100, 900, 100000])
def test_window_of_the_whole_cache_is_causal_attention(window, fp8):
    """A window (or sinks) of at least the length: the bits of sk_paged_prefill_attn are within the same bounds."""
    lens, qs = [900, 300, 77], [130, 300, 1]
    b = batch(lens, qs, 16, 2, fp8, 5, window, 900 if window < 900 else 0)
    out, lse = run(b)
    assert sk.sk_get_device_status() == 0
    ref = reference(b)
    check(b, out, lse, ref)
    w = b["w"]
    o2, l2 = sk.paged_prefill_attention(b["q"], b["kv"], b["bt"], b["lens"], b["cu"], max_q_len=w.max_q_len,
                                        sm_scale=w.sm_scale, k_scale=w.k_scale, v_scale=w.v_scale)
    check(b, o2, l2, ref)


@pytest.mark.parametrize("lens,qs,hq,hkv,window,sinks,fp8", [
    ([30000, 21001], [33, 9], 32, 2, 20000, 4, False), ([50001], [1], 5, 1, 30000, 0, True),
    ([3000] * 30, [1] * 30, 8, 2, 700, 4, False), ([9000] * 5, [4] * 5, 32, 2, 4096, 64, True),
    ([1500, 1, 700, 2999, 40], [900, 1, 700, 100, 40], 8, 4, 333, 7, False), ([4000, 2500], [600, 900], 16, 2, 512, 4, True),
    ([70000, 3], [1, 1], 8, 8, 60000, 100, False), ([5000], [5000], 4, 1, 129, 1, False)])
def test_units_cut_between_runs(lens, qs, hq, hkv, window, sinks, fp8):
    """Long windows of few tokens, whole prompts, ragged chunks: runs start and end inside units, several share one; the
    same bits every time, whatever bound of the lengths the call is given."""
    b = batch(lens, qs, hq, hkv, fp8, 13, window, sinks)
    out, lse = run(b)
    assert sk.sk_get_device_status() == 0
    check(b, out, lse)
    again = run(b)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    ref = reference(b)
    for most in (0, 1000, 2 ** 31 - 1):
        check(b, *run(b, max_seq_len=most), ref)
    assert sk.sk_get_device_status() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("gain", [0.0, 8.0])
def test_flat_and_peaked_scores(gain, fp8):
    """Equal scores, and peaked ones whose maximum lies anywhere in the window."""
    for lens, qs in (([2000, 700], [150, 300]), ([2000, 700], [1, 3])):
        b = batch(lens, qs, 8, 2, fp8, 77, 600, 4, gain=gain)
        out, lse = run(b)
        assert sk.sk_get_device_status() == 0
        check(b, out, lse)


@pytest.mark.parametrize("q", [1, 3, 200])
def test_scores_that_grow_along_the_window(q):
    """Keys that agree with the queries more and more: the running reference moves from tile to tile."""
    b = batch([1500], [q], 8, 2, False, 9, 1100, 4, gain=8.0, forget=False)
    for i in range((1500 + 15) // 16):
        blk = int(b["bt"][0, i])
        b["kv"][blk, :, :, :128] = b["kv"][blk, :, :, :128] * (0.1 + 2.5 * i / 94)
    out, lse = run(b)
    assert sk.sk_get_device_status() == 0
    check(b, out, lse)
