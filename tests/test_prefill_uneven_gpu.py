"""Chunk attention of uneven batches: one long conversation beside many short prompts."""
import pytest
import torch

import paged_split_kv_gb300 as sk
from test_prefill_gpu import batch, check, run

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def took(b, **kw):
    """Microseconds a call, the best of five."""
    w = b["w"]
    ws = {}
    out = torch.empty((w.num_tokens, w.num_q_heads, 128), dtype=torch.bfloat16, device=DEV)
    best = float("inf")
    for i in range(8):
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        sk.sk_paged_prefill_attn(b["q"], b["kv"], b["bt"], b["lens"], b["cu"], out, max_q_len=w.max_q_len,
                                 sm_scale=w.sm_scale, workspace=ws, **kw)
        end.record()
        end.synchronize()
        best = min(best, start.elapsed_time(end) * 1e3) if i >= 3 else best
    return best


@pytest.mark.parametrize("long_first", [True, False])
@pytest.mark.parametrize("long,short,n", [((110000, 64), 500, 19), ((110000, 33), 2000, 39)])
def test_the_work_of_an_uneven_batch_is_divided_evenly(long, short, n, long_first):
    """As fast as the same call that is told of a single key (max_seq_len, a wrong one costs time only), whose work is cut into
    equal runs: 1268 against 166 us, and 2322 against 1207, where whole units were dealt out."""
    lens, qs = [long[0] + long[1]] + [short] * n, [long[1]] + [short] * n
    if not long_first:
        lens, qs = lens[::-1], qs[::-1]
    b = batch(lens, qs, 32, 8, False, 95)
    assert took(b) < 1.6 * took(b, max_seq_len=1)
    assert sk.sk_get_device_status() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,qs,hq,hkv", [
    ([30000] + [300] * 20, [5] + [300] * 20, 32, 8), ([300] * 40 + [0, 1, 25000], [20] * 40 + [0, 1, 100], 160, 8),
    ([6000] * 3 + [0] * 40 + [6001] * 2, [130] * 3 + [0] * 40 + [64] * 2, 160, 8)])
def test_uneven_batches_against_64_bits(lens, qs, hq, hkv, fp8):
    """Larger than the L2 by what the table holds: cut into runs, and (the last) dealt out past empty sequences."""
    b = batch(lens, qs, hq, hkv, fp8, 96)
    out, lse = run(b)
    assert sk.sk_get_device_status() == 0
    check(b, out, lse)
    again, lse2 = run(b)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
