"""Waits that expire in the chunk attention and the attention weights: with a limit of no cycles the calls still
return, the status says so, and the next calls give the bits that they gave before."""
import pytest
import torch

import paged_split_kv_gb300 as sk
from test_prefill_gpu import batch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,qs,hq,hkv", [([20000, 9000, 300], [700, 1200, 300], 16, 2), ([30000] * 6, [3] * 6, 16, 2),
                                            ([700, 130] * 30, [1, 2] * 30, 8, 2)])
def test_expired_waits_are_reported_and_leave_no_trace(lens, qs, hq, hkv, fp8):
    b = batch(lens, qs, hq, hkv, fp8, 71)
    w = b["w"]

    def attend():
        return sk.paged_prefill_attention(b["q"], b["kv"], b["bt"], b["lens"], b["cu"], max_q_len=w.max_q_len,
                                          sm_scale=w.sm_scale, k_scale=w.k_scale, v_scale=w.v_scale)

    def gather(lse):
        acc = torch.zeros(b["kv"].shape[:3], device=DEV)
        sk.sk_accum_attn_weights(b["q"], b["kv"], b["bt"], b["lens"], b["cu"], lse, acc, max_q_len=w.max_q_len,
                                 sm_scale=w.sm_scale, k_scale=w.k_scale)
        return acc

    out, lse = attend()
    acc = gather(lse)
    assert sk.sk_get_device_status() == 0
    limit = sk.sk_set_wait_limit(0)
    try:
        for call in (attend, lambda: gather(lse)):
            for _ in range(3):                   # the calls return; nothing hangs
                call()
            assert sk.sk_get_device_status(clear=True) & sk.SK_DEV_TIMEOUT
    finally:
        sk.sk_set_wait_limit(-1)
    assert limit > 0
    out2, lse2 = attend()
    acc2 = gather(lse2)
    assert sk.sk_get_device_status() == 0
    assert torch.equal(out, out2) and torch.equal(lse, lse2) and torch.equal(acc, acc2)
