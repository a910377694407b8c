"""Steps without query tokens: arrays of no tokens may have no address (torch gives them none); nothing is launched or
written."""
import ctypes

import pytest
import torch

import paged_split_kv_gb300 as sk

FAKE = ctypes.c_void_p(256)   # never dereferenced


def test_c_calls_without_tokens():
    from paged_split_kv_gb300 import build as b
    b.build()
    attend, gather = sk.lib().sk_paged_prefill_attn, sk.lib().sk_accum_attn_weights
    for nt, want in ((0, 0), (4, -1)):
        for max_q in (0, 4):
            assert attend(None, FAKE, 0, 1.0, 1.0, FAKE, 10, 100, 16, FAKE, FAKE, 4, nt, max_q, 32, 2, 128, 0.088, 1, 160,
                          FAKE, 1 << 30, None, None, None) == want
            assert gather(None, FAKE, 0, 1.0, FAKE, 10, 100, 16, FAKE, FAKE, 4, nt, max_q, 32, 2, 128, 0.088, 1, None, FAKE,
                          FAKE, 1 << 30, None) == want


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
def test_calls_without_tokens(dtype):
    dev = "cuda:0"
    kv = torch.zeros(6, 2, 16, 256, device=dev).to(dtype)
    bt = torch.arange(6, dtype=torch.int32, device=dev).view(2, 3)
    lens, cu = torch.tensor([40, 0], dtype=torch.int32, device=dev), torch.zeros(3, dtype=torch.int32, device=dev)
    q = torch.empty(0, 8, 128, dtype=torch.bfloat16, device=dev)
    out, lse = sk.paged_prefill_attention(q, kv, bt, lens, cu, max_q_len=0, sm_scale=0.1)
    assert out.shape == (0, 8, 128) and lse.shape == (0, 8)
    acc = torch.ones(6, 2, 16, device=dev)
    sk.sk_accum_attn_weights(q, kv, bt, lens, cu, lse, acc, max_q_len=0, sm_scale=0.1)
    torch.cuda.synchronize()
    assert sk.sk_get_device_status() == 0 and bool((acc == 1).all())
