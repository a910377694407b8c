"""Query offsets that are no offsets: the sequences that have them are left out and reported, whatever the numbers' differences
come to in 32 bits."""
import pytest
import torch

import paged_split_kv_gb300 as sk
from test_accum_gpu import start
from test_prefill_gpu import batch, reference

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("cu", [[0, 20, 2 ** 31 - 1, -2 ** 31], [0, 20, -2 ** 31, -2 ** 31 + 7], [0, 20, 10, -5], [0, 20, 61, 60]])
def test_sequences_with_bad_offsets_are_left_out(cu, fp8):
    b = batch([200, 90, 70], [20, 30, 10], 16, 2, fp8, 97)
    w = b["w"]
    ref, ref_lse, tol, _ = reference(b)
    offsets = torch.tensor(cu, dtype=torch.int32, device=DEV)
    out = torch.full((60, 16, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((60, 16), 3.0, device=DEV)
    args = dict(max_q_len=30, sm_scale=w.sm_scale, k_scale=w.k_scale)
    sk.sk_get_device_status(clear=True)
    sk.sk_paged_prefill_attn(b["q"], b["kv"], b["bt"], b["lens"], offsets, out, lse, v_scale=w.v_scale, **args)
    assert sk.sk_get_device_status() == sk.SK_DEV_BAD_SEQ
    assert bool(((out.double() - ref).abs() <= tol)[:20].all())
    assert bool((out[20:] == 3).all()) and bool((lse[20:] == 3).all())
    acc0 = start(b, 8)
    for q_len in (30, 4):                        # many rows a sequence; few, of which the first has too many as well
        acc = acc0.clone()
        sk.sk_accum_attn_weights(b["q"], b["kv"], b["bt"], b["lens"], offsets, ref_lse.float(), acc,
                                 **dict(args, max_q_len=q_len))
        assert sk.sk_get_device_status() == sk.SK_DEV_BAD_SEQ
        used = b["bt"][1:][b["bt"][1:] >= 0].long()
        assert torch.equal(acc[used], acc0[used])
        assert torch.equal(acc, acc0) == (q_len == 4)
