"""Attention of a chunk of new tokens against the definition in 64 bits.

Tolerances.  Scores accumulate 128 products in fp32: at most 130 * 2^-24 * scale * sum |q k| off (e: that over the
largest row, plus 2^-20 for the exponential and the sums).  Each probability rounds by at most 2^-8 (bf16; f16 for e4m3
pages) and the output by another 2^-8:
    |out - ref| <= 2^-8 |ref| + (2^-8 + 2 e) sum p |v|.  lse is off by e."""
import math

import numpy as np
import pytest
import torch

import paged_split_kv_gb300 as sk
import sk_inputs as si

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
D, PAGE = 128, 16


def batch(lens, qs, hq, hkv, fp8, seed, causal=True, gain=1.0):
    """Device tensors of a batch; rows past each end and blocks of no sequence hold NaN."""
    w = si.make_workload("t", lens, qs, hq, hkv, seed, kv_dtype=si.KV_FP8 if fp8 else si.KV_BF16,
                         k_scale=0.5 if fp8 else 1.0, v_scale=0.25 if fp8 else 1.0, causal=int(causal), spare_blocks=5)
    kv = si.make_kv(w, DEV)
    si.fill_unused_blocks(w, kv)
    return dict(w=w, q=si.make_q(w, DEV) * gain, kv=kv, bt=torch.as_tensor(w.block_table, device=DEV),
                lens=torch.as_tensor(w.seq_lens, device=DEV), cu=torch.as_tensor(w.cu_q, device=DEV))


def rows_of(b, s, h, part):
    """K (part 0) or V (part 1) of one sequence and head, in 64 bits."""
    w = b["w"]
    n = int(w.seq_lens[s])
    r = torch.arange(n, device=DEV)
    x = b["kv"][b["bt"][s].long()[r // PAGE], h, r % PAGE, part * D:(part + 1) * D]
    if w.kv_dtype == si.KV_FP8:
        return x.view(torch.float8_e4m3fn).double() * (w.v_scale if part else w.k_scale)
    return x.double()


def reference(b):
    """out, lse in 64 bits and the bounds of both."""
    w = b["w"]
    g = w.group
    out = torch.zeros(w.num_tokens, w.num_q_heads, D, dtype=torch.float64, device=DEV)
    lse = torch.full((w.num_tokens, w.num_q_heads), -math.inf, dtype=torch.float64, device=DEV)
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    for s in range(w.bs):
        n, q = int(w.seq_lens[s]), int(w.q_lens[s])
        a = int(w.cu_q[s])
        see = torch.full((q,), n, device=DEV)
        if w.causal:
            see = (n - q + 1 + torch.arange(q, device=DEV)).clamp(0, n)
        hide = torch.arange(n, device=DEV)[None, :] >= see[:, None]
        for h in range(w.num_kv_heads):
            k, v = rows_of(b, s, h, 0), rows_of(b, s, h, 1)
            for i in range(h * g, (h + 1) * g):
                x = b["q"][a:a + q, i].double()
                sc = (x @ k.t()) * w.sm_scale
                e = 130 * 2.0 ** -24 * w.sm_scale * (x.abs() @ k.abs().t()).amax(1) + 2.0 ** -20 if n else \
                    torch.zeros(q, device=DEV)
                sc[hide] = -math.inf
                p = torch.nan_to_num(torch.softmax(sc, 1))
                ref = p @ v
                out[a:a + q, i], lse[a:a + q, i] = ref, torch.logsumexp(sc, 1)
                tol_l[a:a + q, i] = e + 2.0 ** -22 * lse[a:a + q, i].abs().nan_to_num(posinf=0)
                tol_o[a:a + q, i] = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2 * e)[:, None] * (p @ v.abs())
    return out, lse, tol_o, tol_l


def check(b, out, lse, ref=None):
    ro, rl, to, tl = ref or reference(b)
    assert not torch.isnan(out.float()).any()
    err = (out.double() - ro).abs()
    bad = ~(err <= to + 1e-30)
    assert not bool(bad.any()), (int(bad.sum()), float((err / (to + 1e-30)).max()), bad.nonzero()[:4].tolist())
    dead = torch.isinf(rl)
    assert torch.equal(torch.isinf(lse) & (lse < 0), dead)
    le = (lse.double() - rl).abs()[~dead]
    assert bool((le <= tl[~dead]).all()), float((le / tl[~dead]).max())


def run(b, **kw):
    w = b["w"]
    args = dict(max_q_len=max(1, w.max_q_len), sm_scale=w.sm_scale, k_scale=w.k_scale, v_scale=w.v_scale,
                causal=bool(w.causal))
    args.update(kw)
    nt, hq = w.num_tokens, w.num_q_heads
    out = torch.full((nt, hq, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    lse = torch.full((nt, hq), float("nan"), device=DEV)
    sk.paged_prefill_attention(b["q"], b["kv"], b["bt"], b["lens"], b["cu"], out=out, lse=lse, **args)
    torch.cuda.synchronize()
    return out, lse


SHAPES = [
    ([1], [1], 1, 1), ([5], [5], 8, 1), ([128], [16], 8, 1), ([129], [17], 16, 2), ([300], [300], 4, 2),
    ([127, 128, 129, 255, 256, 257], [127, 1, 129, 100, 256, 2], 2, 1),
    ([17, 0, 1, 700, 64], [17, 0, 1, 33, 64], 5, 1),            # an empty sequence without query tokens
    ([3, 0, 40], [5, 4, 60], 16, 2),                            # rows that see no key
    ([1000, 1500], [140, 60], 12, 4), ([900], [7], 40, 1), ([513], [300], 128, 1), ([260, 40], [3, 2], 300, 1),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,qs,hq,hkv", SHAPES)
def test_against_64_bits(lens, qs, hq, hkv, causal, fp8):
    b = batch(lens, qs, hq, hkv, fp8, 31 + len(lens), causal)
    ref = reference(b)
    for most in (0, None):                        # one run for all, and as many as there is work for
        out, lse = run(b, max_seq_len=most)
        assert sk.sk_get_device_status() == 0
        check(b, out, lse, ref)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("gain", [0.0, 8.0])
def test_flat_and_peaked_scores(gain, fp8):
    """Equal scores, and scores whose maximum grows from tile to tile (the output is rescaled on the way)."""
    b = batch([2000, 700], [150, 300], 8, 2, fp8, 77, gain=gain)
    w = b["w"]
    if gain:
        # keys that agree with the queries more and more towards the end
        lift = torch.linspace(0, 1, b["kv"].shape[0] * PAGE, device=DEV)
        order = torch.cat([b["bt"][s, :(int(n) + PAGE - 1) // PAGE] for s, n in enumerate(w.seq_lens)]).long()
        if not fp8:
            for i, blk in enumerate(order.tolist()):
                b["kv"][blk, :, :, :D] = b["kv"][blk, :, :, :D] * (0.2 + 2 * lift[i * PAGE])
    out, lse = run(b)
    assert sk.sk_get_device_status() == 0
    check(b, out, lse)


@pytest.mark.parametrize("lens,qs,hq,hkv,fp8", [
    ([30000, 21001], [33, 9], 32, 2, False), ([50001], [1], 5, 1, True), ([3000] * 30, [1] * 30, 8, 2, False),
    ([1500, 1, 700, 2999, 40], [900, 1, 700, 100, 40], 8, 4, False), ([4000, 2500], [600, 900], 16, 2, True)])
def test_units_cut_between_runs(lens, qs, hq, hkv, fp8):
    """A short follow-up on two long caches, single tokens, ragged chunks: runs start and end inside units, several
    runs share one, and all bits are the same the second time."""
    b = batch(lens, qs, hq, hkv, fp8, 5)
    out, lse = run(b)
    assert sk.sk_get_device_status() == 0
    check(b, out, lse)
    again, lse2 = run(b)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("lens,qs,hq,hkv,fp8", [
    ([20000, 9000, 17], [1400, 300, 17], 32, 8, False), ([2500 + i for i in range(45)], [30 + i % 7 for i in range(45)], 8, 8, True),
    ([6000] * 3 + [0] * 40 + [9001] * 2, [130] * 3 + [0] * 40 + [64] * 2, 160, 8, False)])
def test_units_dealt_out_whole(lens, qs, hq, hkv, fp8):
    """Batches whose K and V do not stay in the L2: whole units first, over more than 32 sequences and past empty ones, then
    the rest in shares."""
    b = batch(lens, qs, hq, hkv, fp8, 15)
    out, lse = run(b)
    assert sk.sk_get_device_status() == 0
    check(b, out, lse)


def test_rows_past_the_last_sequence_stay():
    b = batch([200, 90], [20, 30], 4, 1, False, 6)
    w = b["w"]
    q = torch.cat([b["q"], b["q"][:7]])
    out = torch.full((57, 4, D), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((57, 4), 3.0, device=DEV)
    sk.sk_get_device_status(clear=True)
    sk.sk_paged_prefill_attn(q, b["kv"], b["bt"], b["lens"], b["cu"], out, lse, max_q_len=64,
                             sm_scale=w.sm_scale)
    assert sk.sk_get_device_status() == sk.SK_DEV_BAD_SEQ          # the offsets do not cover the tokens
    check(b, out[:50], lse[:50])
    assert bool((out[50:] == 3).all()) and bool((lse[50:] == 3).all())


def test_bad_blocks_and_query_lengths_are_reported():
    b = batch([400, 300], [20, 30], 4, 1, False, 7)
    w = b["w"]
    bt = b["bt"].clone()
    bt[0, 3], bt[0, 9] = 10 ** 6, -1
    out = torch.empty((50, 4, D), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((50, 4), device=DEV)
    sk.sk_get_device_status(clear=True)
    sk.sk_paged_prefill_attn(b["q"], b["kv"], bt, b["lens"], b["cu"], out, lse, max_q_len=30, sm_scale=w.sm_scale)
    assert sk.sk_get_device_status() == sk.SK_DEV_BAD_BLOCK
    ro, rl, to, tl = reference(b)
    assert bool(((out.double() - ro).abs() <= to)[20:].all())      # the other sequence is untouched by it
    sk.sk_paged_prefill_attn(b["q"], b["kv"], b["bt"], b["lens"], b["cu"], out, lse, max_q_len=20,
                             sm_scale=w.sm_scale)
    assert sk.sk_get_device_status() == sk.SK_DEV_BAD_SEQ
    assert bool(((out.double() - ro).abs() <= to)[:20].all())


def test_like_decode_attention_and_without_lse():
    """The same batch through the decode path: both within their bounds of the other."""
    b = batch([1000, 17, 0, 333], [4, 4, 4, 4], 16, 2, False, 8)
    w = b["w"]
    out, lse = run(b)
    o2, l2 = sk.paged_decode_attention(b["q"], b["kv"], b["bt"], b["lens"], b["cu"], max_q_len=4, sm_scale=w.sm_scale,
                                       num_sms=148)
    _, _, to, tl = reference(b)
    assert bool(((out.double() - o2.double()).abs() <= 2 * to + 1e-30).all())
    o3 = torch.empty_like(out)
    sk.sk_paged_prefill_attn(b["q"], b["kv"], b["bt"], b["lens"], b["cu"], o3, max_q_len=4, sm_scale=w.sm_scale)
    assert torch.equal(out, o3)


def test_two_graphs_and_another_stream():
    """Two captured calls replayed in turn on a side stream, each with buffers of its own; new lengths in place."""
    bs = [batch([3000, 2500], [40, 10], 8, 1, fp8, 9) for fp8 in (False, True)]
    side = torch.cuda.Stream()
    made = []
    for b in bs:
        w = b["w"]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            made.append((graph, sk.paged_prefill_attention(
                b["q"], b["kv"], b["bt"], b["lens"], b["cu"], max_q_len=40, sm_scale=w.sm_scale, k_scale=w.k_scale,
                v_scale=w.v_scale)))
    for b in bs:
        w = b["w"]
        w.seq_lens[:] = [2900, 1777]
        si.poison_unused_rows(w, b["kv"])
        b["lens"].copy_(torch.as_tensor(w.seq_lens, device=DEV))
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(3):
            for graph, _ in made:
                graph.replay()
    torch.cuda.synchronize()
    assert sk.sk_get_device_status() == 0
    for b, (_, (out, lse)) in zip(bs, made):
        check(b, out, lse)
