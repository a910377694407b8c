"""Gathered attention weights against the definition in 64 bits.

Tolerances.  A weight exp(score - lse) is off, relatively, by the score's error (128 products in fp32: 130 * 2^-24 *
scale * sum |q k|; e4m3 pages also 2^-18 * scale * max |q| * sum |k| for q in two terms), by the rounding of the
exponent, 2^-23 (|score| + |lse|), and by the exponential's 2^-22; a key's sum over n rows rounds by n 2^-24, and its
addition to what was there by 2^-24."""
import math

import numpy as np
import pytest
import torch

import paged_split_kv_gb300 as sk
import sk_inputs as si
from test_prefill_gpu import batch, reference as attention, rows_of

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
D, PAGE = 128, 16


def weights(b, lse, acc0):
    """acc after the call in 64 bits, and its bound."""
    w = b["w"]
    g = w.group
    acc, tol = acc0.double(), torch.zeros_like(acc0, dtype=torch.float64)
    for s in range(w.bs):
        n, q, a = int(w.seq_lens[s]), int(w.q_lens[s]), int(w.cu_q[s])
        if n == 0 or q == 0:
            continue
        see = torch.full((q,), n, device=DEV)
        if w.causal:
            see = (n - q + 1 + torch.arange(q, device=DEV)).clamp(0, n)
        hide = torch.arange(n, device=DEV)[None, :] >= see[:, None]
        r = torch.arange(n, device=DEV)
        blk = b["bt"][s].long()[r // PAGE]
        for h in range(w.num_kv_heads):
            k = rows_of(b, s, h, 0)
            total, bound = torch.zeros(n, dtype=torch.float64, device=DEV), torch.zeros(n, dtype=torch.float64, device=DEV)
            for i in range(h * g, (h + 1) * g):
                x = b["q"][a:a + q, i].double()
                sc = (x @ k.t()) * w.sm_scale
                norm = lse[a:a + q, i].double()[:, None]
                e = 130 * 2.0 ** -24 * w.sm_scale * (x.abs() @ k.abs().t()) + 2.0 ** -22
                if w.kv_dtype == si.KV_FP8:
                    e += 2.0 ** -18 * w.sm_scale * x.abs().amax(1, keepdim=True) * k.abs().sum(1)[None, :]
                e += 2.0 ** -23 * (sc.abs() + norm.abs().nan_to_num(posinf=0))
                p = torch.where(hide | torch.isinf(norm), 0.0, torch.exp(sc - norm))
                total += p.sum(0)
                bound += (p * (e + q * g * 2.0 ** -24)).sum(0)
            acc[blk, h, r % PAGE] += total
            tol[blk, h, r % PAGE] += bound + 2.0 ** -24 * acc[blk, h, r % PAGE].abs()
    return acc, tol


def start(b, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.rand(b["kv"].shape[:3], generator=g, device=DEV)


def run(b, lse, acc, **kw):
    w = b["w"]
    args = dict(max_q_len=max(1, w.max_q_len), sm_scale=w.sm_scale, k_scale=w.k_scale, causal=bool(w.causal))
    args.update(kw)
    sk.sk_accum_attn_weights(b["q"], b["kv"], b["bt"], b["lens"], b["cu"], lse, acc, **args)
    torch.cuda.synchronize()


def check(b, lse, acc0, acc):
    want, tol = weights(b, lse, acc0)
    err = (acc.double() - want).abs()
    assert bool((err <= tol).all()), (int((~(err <= tol)).sum()), float((err / (tol + 1e-30)).max()))
    assert torch.equal(acc[tol == 0], acc0[tol == 0])           # places of no key


SHAPES = [
    ([1], [1], 1, 1), ([5, 300], [1, 1], 8, 1), ([128], [16], 8, 1), ([129], [17], 16, 2), ([300], [300], 4, 2),
    ([127, 128, 129, 255, 256, 257], [127, 1, 129, 100, 256, 2], 2, 1),
    ([17, 0, 1, 700, 64], [4, 0, 1, 2, 3], 32, 2), ([3, 0, 40], [5, 4, 60], 16, 2),
    ([1000, 1500], [140, 60], 12, 4), ([900], [7], 40, 1), ([513], [300], 128, 1), ([260, 40], [3, 2], 300, 1),
    ([2500], [1], 5, 1), ([5000, 100, 900], [3, 3, 3], 16, 2),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,qs,hq,hkv", SHAPES)
def test_against_64_bits(lens, qs, hq, hkv, causal, fp8):
    b = batch(lens, qs, hq, hkv, fp8, 41 + len(lens), causal)
    lse = attention(b)[1].float()
    acc0 = start(b, 1)
    acc = acc0.clone()
    run(b, lse, acc)
    assert sk.sk_get_device_status() == 0
    check(b, lse, acc0, acc)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,qs,hq,hkv", [([60000, 20001, 7], [4, 4, 4], 32, 2), ([9000, 12345], [700, 1100], 16, 2),
                                            ([4097] * 40, [1] * 40, 32, 8)])
def test_many_tiles_and_the_same_bits_twice(lens, qs, hq, hkv, fp8):
    """Runs that start and end inside sequences and heads; the library's own lse; the sums add up to the rows."""
    b = batch(lens, qs, hq, hkv, fp8, 51)
    w = b["w"]
    _, lse = sk.paged_prefill_attention(b["q"], b["kv"], b["bt"], b["lens"], b["cu"], max_q_len=w.max_q_len,
                                        sm_scale=w.sm_scale, k_scale=w.k_scale, v_scale=w.v_scale)
    acc0 = torch.zeros(b["kv"].shape[:3], device=DEV)
    acc, again = acc0.clone(), acc0.clone()
    run(b, lse, acc)
    run(b, lse, again)
    assert sk.sk_get_device_status() == 0
    assert torch.equal(acc, again)
    check(b, lse, acc0, acc)
    assert math.isclose(acc.double().sum().item(), w.num_tokens * hq, rel_tol=1e-5)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,qs,hq,hkv", [([700, 1, 400, 1025, 130, 0, 513] * 20, [1, 1, 2, 4, 3, 1, 0] * 20, 16, 8),
                                            ([1500, 260, 129, 2600] * 20, [1, 2, 1, 4] * 20, 32, 8),
                                            ([700, 200, 1800] * 20, [70, 150, 40] * 20, 8, 2)])
def test_many_short_sequences_a_run(lens, qs, hq, hkv, fp8):
    """Every ring of a CTA turns over several times between short items: the same bits in each of many calls."""
    b = batch(lens, qs, hq, hkv, fp8, 52)
    lse = attention(b)[1].float()
    acc0 = start(b, 3)
    acc = acc0.clone()
    run(b, lse, acc)
    for _ in range(20):
        again = acc0.clone()
        run(b, lse, again)
        assert torch.equal(acc, again)
    assert sk.sk_get_device_status() == 0
    check(b, lse, acc0, acc)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,qs,hq,hkv", [([25000, 24999, 129, 30001] * 3, [1, 2, 0, 1] * 3, 16, 8),
                                            ([33000, 1, 20000, 18000, 40001], [4, 1, 3, 4, 2], 256, 16)])
def test_long_batches_of_few_rows(lens, qs, hq, hkv, fp8):
    """The last part of a long batch goes out in short runs; under wide tables a short batch leaves those empty."""
    b = batch(lens, qs, hq, hkv, fp8, 53)
    lse = (torch.randn(b["w"].num_tokens, hq, device=DEV) + 12).contiguous()
    acc0 = start(b, 4)
    acc, again = acc0.clone(), acc0.clone()
    run(b, lse, acc)
    run(b, lse, again)
    assert sk.sk_get_device_status() == 0 and torch.equal(acc, again)
    check(b, lse, acc0, acc)
    few = batch([300, 1, 0, 77], [1, 1, 0, 1], hq, hkv, fp8, 54)
    few["bt"] = torch.nn.functional.pad(few["bt"], (0, 20000), value=-1)
    lse = attention(few)[1].float()
    acc0 = start(few, 5)
    acc = acc0.clone()
    run(few, lse, acc)
    assert sk.sk_get_device_status() == 0
    check(few, lse, acc0, acc)


def test_rows_that_saw_nothing_add_nothing():
    b = batch([500, 200], [3, 2], 4, 1, False, 61)
    lse = attention(b)[1].float()
    lse[1], lse[4, 2] = -math.inf, -math.inf
    acc0 = start(b, 2)
    acc = acc0.clone()
    run(b, lse, acc)
    check(b, lse, acc0, acc)


def test_sequences_that_share_a_block():
    """A common prefix: both sequences' rows add to its keys."""
    b = batch([64, 80], [2, 3], 4, 2, False, 62)
    b["bt"][1, :4] = b["bt"][0, :4]
    lse = attention(b)[1].float()
    acc0 = start(b, 3)
    acc = acc0.clone()
    run(b, lse, acc)
    check(b, lse, acc0, acc)


def test_bad_blocks_and_lengths_are_reported():
    b = batch([400, 300], [2, 3], 4, 1, False, 63)
    lse = attention(b)[1].float()
    acc0 = start(b, 4)
    acc = acc0.clone()
    keep = b["bt"].clone()
    b["bt"][0, 3] = 10 ** 6
    sk.sk_get_device_status(clear=True)
    run(b, lse, acc)
    assert sk.sk_get_device_status() == sk.SK_DEV_BAD_BLOCK
    assert torch.equal(acc[keep[0, 3]], acc0[keep[0, 3]])
    b["bt"].copy_(keep)
    acc = acc0.clone()
    run(b, lse, acc, max_q_len=2)                               # the second sequence is longer: left out
    assert sk.sk_get_device_status() == sk.SK_DEV_BAD_SEQ
    assert torch.equal(acc[b["bt"][1, :19].long()], acc0[b["bt"][1, :19].long()])
    assert not torch.equal(acc, acc0)


def test_many_sequences_of_uneven_lengths():
    """More sequences than threads: the run of each CTA is found among several sequences per thread."""
    rng = np.random.default_rng(9)
    lens = rng.integers(0, 300, size=1500)
    qs = np.minimum(lens, rng.integers(0, 3, size=1500))
    b = batch(lens, qs, 4, 1, False, 64)
    acc0 = start(b, 5)
    acc = acc0.clone()
    lse = torch.full((b["w"].num_tokens, 4), 3.0, device=DEV)
    run(b, lse, acc)
    assert sk.sk_get_device_status() == 0
    # the sum of the gathered weights of each sequence, in 64 bits
    w = b["w"]
    diff = (acc.double() - acc0.double()).sum((1, 2))
    for s in rng.choice(1500, size=60, replace=False):
        n, q, a = int(w.seq_lens[s]), int(w.q_lens[s]), int(w.cu_q[s])
        got = diff[b["bt"][s, :(n + PAGE - 1) // PAGE].long()].sum().item()
        want = 0.0
        if n and q:
            sc = torch.einsum("qhd,nd->qhn", b["q"][a:a + q].double(), rows_of(b, s, 0, 0)) * w.sm_scale
            seen = torch.arange(n, device=DEV)[None, :] <= (n - q + torch.arange(q, device=DEV))[:, None]
            want = float((torch.exp(sc - 3.0) * seen[:, None, :]).sum())
        assert abs(got - want) <= 1e-4 * want + n * 2.0 ** -23, (s, got, want)    # false for NaN


def test_captured_with_new_lengths():
    b = batch([3000, 2500], [4, 2], 8, 1, True, 65)
    w = b["w"]
    lse = torch.full((6, 8), 8.0, device=DEV)
    acc0 = start(b, 6)
    acc = acc0.clone()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        sk.sk_accum_attn_weights(b["q"], b["kv"], b["bt"], b["lens"], b["cu"], lse, acc, max_q_len=4,
                                 sm_scale=w.sm_scale, k_scale=w.k_scale)
    w.seq_lens[:] = [2900, 1777]
    b["lens"].copy_(torch.as_tensor(w.seq_lens, device=DEV))
    graph.replay()
    torch.cuda.synchronize()
    check(b, lse, acc0, acc)
