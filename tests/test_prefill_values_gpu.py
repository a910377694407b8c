"""Chunk attention where values are at the edge: keys whose scores are minus infinity, and a key far above the rest on
e4m3 pages.

Tolerances, as for the other batches: a score is off by e = 130 * 2^-24 * scale * sum |q k| (128 products in fp32) and
2^-20 (the exponential and the sums), the output rounds by 2^-8, a probability by 2^-8 of itself in bf16.  In f16 (e4m3
pages) it rounds by 2^-11 of itself or by a fixed 2^-25, whichever is more; a key that the row sees has at least 2^8 there,
so that is at most 2^-33 of the row's sum.
    |out - ref| <= 2^-8 |ref| + sum (2^-8 p + 2 e p + 2^-33) |v|,  without the last term for bf16"""
import math

import pytest
import torch

import paged_split_kv_gb300 as sk
from test_prefill_gpu import batch, rows_of, run

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
D, PAGE = 128, 16


def check(b, out, lse, gone=()):
    """Compares with the definition in 64 bits; keys `gone` of every sequence have the weight 0."""
    w = b["w"]
    fp8 = b["kv"].element_size() == 1
    assert not torch.isnan(out.float()).any() and not torch.isnan(lse).any()
    for s in range(w.bs):
        n, q, a = int(w.seq_lens[s]), int(w.q_lens[s]), int(w.cu_q[s])
        p_at = torch.arange(n, device=DEV)
        hide = p_at[None, :] >= (n - q + 1 + torch.arange(q, device=DEV))[:, None]
        drop = torch.zeros(n, dtype=torch.bool, device=DEV)
        drop[[k for k in gone if k < n]] = True
        for h in range(w.num_kv_heads):
            k, v = rows_of(b, s, h, 0), rows_of(b, s, h, 1)
            k = torch.where(drop[:, None], 0.0, k)
            for i in range(h * w.group, (h + 1) * w.group):
                x = b["q"][a:a + q, i].double()
                sc = (x @ k.t()) * w.sm_scale
                sc[hide | drop[None, :]] = -math.inf
                e = 130 * 2.0 ** -24 * w.sm_scale * (x.abs() @ k.abs().t()).amax(1) + 2.0 ** -20
                p = torch.softmax(sc, 1)
                ref, want = p @ v, torch.logsumexp(sc, 1)
                floor = 2.0 ** -33 if fp8 else 0.0
                tol = 2.0 ** -8 * ref.abs() + ((2.0 ** -8 + 2 * e)[:, None] * p + floor * ~hide) @ v.abs()
                err = (out[a:a + q, i].double() - ref).abs()
                assert bool((err <= tol).all()), (s, i, float((err / tol).max()))
                off = (lse[a:a + q, i].double() - want).abs()
                assert bool((off <= e + 2.0 ** -22 * want.abs()).all()), (s, i, float(off.max()))


@pytest.mark.parametrize("most", [0, None])
@pytest.mark.parametrize("lens,qs,hq,hkv,gone", [
    ([100], [20], 4, 1, range(16)),                              # the first 16 keys of the only tile
    ([128, 90, 17], [30, 7, 1], 8, 2, range(16)),
    ([1000, 700], [140, 33], 16, 2, range(16)),                  # of the first tile
    ([1000, 700], [140, 33], 16, 2, range(128, 144)),
    ([1000, 700], [140, 33], 16, 2, range(300)),                 # whole tiles and more
    ([1000], [3], 5, 1, [k for k in range(900) if k % 128 < 16 or k % 128 > 100]),
    ([20000], [33], 8, 1, [k for k in range(19900) if k % 128 < 16]),      # of every tile, in the pieces of many runs
    ([20000], [33], 8, 1, range(15000)),                         # and of all tiles of some
])
def test_scores_of_minus_infinity(lens, qs, hq, hkv, gone, most):
    """Keys with an element of minus infinity where the queries are positive weigh nothing, wherever they lie."""
    b = batch(lens, qs, hq, hkv, False, 91)
    b["q"][..., 0] = b["q"][..., 0].abs() + 0.5
    at = torch.tensor(list(gone), device=DEV)
    for s, n in enumerate(lens):
        k = at[at < n]
        b["kv"][b["bt"][s].long()[k // PAGE], :, k % PAGE, 0] = -math.inf
    out, lse = run(b, max_seq_len=most)
    assert sk.sk_get_device_status() == 0
    check(b, out, lse, list(gone))


@pytest.mark.parametrize("most", [0, None])
@pytest.mark.parametrize("code,nats", [(36.0, 12.7), (44.0, 15.6), (52.0, 18.4), (56.0, 19.8)])
@pytest.mark.parametrize("lens,qs,hq,hkv", [([20000], [16], 8, 1), ([6000, 3000], [200, 64], 8, 2)])
def test_a_key_far_above_the_rest_on_e4m3_pages(lens, qs, hq, hkv, code, nats, most):
    """The first key of each sequence lies `nats` above scores that are nearly equal, and its V is 0: the output is what the
    others give."""
    b = batch(lens, qs, hq, hkv, True, 92)
    b["q"] *= 0.125
    b["q"][..., 0] = 8.0
    kv = b["kv"].view(torch.float8_e4m3fn)
    for s in range(len(lens)):
        kv[b["bt"][s, :(lens[s] + PAGE - 1) // PAGE].long(), :, :, 0] = 0.0
        kv[b["bt"][s, 0].long(), :, 0, 0] = code
        kv[b["bt"][s, 0].long(), :, 0, D:] = 0.0
    assert abs(8 * code * b["w"].k_scale * b["w"].sm_scale - nats) < 0.1
    out, lse = run(b, max_seq_len=most)
    assert sk.sk_get_device_status() == 0
    check(b, out, lse)
