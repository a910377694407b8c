"""Batches with a sliding window and sinks, and their attention in 64 bits.

Bounds.  Scores accumulate 128 products in fp32: at most 130 * 2^-24 * scale * sum |q k| off (e: that over the largest
row, plus 2^-20 for the exponential and the sums).  Each probability rounds by at most 2^-8 (bf16; f16 for e4m3 pages)
and the output by another 2^-8:
    |out - ref| <= 2^-8 |ref| + (2^-8 + 2 e) sum p |v|.  lse is off by e.
On e4m3 pages q is two e4m3 terms of q 2^e, its row's largest element there in [128, 256): hi has 4 bits of an element's 8, lo the
others exactly unless their last is below 2^-9, the type's least, so for elements of 2^-9 of the largest or less lo is off
by up to 2^-10, which is 2^-17 of the largest.  That adds scale * 2^-17 max |q| sum |k| over those elements to e.
f16 has a fixed half step of 2^-25 below 2^-14, and the row's largest probability is held as 2^8 or more: each probability
of e4m3 pages may also be off by 2^-25 / 2^8 = 2^-33 of the row's sum, which adds 2^-33 sum |v| over the rows seen."""
import math

import torch

import paged_split_kv_gb300 as sk
import sk_inputs as si

DEV = "cuda:0"
D, PAGE = 128, 16


def seen_rows(n, q, window, sinks):
    """[q, n] bool: the rows that each token of a sequence of n rows sees."""
    own = n - q + torch.arange(q)[:, None]
    r = torch.arange(n)[None, :]
    return (r <= own) & ((r < sinks) | (r > own - window))


def batch(lens, qs, hq, hkv, fp8, seed, window, sinks, gain=1.0, forget=True):
    """Device tensors of a batch.  Every row that no token sees holds NaN, in blocks of no sequence too; with `forget`
    the table entries of pages that no token sees name no block, or another's."""
    w = si.make_workload("t", lens, qs, hq, hkv, seed, kv_dtype=si.KV_FP8 if fp8 else si.KV_BF16,
                         k_scale=0.5 if fp8 else 1.0, v_scale=0.25 if fp8 else 1.0, causal=1, spare_blocks=5)
    kv = si.make_kv(w, DEV)
    si.fill_unused_blocks(w, kv)
    bt = torch.as_tensor(w.block_table.copy())
    raw = kv.view(torch.uint8) if fp8 else kv.view(torch.int16)
    for s in range(w.bs):
        n, q = int(w.seq_lens[s]), int(w.q_lens[s])
        unseen = ~seen_rows(n, q, window, sinks).any(0) if q else torch.ones(n, dtype=torch.bool)
        r = unseen.nonzero()[:, 0]
        raw[bt[s, r // PAGE].long().to(DEV), :, (r % PAGE).to(DEV)] = 0x7F if fp8 else 0x7FC0
        for pg in range((n + PAGE - 1) // PAGE if forget else 0):
            if bool(unseen[pg * PAGE:(pg + 1) * PAGE].all()):
                bt[s, pg] = (-1, 1 << 30, -(1 << 31), 0)[pg % 4]
    return dict(w=w, q=si.make_q(w, DEV) * gain, kv=kv, bt=bt.to(DEV), table=torch.as_tensor(w.block_table, device=DEV),
                lens=torch.as_tensor(w.seq_lens, device=DEV), cu=torch.as_tensor(w.cu_q, device=DEV), window=window,
                sinks=sinks)


def rows_of(b, s, h, rows, part):
    """K (part 0) or V (part 1) of some rows of one sequence and head, in 64 bits."""
    w = b["w"]
    x = b["kv"][b["table"][s].long()[rows // PAGE], h, rows % PAGE, part * D:(part + 1) * D]
    if w.kv_dtype == si.KV_FP8:
        return x.view(torch.float8_e4m3fn).double() * (w.v_scale if part else w.k_scale)
    return x.double()


def reference(b, gone=()):
    """out, lse in 64 bits and the bounds of both; keys `gone` of every sequence have the weight 0."""
    w = b["w"]
    g = w.group
    out = torch.zeros(w.num_tokens, w.num_q_heads, D, dtype=torch.float64, device=DEV)
    lse = torch.full((w.num_tokens, w.num_q_heads), -math.inf, dtype=torch.float64, device=DEV)
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    for s in range(w.bs):
        n, q, a = int(w.seq_lens[s]), int(w.q_lens[s]), int(w.cu_q[s])
        see = seen_rows(n, q, b["window"], b["sinks"])
        rows = see.any(0).nonzero()[:, 0].to(DEV)
        if q == 0 or rows.numel() == 0:
            continue
        drop = torch.isin(rows, torch.tensor(list(gone), dtype=torch.int64, device=DEV))
        hide = ~see.to(DEV)[:, rows] | drop[None]
        for h in range(w.num_kv_heads):
            k, v = rows_of(b, s, h, rows, 0), rows_of(b, s, h, rows, 1)
            k = torch.where(drop[:, None], 0.0, k)
            x = b["q"][a:a + q, h * g:(h + 1) * g].double()
            sc = torch.einsum("tgd,nd->tgn", x, k) * w.sm_scale
            e = 130 * 2.0 ** -24 * w.sm_scale * torch.einsum("tgd,nd->tgn", x.abs(), k.abs()).amax(2) + 2.0 ** -20
            if w.kv_dtype == si.KV_FP8:
                top = x.abs().amax(2, keepdim=True)
                small = (x.abs() < 2.0 ** -8 * top).double()
                e = e + w.sm_scale * 2.0 ** -17 * top[..., 0] * torch.einsum("tgd,nd->tgn", small, k.abs()).amax(2)
            sc.masked_fill_(hide[:, None, :], -math.inf)
            p = torch.nan_to_num(torch.softmax(sc, 2))
            ref, l = torch.einsum("tgn,nd->tgd", p, v), torch.logsumexp(sc, 2)
            out[a:a + q, h * g:(h + 1) * g], lse[a:a + q, h * g:(h + 1) * g] = ref, l
            tol_l[a:a + q, h * g:(h + 1) * g] = e + 2.0 ** -22 * l.abs().nan_to_num(posinf=0)
            tol_o[a:a + q, h * g:(h + 1) * g] = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2 * e)[..., None] * \
                torch.einsum("tgn,nd->tgd", p, v.abs())
            if w.kv_dtype == si.KV_FP8:
                tol_o[a:a + q, h * g:(h + 1) * g] += 2.0 ** -33 * ((~hide).double() @ v.abs())[:, None, :]
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
    args = dict(window=b["window"], sinks=b["sinks"], max_q_len=max(1, w.max_q_len), sm_scale=w.sm_scale,
                k_scale=w.k_scale, v_scale=w.v_scale)
    args.update(kw)
    nt, hq = w.num_tokens, w.num_q_heads
    out = torch.full((nt, hq, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    lse = torch.full((nt, hq), float("nan"), device=DEV)
    sk.paged_window_attention(b["q"], b["kv"], b["bt"], b["lens"], b["cu"], out=out, lse=lse, **args)
    torch.cuda.synchronize()
    return out, lse
