"""The cache operators beside decode attention, as they are measured.

Five operators of one serving loop over standard KV pages ([num_blocks, H_kv, 16, 2 * 128], bf16 or
OCP e4m3fn): the rotary positions with the KV write, attention of a chunk of new tokens over the paged
cache, the attention weight that each cached key has gathered, and the two steps of an eviction by that
weight (which rows stay, and the move of the rows that stay into the places of those that go).

`run` computes each of them in plain torch (`own` false) or through the framework's calls (`own` true);
`exact` gives the definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

D = 128
PAGE = 16
DEV = "cuda"
SPARE = 8           # blocks that no sequence uses; the last one takes a plain form's skipped writes
SCORES = 4_900_000_000   # largest padded score array of a plain form (elements)


# ---------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one verify step's 64 query tokens (16 sequences x 4): a few microseconds, latency counts
        dict(name="rope_verify_step", op="rope", nt=64, hq=32, hkv=2, rot=128, inter=False, fp8=False, far=119000,
             track=False),
        # a prefill chunk quantised on its way into e4m3 pages, half of each head rotated, pairs interleaved,
        # far positions, with the eviction state set up beside the pages
        dict(name="rope_chunk_e4m3", op="rope", nt=8191, hq=32, hkv=8, rot=64, inter=True, fp8=True, far=900000,
             track=True),
        # 24 whole prompts of 1 to 2000 tokens, nothing cached before them
        dict(name="prefill_prompts", op="prefill", bs=24, q=2000, ctx=0, ragged=True, hq=16, hkv=2, fp8=False,
             causal=True, mix=1),
        # one chunk of a long prompt over a cache of 32 k keys: the largest product
        dict(name="prefill_chunk_32k", op="prefill", bs=1, q=4096, ctx=32768, ragged=False, hq=32, hkv=8, fp8=False,
             causal=True, mix=2),
        # a short follow-up question on two long conversations: few rows, long axis
        dict(name="prefill_followup_110k", op="prefill", bs=2, q=33, ctx=110000, ragged=True, hq=32, hkv=2,
             fp8=False, causal=True, mix=3),
        # chunks of four prompts on e4m3 pages
        dict(name="prefill_chunk_e4m3", op="prefill", bs=4, q=1024, ctx=16000, ragged=True, hq=16, hkv=2, fp8=True,
             causal=True, mix=4),
        # the weights of a verify step over 16 x 119k keys: the K half of the cache read once
        dict(name="accum_verify_16x119k", op="accum", bs=16, q=4, ctx=118996, ragged=False, hq=32, hkv=2, fp8=False,
             causal=True, mix=5),
        # the weights that a prompt's chunk gives to the keys before and inside it, on e4m3 pages
        dict(name="accum_chunk_e4m3", op="accum", bs=2, q=1500, ctx=20000, ragged=True, hq=16, hkv=2, fp8=True,
             causal=True, mix=6),
        # every step of a bounded cache: a verify step's four rows over the budget
        dict(name="select_step", op="select", bs=16, len=2052, ragged=False, hkv=2, budget=2048, recent=256, mix=7),
        # a long prompt cut down to its budget after its prefill
        dict(name="select_248k", op="select", bs=4, len=248000, ragged=True, hkv=8, budget=32768, recent=2048,
             mix=8),
        # the same step's rows moved: a few rows for each head
        dict(name="move_step", op="move", bs=16, len=2052, ragged=False, hkv=2, budget=2048, recent=256, fp8=False,
             mix=9),
        # the rows of long prompts moved together after their prefill
        dict(name="move_32k", op="move", bs=8, len=32000, ragged=True, hkv=8, budget=8192, recent=512, fp8=False,
             mix=10),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "prefill", "prefill", "accum", "accum", "select", "move"])
    hq, hkv = rng.choice([(8, 1), (16, 2), (32, 2), (32, 8), (16, 16), (12, 4), (5, 1), (40, 8)])
    mix = rng.randrange(1 << 20)
    fp8 = rng.random() < 0.4
    if op == "rope":
        return dict(op=op, nt=_log(rng, 1, 8191), hq=min(hq, 32), hkv=hkv if hq <= 32 else 8,
                    rot=rng.choice([32, 64, 96, 128]), inter=rng.random() < 0.5, fp8=fp8,
                    far=_log(rng, 64, 900000), track=rng.random() < 0.5)
    if op in ("prefill", "accum"):
        while True:
            bs = _log(rng, 1, 24)
            q = _log(rng, 1, 4096)
            ctx = _log(rng, 1, 110000) - 1
            pairs = bs * hq * q * (ctx + q)
            # no more than the largest listed case of the operator, and a plain form that fits
            most = 4096 * 32 * (32768 + 2048) if op == "prefill" else 2 * 1500 * 16 * 21500
            kv = bs * (ctx + q) * hkv
            if pairs <= min(SCORES, most) and kv <= 16 * 119000 * 2:
                break
        return dict(op=op, bs=bs, q=q, ctx=ctx, ragged=rng.random() < 0.7, hq=hq, hkv=hkv, fp8=fp8,
                    causal=rng.random() < 0.8, mix=mix)
    while True:
        bs = _log(rng, 1, 64)
        length = _log(rng, 64, 248000)
        rows = bs * length * hkv
        if rows <= (4 * 200000 * 8 if op == "select" else 8 * 28000 * 8):
            break
    budget = max(16, min(length - 1, _log(rng, 16, length)))
    recent = rng.randrange(0, budget // 2 + 1)
    c = dict(op=op, bs=bs, len=length, ragged=rng.random() < 0.5, hkv=hkv, budget=budget, recent=recent, mix=mix)
    if op == "move":
        c["fp8"] = fp8
    return c


def lengths(case):
    """(cache lengths with this step's tokens, query lengths) of a prefill or accum case."""
    r = random.Random(case["mix"])
    bs, q, ctx = case["bs"], case["q"], case["ctx"]
    if not case["ragged"]:
        return [ctx + q] * bs, [q] * bs
    qs = [max(1, int(round(q * r.uniform(0.0, 1.0)))) for _ in range(bs)]
    qs[r.randrange(bs)] = q
    cs = [int(round(ctx * r.uniform(0.3, 1.0))) for _ in range(bs)]
    return [c + n for c, n in zip(cs, qs)], qs


def row_lengths(case):
    """Cache lengths of a select or move case."""
    r = random.Random(case["mix"])
    if not case["ragged"]:
        return [case["len"]] * case["bs"]
    out = [max(1, int(round(case["len"] * r.uniform(0.4, 1.0)))) for _ in range(case["bs"])]
    out[0] = case["len"]
    return out


# --------------------------------------------------------------------------------- the inputs
def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32)


def _table(lens, seed):
    """Block table from a permutation of every block; unused entries hold -1. Returns it and the block count."""
    pages = [(n + PAGE - 1) // PAGE for n in lens]
    nb = sum(pages) + SPARE
    perm = np.random.default_rng(seed).permutation(nb - 1).astype(np.int32)   # the last block stays unused
    bt = np.full((len(lens), max(1, max(pages))), -1, np.int32)
    k = 0
    for s, n in enumerate(pages):
        bt[s, :n] = perm[k:k + n]
        k += n
    return torch.from_numpy(bt).to(DEV), nb


def _pages(gen, nb, hkv, fp8, ks, vs):
    if not fp8:
        out = torch.empty((nb, hkv, PAGE, 2 * D), dtype=torch.bfloat16, device=DEV)
    else:
        out = torch.empty((nb, hkv, PAGE, 2 * D), dtype=torch.float8_e4m3fn, device=DEV)
    inv = torch.ones(2 * D, device=DEV)
    if fp8:
        inv[:D] = 1.0 / ks
        inv[D:] = 1.0 / vs
    step = max(1, (1 << 27) // (hkv * PAGE * 2 * D))
    for b in range(0, nb, step):
        x = _randn(gen, min(step, nb - b), hkv, PAGE, 2 * D)
        out[b:b + step] = ((x * inv).clamp_(-448, 448) if fp8 else x).to(out.dtype)
    return out


def _poison_tails(pages, bt, lens):
    """NaN in the rows past a sequence's end in its last page: nothing may read them into a result."""
    last = [(s, n) for s, n in enumerate(lens) if n % PAGE]
    if not last:
        return
    blk = bt.cpu().numpy()
    b = torch.tensor([int(blk[s, n // PAGE]) for s, n in last], device=DEV)
    at = torch.tensor([n % PAGE for _, n in last], device=DEV)
    dead = torch.arange(PAGE, device=DEV)[None, :] >= at[:, None]
    raw = pages.view(torch.uint8 if pages.element_size() == 1 else torch.int16)
    nan = 0x7F if pages.element_size() == 1 else 0x7FC0
    raw[b] = raw[b].masked_fill_(dead[:, None, :, None], nan)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    c = case
    st = dict(case=case)
    if c["op"] == "rope":
        nt, hq, hkv, fp8 = c["nt"], c["hq"], c["hkv"], c["fp8"]
        st["ks"], st["vs"] = (0.03, 0.02) if fp8 else (1.0, 1.0)
        nb = (nt + PAGE - 1) // PAGE + SPARE
        st["pages"] = _pages(gen, nb, hkv, fp8, st["ks"], st["vs"])
        # one projection's output, of which q, k and v are views
        qkv = _randn(gen, nt, (hq + 2 * hkv) * D).to(torch.bfloat16)
        st["q"] = qkv[:, :hq * D].view(nt, hq, D)
        st["k"] = qkv[:, hq * D:(hq + hkv) * D].view(nt, hkv, D)
        st["v"] = qkv[:, (hq + hkv) * D:].view(nt, hkv, D)
        rng = np.random.default_rng(seed)
        slots = rng.permutation((nb - 1) * PAGE)[:nt].astype(np.int64)
        if nt > 8:
            slots[rng.integers(0, nt, size=nt // 8)] = -1          # padding tokens without a slot
        st["slots"] = torch.from_numpy(slots).to(DEV)
        st["pos"] = torch.from_numpy(rng.integers(0, c["far"] + 1, size=nt).astype(np.int64)).to(DEV)
        half = c["rot"] // 2
        st["freqs"] = 500000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)
        st["factor"] = 1.0 if not c["inter"] else 1.1386294361119891       # 0.1 ln(4) + 1
        st["q_out"] = torch.empty((nt, hq, D), dtype=torch.bfloat16, device=DEV)
        st["acc"] = _randn(gen, nb, hkv, PAGE).abs() if c["track"] else None
        st["pos_pages"] = torch.full((nb, hkv, PAGE), -1, dtype=torch.int32, device=DEV) if c["track"] else None
        return st
    if c["op"] in ("prefill", "accum"):
        lens, qs = lengths(c)
        fp8, hq, hkv = c["fp8"], c["hq"], c["hkv"]
        st["ks"], st["vs"] = (0.5, 0.25) if fp8 else (1.0, 1.0)
        st["bt"], nb = _table(lens, seed)
        st["pages"] = _pages(gen, nb, hkv, fp8, st["ks"], st["vs"])
        _poison_tails(st["pages"], st["bt"], lens)
        st["q"] = _randn(gen, sum(qs), hq, D).to(torch.bfloat16)
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        st["cu"] = torch.tensor([0] + list(np.cumsum(qs)), dtype=torch.int32, device=DEV)
        st["max_q"], st["max_len"] = max(qs), max(lens)
        st["scale"] = 1.0 / math.sqrt(D)
        st["ws"] = {}
        if c["op"] == "accum":
            st["lse"] = _lse_of(st)
            st["acc"] = torch.rand(nb, hkv, PAGE, generator=gen, device=DEV) * 1e-3
        return st
    lens = row_lengths(c)
    hkv, bs = c["hkv"], c["bs"]
    st["bt"], nb = _table(lens, seed)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    st["max_len"] = max(lens)
    # weights with the heavy tail that attention gives, and exact zeros among them (keys never looked at)
    acc = torch.exp(_randn(gen, nb, hkv, PAGE) * 2.0)
    st["acc"] = acc.masked_fill_(torch.rand(nb, hkv, PAGE, generator=gen, device=DEV) < 0.02, 0.0)
    # positions: rows are in no order after earlier evictions
    pos = torch.full((nb * PAGE, hkv), -1, dtype=torch.int32, device=DEV)
    used = st["bt"].repeat_interleave(PAGE, dim=1).to(torch.int64) * PAGE \
        + torch.arange(PAGE, device=DEV).repeat(st["bt"].shape[1])[None, :]
    for s, n in enumerate(lens):
        order = torch.argsort(torch.rand(hkv, n, generator=gen, device=DEV), dim=1)
        pos[used[s, :n]] = (order.to(torch.int32) + 1000).t().contiguous()
    st["pos_pages"] = pos.view(nb, PAGE, hkv).permute(0, 2, 1).contiguous()
    st["next_pos"] = st["lens"] + 1000
    cap = max(1, min(c["budget"], max(lens) - c["budget"])) if max(lens) > c["budget"] else 1
    st["src"] = torch.full((bs, hkv, cap), -1, dtype=torch.int32, device=DEV)
    st["dst"] = torch.full((bs, hkv, cap), -1, dtype=torch.int32, device=DEV)
    st["counts"] = torch.zeros((bs, hkv), dtype=torch.int32, device=DEV)
    st["new_lens"] = torch.zeros(bs, dtype=torch.int32, device=DEV)
    if c["op"] == "move":
        st["pages"] = _pages(gen, nb, hkv, c["fp8"], 1.0, 1.0)
        _plain_select(st)                    # the lists that the select step hands to the move
    return st


# ----------------------------------------------------------------------------- the plain forms
def _plain_rope(st):
    c = st["case"]
    rot, half = c["rot"], c["rot"] // 2
    ang = st["pos"].to(torch.float64)[:, None] * st["freqs"][None, :]      # 64 bits: far positions
    cos = (torch.cos(ang) * st["factor"]).float()[:, None, :]
    sin = (torch.sin(ang) * st["factor"]).float()[:, None, :]

    def turned(x):
        x = x.float()
        r = x[..., :rot]
        if c["inter"]:
            a, b = r[..., 0::2], r[..., 1::2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
        else:
            a, b = r[..., :half], r[..., half:]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
        return torch.cat([y, x[..., rot:]], dim=-1)

    st["q_out"].copy_(turned(st["q"]))
    pages = st["pages"]
    k, v = turned(st["k"]) / st["ks"], st["v"].float() / st["vs"]
    if pages.element_size() == 1:
        k, v = k.clamp(-448, 448), v.clamp(-448, 448)
    new = torch.cat([k, v], dim=-1).to(pages.dtype)
    raw = pages.view(torch.uint8 if pages.element_size() == 1 else torch.int16)
    skip = st["slots"] < 0
    at = torch.where(skip, pages.shape[0] * PAGE - 1, st["slots"])         # the unused block's last row
    blk, row = at // PAGE, at % PAGE
    raw[blk, :, row] = torch.where(skip[:, None, None], raw[blk, :, row], new.view(raw.dtype))
    if c["track"]:
        acc, pp = st["acc"], st["pos_pages"]
        acc[blk, :, row] = torch.where(skip[:, None], acc[blk, :, row], torch.zeros_like(acc[blk, :, row]))
        pp[blk, :, row] = torch.where(skip[:, None], pp[blk, :, row], st["pos"].to(torch.int32)[:, None])
        return [st["q_out"], pages, acc, pp]
    return [st["q_out"], pages]


def _gather(st, lo, hi, scale):
    """Columns [lo, hi) of every sequence's rows in 32 bits, [bs, H_kv, rows, hi - lo], zero past its end."""
    bt, pages = st["bt"], st["pages"]
    x = pages[bt.clamp(min=0).to(torch.int64)][..., lo:hi].float() * scale  # [bs, n, H, 16, .]
    x = x.permute(0, 2, 1, 3, 4).flatten(2, 3)
    live = torch.arange(x.shape[2], device=DEV)[None, :] < st["lens"][:, None]
    return torch.where(live[:, None, :, None], x, torch.zeros((), device=DEV))


def _plain_scores(st):
    """Scores of the padded batch [bs, H_kv, max_q, G, keys], -inf where a row does not see a key; and the
    token of each (sequence, j), and which of them exist."""
    c = st["case"]
    cu, lens, q = st["cu"].to(torch.int64), st["lens"].to(torch.int64), st["q"]
    hkv = c["hkv"]
    g = c["hq"] // hkv
    qn = cu[1:] - cu[:-1]
    j = torch.arange(st["max_q"], device=DEV)
    there = j[None, :] < qn[:, None]
    tok = torch.where(there, cu[:-1, None] + j[None, :], 0)
    qp = q[tok].float().view(len(lens), st["max_q"], hkv, g, D).permute(0, 2, 1, 3, 4)
    k = _gather(st, 0, D, st["ks"])
    s = torch.matmul(qp.flatten(2, 3), k.transpose(2, 3)).mul_(st["scale"])
    s = s.view(s.shape[0], hkv, st["max_q"], g, -1)
    p = torch.arange(s.shape[-1], device=DEV)
    limit = lens[:, None] - (qn[:, None] - j[None, :] - 1) * (1 if c["causal"] else 0)
    limit = torch.minimum(limit, lens[:, None])
    hidden = (p[None, None, :] >= limit[:, :, None]) | ~there[:, :, None]
    return s.masked_fill_(hidden[:, None, :, None, :], -math.inf), tok, there


def _lse_of(st):
    s, tok, there = _plain_scores(st)
    lse = torch.logsumexp(s, dim=-1)                                       # [bs, H, max_q, G]
    return _to_tokens(lse.permute(0, 2, 1, 3).flatten(2), st).contiguous()


def _to_tokens(x, st):
    """[bs, max_q, ...] back to [tokens, ...]."""
    cu = st["cu"].to(torch.int64)
    t = torch.arange(st["q"].shape[0], device=DEV)
    s = torch.searchsorted(cu, t, right=True) - 1
    return x[s, t - cu[s]]


def _plain_prefill(st):
    s, tok, there = _plain_scores(st)
    m = s.amax(dim=-1, keepdim=True)
    m0 = torch.where(torch.isinf(m), 0.0, m)
    p = s.sub_(m0).exp_()
    l = p.sum(dim=-1, keepdim=True)
    v = _gather(st, D, 2 * D, st["vs"])
    o = torch.matmul(p.flatten(2, 3), v).view(*p.shape[:-1], D)
    o = torch.where(l > 0, o / l, 0.0)
    lse = torch.where(l > 0, m0 + torch.log(l), -math.inf)[..., 0]
    out = _to_tokens(o.permute(0, 2, 1, 3, 4).flatten(2, 3), st).to(torch.bfloat16)
    return [out, _to_tokens(lse.permute(0, 2, 1, 3).flatten(2), st)]


def _plain_accum(st):
    s, tok, there = _plain_scores(st)
    c = st["case"]
    lse = st["lse"][tok].view(s.shape[0], s.shape[2], c["hkv"], -1).permute(0, 2, 1, 3)[..., None]
    w = torch.where(torch.isinf(lse), 0.0, s.sub_(torch.where(torch.isinf(lse), 0.0, lse)).exp_())
    w = w.sum(dim=(2, 3))                                                  # [bs, H, keys]
    acc, bt = st["acc"], st["bt"]
    w = w.view(w.shape[0], w.shape[1], -1, PAGE).permute(0, 2, 1, 3)       # [bs, pages, H, 16]
    blk = torch.where(bt >= 0, bt, acc.shape[0] - 1).to(torch.int64)       # the unused block takes zeros
    acc.index_put_((blk.flatten(),), torch.where((bt >= 0)[..., None, None], w, 0.0).flatten(0, 1), accumulate=True)
    return [acc]


def _plain_select(st):
    c = st["case"]
    bt = st["bt"]
    blk = bt.clamp(min=0).to(torch.int64)
    lens, budget = st["lens"].to(torch.int64), c["budget"]
    acc = st["acc"][blk].permute(0, 2, 1, 3).flatten(2)                    # [bs, H, rows]
    pos = st["pos_pages"][blk].permute(0, 2, 1, 3).flatten(2)
    rows = acc.shape[2]
    r = torch.arange(rows, device=DEV)
    live = (r[None, :] < lens[:, None])[:, None, :].expand_as(acc)
    near = pos >= (st["next_pos"] - c["recent"])[:, None, None]
    # a row's key: past the end, then the rest by weight, then the recent ones; ties to the lowest row
    key = torch.where(near, math.inf, torch.nan_to_num(acc, nan=-math.inf, posinf=3.4e38))
    key = torch.where(live, key.double(), -math.inf)
    key = torch.where(live & torch.isinf(key) & (key < 0), -1e300, key)
    order = torch.sort(key, dim=2, descending=True, stable=True).indices
    stays = torch.zeros_like(live).scatter(2, order, (r < budget).expand_as(order)) & live
    over = (lens > budget)[:, None, None]
    hole = live & ~stays & (r < budget) & over
    tail = stays & (r >= budget) & over
    cap = st["src"].shape[2]

    def listed_in(mask, out):
        at = torch.where(mask, torch.cumsum(mask, 2) - 1, cap)             # place `cap` takes the others
        wide = torch.cat([out, out[..., :1]], dim=2)
        wide.scatter_(2, at, r.to(torch.int32).expand_as(mask).contiguous())
        out.copy_(wide[..., :cap])

    listed_in(hole, st["dst"])
    listed_in(tail, st["src"])
    st["counts"].copy_(tail.sum(2))
    st["new_lens"].copy_(torch.minimum(lens, torch.full_like(lens, budget)))
    return [st["src"], st["dst"], st["counts"], st["new_lens"]]


def _plain_move(st):
    src, dst = st["src"].to(torch.int64), st["dst"].to(torch.int64)
    bs, hkv, cap = src.shape
    there = torch.arange(cap, device=DEV) < st["counts"][..., None]
    bt = st["bt"].to(torch.int64)
    s = torch.arange(bs, device=DEV)[:, None, None]
    h = torch.arange(hkv, device=DEV)[None, :, None].expand_as(src)
    spare = st["acc"].shape[0] - 1                                         # the unused block's row, onto itself

    def place(row):
        row = torch.where(there, row, 0)
        return torch.where(there, bt[s, row // PAGE], spare), h, torch.where(there, row % PAGE, PAGE - 1)

    a, b = place(src), place(dst)
    raw = st["pages"].view(torch.uint8 if st["pages"].element_size() == 1 else torch.int16)
    raw[b] = raw[a]
    st["acc"][b] = st["acc"][a]
    st["pos_pages"][b] = st["pos_pages"][a]
    return [st["pages"], st["acc"], st["pos_pages"]]


# -------------------------------------------------------------------------------- one pass
def run(state):
    st, c = state, state["case"]
    if not own:
        return {"rope": _plain_rope, "prefill": _plain_prefill, "accum": _plain_accum, "select": _plain_select,
                "move": _plain_move}[c["op"]](st)
    import paged_split_kv_gb300 as sk
    if c["op"] == "rope":
        sk.sk_rope_and_cache(st["q"], st["k"], st["v"], st["pos"], st["freqs"], st["slots"], st["pages"],
                             st["q_out"], interleaved=c["inter"], attn_factor=st["factor"], k_scale=st["ks"],
                             v_scale=st["vs"], acc_pages=st["acc"], pos_pages=st["pos_pages"])
        return [st["q_out"], st["pages"]] + ([st["acc"], st["pos_pages"]] if c["track"] else [])
    if c["op"] == "prefill":
        out, lse = sk.paged_prefill_attention(st["q"], st["pages"], st["bt"], st["lens"], st["cu"],
                                              max_q_len=st["max_q"], max_seq_len=st["max_len"],
                                              sm_scale=st["scale"], k_scale=st["ks"], v_scale=st["vs"],
                                              causal=c["causal"], workspace=st["ws"])
        return [out, lse]
    if c["op"] == "accum":
        sk.sk_accum_attn_weights(st["q"], st["pages"], st["bt"], st["lens"], st["cu"], st["lse"], st["acc"],
                                 max_q_len=st["max_q"], sm_scale=st["scale"], k_scale=st["ks"],
                                 causal=c["causal"], workspace=st["ws"])
        return [st["acc"]]
    if c["op"] == "select":
        sk.sk_evict_select(st["acc"], st["pos_pages"], st["bt"], st["lens"], st["next_pos"], st["src"], st["dst"],
                           st["counts"], st["new_lens"], budget=c["budget"], recent=c["recent"],
                           max_seq_len=st["max_len"])
        return [st["src"], st["dst"], st["counts"], st["new_lens"]]
    sk.sk_evict_move(st["src"], st["dst"], st["counts"], st["bt"], st["pages"], st["acc"], st["pos_pages"])
    return [st["pages"], st["acc"], st["pos_pages"]]


# ---------------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "rope":
        nt, el = c["nt"], 1 if c["fp8"] else 2
        b = nt * c["hq"] * D * 4 + nt * c["hkv"] * 2 * D * (2 + el) + nt * 16 + (nt * c["hkv"] * 8 if c["track"] else 0)
        return {"bytes": b, "flops": 3 * nt * (c["hq"] + c["hkv"]) * c["rot"]}
    if c["op"] in ("prefill", "accum"):
        lens, qs = lengths(c)
        pairs = sum(q * n - (q * (q - 1) // 2 if c["causal"] else 0) for n, q in zip(lens, qs))
        el = 1 if c["fp8"] else 2
        keys, nt = sum(lens) * c["hkv"], sum(qs) * c["hq"]
        if c["op"] == "prefill":
            return {"bytes": keys * 2 * D * el + nt * (4 * D + 4), "flops": 4 * D * c["hq"] * pairs}
        return {"bytes": keys * (D * el + 8) + nt * (2 * D + 4), "flops": 2 * D * c["hq"] * pairs}
    lens = row_lengths(c)
    # rows that move, if the rows that stay lie anywhere
    moved = sum(c["budget"] * (n - c["budget"]) / n for n in lens if n > c["budget"]) * c["hkv"]
    if c["op"] == "select":
        return {"bytes": sum(lens) * c["hkv"] * 8 + moved * 8, "flops": sum(lens) * c["hkv"]}
    return {"bytes": moved * (2 * (2 * D * (1 if c["fp8"] else 2) + 8) + 8), "flops": 0}


# --------------------------------------------------------------------- the definitions in 64 bits
def _exact_rows(st, s, h, part):
    """K (part 0) or V (part 1) of sequence s and head h in 64 bits, [L, 128]."""
    n = int(st["lens"][s])
    r = torch.arange(n, device=DEV)
    b = st["bt"][s].long()[r // PAGE]
    x = st["pages"][b, h, r % PAGE, part * D:(part + 1) * D].double()
    return x * (st["ks"] if part == 0 else st["vs"])


def exact(case, seed):
    st = prepare(case, seed)
    c = case
    if c["op"] == "rope":
        nt = c["nt"]
        rad = torch.outer(st["pos"].double(), st["freqs"])
        turn = torch.polar(torch.full_like(rad, st["factor"]), rad)[:, None, :]
        n = c["rot"] // 2

        def rotated(x):
            x = x.double().clone()
            even = slice(0, c["rot"], 2) if c["inter"] else slice(0, n)
            odd = slice(1, c["rot"], 2) if c["inter"] else slice(n, c["rot"])
            z = torch.complex(x[..., even].contiguous(), x[..., odd].contiguous()) * turn
            x[..., even], x[..., odd] = z.real, z.imag
            return x

        pages = st["pages"].double()
        q, k, v = rotated(st["q"]), rotated(st["k"]) / st["ks"], st["v"].double() / st["vs"]
        ok = (st["slots"] >= 0).nonzero()[:, 0]
        slot = st["slots"][ok]
        pages[slot // PAGE, :, slot % PAGE, :D] = k[ok]
        pages[slot // PAGE, :, slot % PAGE, D:] = v[ok]
        if not c["track"]:
            return [q, pages]
        acc = st["acc"].double()
        acc[slot // PAGE, :, slot % PAGE] = 0.0
        return [q, pages, acc, None]
    if c["op"] in ("prefill", "accum"):
        g = c["hq"] // c["hkv"]
        cu = st["cu"].tolist()
        nt = cu[-1]
        out = torch.zeros(nt, c["hq"], D, dtype=torch.float64, device=DEV)
        lse = torch.full((nt, c["hq"]), -math.inf, dtype=torch.float64, device=DEV)
        acc = st["acc"].double() if c["op"] == "accum" else None
        for s, n in enumerate(st["lens"].tolist()):
            a, b = cu[s], cu[s + 1]
            seen = torch.full((b - a,), n, device=DEV)
            if c["causal"]:
                seen = (n - (b - a) + 1 + torch.arange(b - a, device=DEV)).clamp(0, n)
            hide = torch.arange(n, device=DEV)[None, :] >= seen[:, None]
            rows = torch.arange(n, device=DEV)
            blk = st["bt"][s].long()[rows // PAGE]
            for h in range(c["hkv"]):
                k = _exact_rows(st, s, h, 0)
                total = torch.zeros(n, dtype=torch.float64, device=DEV)
                for i in range(h * g, (h + 1) * g):
                    x = (st["q"][a:b, i].double() @ k.t()) * st["scale"]
                    x[hide] = -math.inf
                    if acc is not None:
                        norm = st["lse"][a:b, i].double()[:, None]
                        total += torch.where(norm == -math.inf, 0.0, torch.exp(x - norm)).sum(0)
                        continue
                    lse[a:b, i] = torch.logsumexp(x, dim=1)
                    out[a:b, i] = torch.nan_to_num(torch.softmax(x, dim=1)) @ _exact_rows(st, s, h, 1)
                if acc is not None:
                    acc[blk, h, rows % PAGE] += total
        return [acc] if acc is not None else [out, lse]
    if c["op"] == "select":
        return None
    pages, acc = st["pages"].double(), st["acc"].double()
    counts, src, dst, bt = (st[k].cpu().numpy() for k in ("counts", "src", "dst", "bt"))
    at = [[], [], [], [], []]
    for s in range(c["bs"]):
        for h in range(c["hkv"]):
            m = int(counts[s, h])
            x, y = src[s, h, :m], dst[s, h, :m]
            for col, v in zip(at, (bt[s, x // PAGE], x % PAGE, bt[s, y // PAGE], y % PAGE, np.full(m, h))):
                col.append(v)
    a, ar, b, br, h = (torch.from_numpy(np.concatenate(v).astype(np.int64)).to(DEV) for v in at)
    pages[b, h, br] = pages[a, h, ar]
    acc[b, h, br] = acc[a, h, ar]
    return [pages, acc, None]
