"""Windowed attention with sinks over the paged cache and the rotary write with several axes, as they are measured.

Three operators of serving over standard KV pages ([num_blocks, H_kv, 16, 2 * 128], bf16 or OCP e4m3fn):
attention that sees the last `window` keys and the first `sinks` ones, for a step of one or a few tokens a sequence
and for chunks of prompts, and the KV write whose rotary positions have several axes (time, height, width).

`run` computes each in plain torch (`own` false) or through the framework's calls (`own` true); `exact` gives
the definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

D = 128
PAGE = 16
DEV = "cuda"
SPARE = 8                # blocks that no sequence uses; the last one takes a plain form's skipped writes
SCORES = 4_900_000_000   # largest padded score array of a plain form (elements)


# ---------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one conversation, one token: the smallest step, where latency counts
        dict(name="step_bs1", op="window", bs=1, q=1, ctx=8191, ragged=False, hq=32, hkv=8, fp8=False, window=4096,
             sinks=4, freed=False, mix=1),
        # a server's step: 64 conversations of different lengths, pages behind the window handed back
        dict(name="step_64", op="window", bs=64, q=1, ctx=8191, ragged=True, hq=32, hkv=8, fp8=False, window=1024,
             sinks=4, freed=True, mix=2),
        # a verify step of four drafted tokens on long caches, e4m3 pages, sinks that fill whole pages
        dict(name="step_verify_e4m3", op="window", bs=16, q=4, ctx=118996, ragged=False, hq=32, hkv=2, fp8=True,
             window=4096, sinks=64, freed=True, mix=3),
        # the large decode batch with half of its cache in the window: the most bytes
        dict(name="step_128x4096", op="window", bs=128, q=1, ctx=8191, ragged=False, hq=32, hkv=8, fp8=False,
             window=4096, sinks=4, freed=False, mix=4),
        # 24 whole prompts of 1 to 2000 tokens
        dict(name="chunk_prompts", op="window", bs=24, q=2000, ctx=0, ragged=True, hq=16, hkv=2, fp8=False,
             window=512, sinks=4, freed=False, mix=5),
        # a chunk of a long prompt: the largest products
        dict(name="chunk_32k", op="window", bs=1, q=4096, ctx=32768, ragged=False, hq=32, hkv=8, fp8=False,
             window=4096, sinks=4, freed=True, mix=6),
        # chunks of four prompts on e4m3 pages
        dict(name="chunk_e4m3", op="window", bs=4, q=1024, ctx=16000, ragged=True, hq=16, hkv=2, fp8=True,
             window=2048, sinks=16, freed=True, mix=7),
        # a whole long prompt in a layer with a short window and no sinks: little work per token
        dict(name="chunk_short_window", op="window", bs=1, q=16001, ctx=0, ragged=False, hq=16, hkv=2, fp8=False,
             window=128, sinks=0, freed=False, mix=8),
        # one verify step's 64 tokens: a few microseconds
        dict(name="axes_step", op="axes", nt=64, hq=32, hkv=2, rot=128, axes=3, each=24, cycled=False,
             inter=False, fp8=False, images=False, far=119000, track=False),
        # a chunk of images and text, all dimensions turned in halves, an axis for each run of pairs
        dict(name="axes_images", op="axes", nt=8191, hq=32, hkv=8, rot=128, axes=3, each=24, cycled=False,
             inter=False, fp8=False, images=True, far=30000, track=False),
        # the same on e4m3 pages, axes in turn along the pairs, neighbours paired, with the eviction state beside
        # the pages
        dict(name="axes_images_e4m3", op="axes", nt=8191, hq=32, hkv=8, rot=128, axes=3, each=20, cycled=True,
             inter=True, fp8=True, images=True, far=30000, track=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    hq, hkv = rng.choice([(8, 1), (16, 2), (32, 2), (32, 8), (16, 16), (12, 4), (5, 1), (40, 8)])
    fp8 = rng.random() < 0.4
    kind = rng.choice(["axes", "step", "step", "chunk", "chunk"])
    if kind == "axes":
        rot = rng.choice([32, 64, 96, 128])
        cycled = rng.random() < 0.5
        naxes = rng.choice([2, 3])
        each = rng.randrange(1, rot // 2 // naxes + 1)
        return dict(op="axes", nt=_log(rng, 1, 8191), hq=min(hq, 32), hkv=hkv, rot=rot, axes=naxes, each=each,
                    cycled=cycled, inter=rng.random() < 0.5, fp8=fp8, images=rng.random() < 0.7,
                    far=_log(rng, 64, 900000), track=rng.random() < 0.5)
    while True:
        window = _log(rng, 16, 16384)
        sinks = rng.choice([0, 0, 1, 4, 4, 16, 64, 100])
        if kind == "step":
            bs, q, ctx = _log(rng, 1, 128), rng.choice([1, 1, 2, 3, 4, 7]), _log(rng, 1, 119000) - 1
        else:
            bs, q, ctx = _log(rng, 1, 24), _log(rng, 8, 16000), _log(rng, 1, 110000) - 1
        keys = min(ctx + q, sinks + window + q)
        seen = min(ctx + q, sinks + window)
        # no more than the largest listed cases, a plain form that fits, and a cache that does
        if bs * keys * hkv <= 128 * 4200 * 8 and bs * hq * q * seen <= 4096 * 32 * 4200 and \
                bs * hq * q * keys <= SCORES and bs * (ctx + q) * hkv <= 16 * 119000 * 4:
            break
    return dict(op="window", bs=bs, q=q, ctx=ctx, ragged=rng.random() < 0.7, hq=hq, hkv=hkv, fp8=fp8, window=window,
                sinks=sinks, freed=rng.random() < 0.5, mix=rng.randrange(1 << 20))


def lengths(case):
    """(cache lengths with this step's tokens, query lengths) of a window case."""
    r = random.Random(case["mix"])
    bs, q, ctx = case["bs"], case["q"], case["ctx"]
    if not case["ragged"]:
        return [ctx + q] * bs, [q] * bs
    qs = [max(1, int(round(q * r.uniform(0.0, 1.0)))) for _ in range(bs)]
    qs[r.randrange(bs)] = q
    cs = [int(round(ctx * r.uniform(0.1, 1.0))) for _ in range(bs)]
    return [c + n for c, n in zip(cs, qs)], qs


# --------------------------------------------------------------------------------- the inputs
def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32)


def _pages(gen, nb, hkv, fp8, ks, vs):
    out = torch.empty((nb, hkv, PAGE, 2 * D), dtype=torch.float8_e4m3fn if fp8 else torch.bfloat16, device=DEV)
    inv = torch.ones(2 * D, device=DEV)
    if fp8:
        inv[:D] = 1.0 / ks
        inv[D:] = 1.0 / vs
    step = max(1, (1 << 27) // (hkv * PAGE * 2 * D))
    for b in range(0, nb, step):
        x = _randn(gen, min(step, nb - b), hkv, PAGE, 2 * D)
        out[b:b + step] = ((x * inv).clamp_(-448, 448) if fp8 else x).to(out.dtype)
    return out


def _prepare_window(c, st, gen, seed):
    lens, qs = lengths(c)
    fp8, hq, hkv = c["fp8"], c["hq"], c["hkv"]
    st["ks"], st["vs"] = (0.5, 0.25) if fp8 else (1.0, 1.0)
    pages = [(n + PAGE - 1) // PAGE for n in lens]
    nb = sum(pages) + SPARE
    perm = np.random.default_rng(seed).permutation(nb - 1).astype(np.int32)   # the last block stays unused
    bt = np.full((len(lens), max(pages)), -1, np.int32)
    at = 0
    gone = []
    for s, n in enumerate(pages):
        bt[s, :n] = perm[at:at + n]
        at += n
        if c["freed"]:
            # pages that no token of this step sees have been handed back: their entries are gone
            lo = max(0, lens[s] - qs[s] + 1 - c["window"]) // PAGE
            first = (c["sinks"] + PAGE - 1) // PAGE
            if lo > first:
                gone.append(bt[s, first:lo].copy())
                bt[s, first:lo] = -1
    st["bt"] = torch.from_numpy(bt).to(DEV)
    st["pages"] = _pages(gen, nb, hkv, fp8, st["ks"], st["vs"])
    # NaN in the rows past a sequence's end in its last page, and in some pages that were handed back
    raw = st["pages"].view(torch.uint8 if fp8 else torch.int16)
    nan = 0x7F if fp8 else 0x7FC0
    last = [(s, n) for s, n in enumerate(lens) if n % PAGE]
    if last:
        b = torch.tensor([int(bt[s, n // PAGE]) for s, n in last], device=DEV)
        end = torch.tensor([n % PAGE for _, n in last], device=DEV)
        dead = torch.arange(PAGE, device=DEV)[None, :] >= end[:, None]
        raw[b] = raw[b].masked_fill_(dead[:, None, :, None], nan)
    if gone:
        raw[torch.from_numpy(np.concatenate(gone)[::5].astype(np.int64)).to(DEV)] = nan
    st["q"] = _randn(gen, sum(qs), hq, D).to(torch.bfloat16)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    st["cu"] = torch.tensor([0] + list(np.cumsum(qs)), dtype=torch.int32, device=DEV)
    st["max_q"], st["max_len"] = max(qs), max(lens)
    st["scale"] = 1.0 / math.sqrt(D)
    st["ws"] = {}
    return st


def axis_of_pairs(c):
    """The axis whose position turns each pair, every axis but the first having `each` of them: runs of pairs, or the
    axes in turn until each has its share (what is left at the end belongs to the first)."""
    half, n, each = c["rot"] // 2, c["axes"], c["each"]
    if c["cycled"]:
        return [i % n if i < n * each else 0 for i in range(half)]
    first = half - each * (n - 1)
    return [0 if i < first else 1 + (i - first) // each for i in range(half)]


def _axis_positions(c, seed):
    """[axes, tokens]: text, whose axes agree, and grids of image or video patches, one after the other. After a
    grid the text goes on behind the largest position in it."""
    r = random.Random(seed)
    n, nt = c["axes"], c["nt"]
    if not c["images"]:
        p = np.random.default_rng(seed).integers(0, c["far"] + 1, size=nt)
        return np.repeat(p[None], n, axis=0)
    runs, total = [], 0
    at = r.randrange(0, c["far"] + 1)
    while total < nt:
        words = r.randrange(1, 65)
        runs.append(np.repeat(np.arange(at, at + words)[None], n, axis=0))
        at += words
        grid = [r.randrange(1, 5)] + [r.randrange(4, 41) for _ in range(n - 1)]
        cells = np.stack(np.meshgrid(*[np.arange(g) for g in grid], indexing="ij")).reshape(n, -1) + at
        runs.append(cells)
        at += max(grid)
        total += words + cells.shape[1]
    return np.concatenate(runs, axis=1)[:, :nt]


def _prepare_axes(c, st, gen, seed):
    nt, hq, hkv, fp8 = c["nt"], c["hq"], c["hkv"], c["fp8"]
    st["ks"], st["vs"] = (0.03, 0.02) if fp8 else (1.0, 1.0)
    nb = (nt + PAGE - 1) // PAGE + SPARE
    st["pages"] = _pages(gen, nb, hkv, fp8, st["ks"], st["vs"])
    # one projection's output, of which q, k and v are views
    qkv = _randn(gen, nt, (hq + 2 * hkv) * D).to(torch.bfloat16)
    st["q"] = qkv[:, :hq * D].view(nt, hq, D)
    st["k"] = qkv[:, hq * D:(hq + hkv) * D].view(nt, hkv, D)
    st["v"] = qkv[:, (hq + hkv) * D:].view(nt, hkv, D)
    # a sequence's slots lie page by page in blocks from anywhere; a few tokens are padding without a slot
    rng = np.random.default_rng(seed)
    slots = (rng.permutation(nb - 1)[:, None] * PAGE + np.arange(PAGE)[None]).reshape(-1)[:nt].astype(np.int64)
    if nt > 8:
        slots[rng.integers(0, nt, size=nt // 16)] = -1
    st["slots"] = torch.from_numpy(slots).to(DEV)
    # the runner's buffer of positions is longer than this step
    pos = np.zeros((c["axes"], nt + 3), np.int64)
    pos[:, :nt] = _axis_positions(c, seed)
    st["pos"] = torch.from_numpy(pos).to(DEV)[:, :nt]
    half = c["rot"] // 2
    st["freqs"] = 1000000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)
    st["axes"] = torch.tensor(axis_of_pairs(c), dtype=torch.uint8, device=DEV)
    st["q_out"] = torch.empty((nt, hq, D), dtype=torch.bfloat16, device=DEV)
    st["acc"] = _randn(gen, nb, hkv, PAGE).abs() if c["track"] else None
    st["pos_pages"] = torch.full((nb, hkv, PAGE), -1, dtype=torch.int32, device=DEV) if c["track"] else None
    return st


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return (_prepare_window if case["op"] == "window" else _prepare_axes)(case, dict(case=case), gen, seed)


# ----------------------------------------------------------------------------- the plain forms
def _plain_window(st):
    c = st["case"]
    cu, lens, q = st["cu"].to(torch.int64), st["lens"].to(torch.int64), st["q"]
    hkv, w, sinks = c["hkv"], c["window"], c["sinks"]
    g, bs, mq = c["hq"] // hkv, c["bs"], st["max_q"]
    qn = cu[1:] - cu[:-1]
    # the rows that some token of a sequence sees: the sinks, then from the first token's window on
    lo = (lens - qn + 1 - w).clamp(min=0)
    skip = (lo - sinks).clamp(min=0)                                       # rows between the two
    n = min(st["max_len"], sinks + w + mq)
    i = torch.arange(n, device=DEV)[None, :]
    row = torch.where(i < sinks, i, i + skip[:, None])                     # [bs, n]
    live = row < lens[:, None]
    safe = torch.where(live, row, 0)
    blk = torch.gather(st["bt"], 1, safe // PAGE).to(torch.int64)
    blk = torch.where(live, blk, st["pages"].shape[0] - 1)

    def gathered(part, scale):
        x = st["pages"][..., part * D:(part + 1) * D][blk, :, safe % PAGE].float() * scale     # [bs, n, H, 128]
        return torch.where(live[:, :, None, None], x, 0.0).permute(0, 2, 1, 3)

    j = torch.arange(mq, device=DEV)
    there = j[None, :] < qn[:, None]
    tok = torch.where(there, cu[:-1, None] + j[None, :], 0)
    qp = q[tok].float().view(bs, mq, hkv, g, D).permute(0, 2, 1, 3, 4).flatten(2, 3)
    s = torch.matmul(qp, gathered(0, st["ks"]).transpose(2, 3)).mul_(st["scale"]).view(bs, hkv, mq, g, n)
    at = lens[:, None] - qn[:, None] + j[None, :]                          # each token's own row
    r, at = row[:, None, :], at[:, :, None]
    seen = live[:, None, :] & there[:, :, None] & (r <= at) & ((r < sinks) | (r > at - w))
    s = s.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    m = s.amax(dim=-1, keepdim=True)
    m = torch.where(torch.isinf(m), 0.0, m)
    p = s.sub_(m).exp_()
    l = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), gathered(1, st["vs"])).view(bs, hkv, mq, g, D)
    o = torch.where(l > 0, o / l, 0.0)
    lse = torch.where(l > 0, m + torch.log(l), -math.inf)[..., 0]
    t = torch.arange(q.shape[0], device=DEV)
    of = torch.searchsorted(cu, t, right=True) - 1
    o = o.permute(0, 2, 1, 3, 4).flatten(2, 3)[of, t - cu[of]].to(torch.bfloat16)
    return [o, lse.permute(0, 2, 1, 3).flatten(2)[of, t - cu[of]]]


def _plain_axes(st):
    c = st["case"]
    rot, half = c["rot"], c["rot"] // 2
    pos = st["pos"][st["axes"].to(torch.int64)].t().to(torch.float64)      # [tokens, pairs]
    ang = pos * st["freqs"][None, :]                                       # 64 bits: far positions
    cos, sin = torch.cos(ang).float()[:, None, :], torch.sin(ang).float()[:, None, :]

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
        pp[blk, :, row] = torch.where(skip[:, None], pp[blk, :, row], st["pos"][0].to(torch.int32)[:, None])
        return [st["q_out"], pages, acc, pp]
    return [st["q_out"], pages]


# -------------------------------------------------------------------------------- one pass
def run(state):
    st, c = state, state["case"]
    if not own:
        return (_plain_window if c["op"] == "window" else _plain_axes)(st)
    import paged_split_kv_gb300 as sk
    if c["op"] == "window":
        out, lse = sk.paged_window_attention(st["q"], st["pages"], st["bt"], st["lens"], st["cu"],
                                             window=c["window"], sinks=c["sinks"], max_q_len=st["max_q"],
                                             max_seq_len=st["max_len"], sm_scale=st["scale"], k_scale=st["ks"],
                                             v_scale=st["vs"], workspace=st["ws"])
        return [out, lse]
    sk.sk_rope_axes_and_cache(st["q"], st["k"], st["v"], st["pos"], st["freqs"], st["axes"], st["slots"],
                              st["pages"], st["q_out"], interleaved=c["inter"], k_scale=st["ks"], v_scale=st["vs"],
                              acc_pages=st["acc"], pos_pages=st["pos_pages"])
    return [st["q_out"], st["pages"]] + ([st["acc"], st["pos_pages"]] if c["track"] else [])


# ---------------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "axes":
        nt, el, n = c["nt"], 1 if c["fp8"] else 2, c["axes"]
        b = nt * c["hq"] * D * 4 + nt * c["hkv"] * 2 * D * (2 + el) + nt * 8 * (n + 1) \
            + (nt * c["hkv"] * 8 if c["track"] else 0)
        return {"bytes": b, "flops": 3 * nt * (c["hq"] + c["hkv"]) * c["rot"]}
    lens, qs = lengths(c)
    w, sinks = c["window"], c["sinks"]
    keys = pairs = 0
    for n, q in zip(lens, qs):
        keys += min(n, min(sinks, n) + min(n, w + q - 1))
        # a token sees the rows up to its own, and no more than the sinks and the window hold
        pairs += sum(min(r, sinks + w) for r in range(n - q + 1, n + 1))
    el = 1 if c["fp8"] else 2
    return {"bytes": keys * c["hkv"] * 2 * D * el + sum(qs) * c["hq"] * (4 * D + 4), "flops": 4 * D * c["hq"] * pairs}


# --------------------------------------------------------------------- the definitions in 64 bits
def _exact_window(st, c):
    g = c["hq"] // c["hkv"]
    cu, w, sinks = st["cu"].tolist(), c["window"], c["sinks"]
    out = torch.zeros(cu[-1], c["hq"], D, dtype=torch.float64, device=DEV)
    lse = torch.full((cu[-1], c["hq"]), -math.inf, dtype=torch.float64, device=DEV)
    for s, n in enumerate(st["lens"].tolist()):
        first = n - (cu[s + 1] - cu[s])                    # the first token's own row
        for a in range(cu[s], cu[s + 1], 1024):
            b = min(a + 1024, cu[s + 1])
            mine = first + torch.arange(a - cu[s], b - cu[s], device=DEV)
            lo, hi = max(sinks, int(mine[0]) - w + 1), int(mine[-1]) + 1
            rows = torch.cat([torch.arange(0, min(sinks, hi), device=DEV), torch.arange(lo, max(lo, hi), device=DEV)])
            blk = st["bt"][s].long()[rows // PAGE]
            past = mine[:, None] - rows[None, :]
            hide = (past < 0) | ((past >= w) & (rows >= sinks)[None, :])
            for h in range(c["hkv"]):
                kv = st["pages"][blk, h, rows % PAGE].double()
                k, v = kv[:, :D] * st["ks"], kv[:, D:] * st["vs"]
                x = torch.einsum("tgd,nd->gtn", st["q"][a:b, h * g:(h + 1) * g].double(), k) * st["scale"]
                x[:, hide] = -math.inf
                lse[a:b, h * g:(h + 1) * g] = torch.logsumexp(x, dim=2).t()
                out[a:b, h * g:(h + 1) * g] = torch.einsum("gtn,nd->tgd", torch.softmax(x, dim=2), v)
    return [out, lse]


def _exact_axes(st, c):
    n = c["rot"] // 2
    axis = axis_of_pairs(c)
    rad = torch.stack([st["pos"][a].double() * st["freqs"][i] for i, a in enumerate(axis)], dim=1)
    turn = torch.polar(torch.ones_like(rad), rad)[:, None, :]

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


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_window(st, case) if case["op"] == "window" else _exact_axes(st, case)
