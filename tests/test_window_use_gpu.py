"""Attention with a sliding window and sinks as a server calls it: captured and replayed, on other streams, with workspaces
that are shared and outgrown, on bad tables and offsets, with waits that expire, and after the rotary write with several
axes (bounds: window_helpers)."""
import random
import subprocess
import sys

import pytest
import torch

import paged_split_kv_gb300 as sk
import sk_inputs as si
from window_helpers import DEV, batch, check, reference, run

pytestmark = pytest.mark.gpu

# a cluster of CTAs for each unit, runs of the batch, whole prompts and chunks
CALLS = {"clusters": ([3000, 700, 1500], [2, 1, 3], 16, 2, 600, 4), "runs": ([700, 130, 1] * 40, [1, 2, 1] * 40, 16, 2, 300, 4),
         "chunks": ([1500, 300, 900], [400, 300, 17], 16, 2, 300, 4)}


def args_of(b, **kw):
    w = b["w"]
    return dict(dict(window=b["window"], sinks=b["sinks"], max_q_len=w.max_q_len, sm_scale=w.sm_scale, k_scale=w.k_scale,
                     v_scale=w.v_scale), **kw)


def attend(b, **kw):
    return sk.paged_window_attention(b["q"], b["kv"], b["bt"], b["lens"], b["cu"], **args_of(b, **kw))


def made(name, fp8, seed=3, **kw):
    lens, qs, hq, hkv, window, sinks = CALLS[name]
    return batch(lens, qs, hq, hkv, fp8, seed, window, sinks, **kw)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("name", CALLS)
def test_replayed_with_other_lengths_tables_and_queries(name, fp8):
    """One capture, replayed on what the arrays hold by then: the bits of the call made outside of it."""
    b = made(name, fp8)
    attend(b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = attend(b)
    graph.replay()
    torch.cuda.synchronize()
    check(b, out, lse)
    g = torch.Generator().manual_seed(5)
    full = b["table"].clone()
    for turn in range(3):
        w = b["w"]
        n = torch.tensor([int(torch.randint(0, int(x) + 1, (1,), generator=g)) for x in w.seq_lens], dtype=torch.int32)
        b["lens"].copy_(n)
        b["bt"].copy_(full)
        b["q"].copy_(b["q"].flip(0))
        b["kv"].view(torch.uint8).bitwise_and_(0x3F)       # (rows that had been out of every window: finite now)
        graph.replay()
        want = attend(b)
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert sk.sk_get_device_status() == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_two_graphs_and_calls_between_them_share_a_workspace(fp8):
    ws = {}
    bs = [made(name, fp8, 7) for name in CALLS]
    want = [attend(b) for b in bs]
    graphs = []
    for b in bs:
        attend(b, workspace=ws)                  # (grows: the small one first)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = attend(b, workspace=ws)
        graphs.append((graph, got))
    for order in ((0, 1, 2), (2, 1, 0), (1, 1, 2, 0)):
        for i in order:
            graphs[i][1][0].fill_(3)
            graphs[i][0].replay()
            eager = attend(bs[i - 1], workspace=ws)
            torch.cuda.synchronize()
            assert torch.equal(graphs[i][1][0], want[i][0]) and torch.equal(graphs[i][1][1], want[i][1])
            assert torch.equal(eager[0], want[i - 1][0])
    assert sk.sk_get_device_status() == 0


def test_a_captured_call_after_its_workspace_was_outgrown():
    small, large = made("clusters", True, 81), made("chunks", True, 82)
    ws = {}
    want = attend(small, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = attend(small, workspace=ws)
    before = ws["window"].numel()
    attend(large, workspace=ws)
    assert ws["window"].numel() > before
    held = [torch.full((before,), 0xA5, dtype=torch.uint8, device=DEV) for _ in range(4)]
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert all(bool((t == 0xA5).all()) for t in held)
    again = attend(small, workspace=ws)          # the larger buffer serves the small call as well
    assert torch.equal(again[0], want[0]) and sk.sk_get_device_status() == 0


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("name", CALLS)
def test_on_another_stream(name, given):
    """As the current stream and as an argument; the query comes late on that stream, and the workspace is dropped while
    the call still waits."""
    b = made(name, True, 83)
    want = attend(b)
    ws = {}
    attend(b, workspace=ws)
    q, size = b["q"].clone(), ws["window"].numel()
    b["q"].zero_()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
        b["q"].copy_(q)
        if not given:
            got = attend(b, workspace=ws)
    if given:
        got = attend(b, workspace=ws, stream=side)
    ws.clear()
    held = [torch.full((size,), 0xA5, dtype=torch.uint8, device=DEV) for _ in range(4)]
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert all(bool((t == 0xA5).all()) for t in held) and sk.sk_get_device_status() == 0


def test_two_streams_at_once():
    bs = [made(name, fp8, 84) for name in CALLS for fp8 in (False, True)]
    want = [attend(b) for b in bs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in bs]
    got = [[] for _ in bs]
    for _ in range(5):
        for i, b in enumerate(bs):
            got[i].append(attend(b, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(len(bs)):
        assert all(torch.equal(o, want[i][0]) and torch.equal(l, want[i][1]) for o, l in got[i])
    assert sk.sk_get_device_status() == 0


def test_the_first_call_of_a_process_may_be_a_captured_one():
    code = """
import torch, paged_split_kv_gb300 as sk
sk.sk_get_device_status()
dev = "cuda:0"
q = torch.randn(2, 8, 128, device=dev).bfloat16()
kv = torch.randn(64, 1, 16, 256, device=dev).bfloat16()
bt = torch.arange(60, device=dev, dtype=torch.int32).view(2, 30)
n = torch.full((2,), 480, device=dev, dtype=torch.int32)
cu = torch.arange(3, device=dev, dtype=torch.int32)
def call():
    return sk.paged_window_attention(q, kv, bt, n, cu, window=300, sinks=4, max_q_len=1, sm_scale=0.1)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out, lse = call()
g.replay()
torch.cuda.synchronize()
want = call()
assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and sk.sk_get_device_status() == 0
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("name", CALLS)
def test_bad_blocks_and_lengths_are_reported(name, fp8):
    """What one sequence's table, length or query length has wrong is reported, and leaves the others' results alone."""
    b = made(name, fp8, 17, forget=False)
    w = b["w"]
    ref = reference(b)
    n0, t0 = int(w.q_lens[0]), int(w.cu_q[1])
    for bad in (-1, 1 << 30, int(b["kv"].shape[0])):
        bt = b["bt"].clone()
        b["bt"][0, (int(w.seq_lens[0]) - 1) // 16] = bad
        out, lse = attend(b)
        assert sk.sk_get_device_status(clear=True) == sk.SK_DEV_BAD_BLOCK
        b["bt"].copy_(bt)
        assert bool(((out.double() - ref[0]).abs() <= ref[2] + 1e-30)[t0:].all()) and not torch.isnan(out.float()).any()
    for length in (-1, b["bt"].shape[1] * 16 + 1, 2 ** 31 - 1, -2 ** 31):
        lens = b["lens"].clone()
        lens[0] = length
        out = torch.full((w.num_tokens, w.num_q_heads, 128), 3.0, dtype=torch.bfloat16, device=DEV)
        sk.sk_paged_window_attn(b["q"], b["kv"], b["bt"], lens, b["cu"], out, **args_of(b))
        assert sk.sk_get_device_status(clear=True) == sk.SK_DEV_BAD_SEQ
        assert bool((out[:n0] == 3).all()) and bool(((out.double() - ref[0]).abs() <= ref[2] + 1e-30)[t0:].all())
    out, lse = attend(b)
    assert sk.sk_get_device_status() == 0
    check(b, out, lse, ref)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("qs,cu", [([20, 30, 10], [0, 20, 2 ** 31 - 1, -2 ** 31]), ([20, 30, 10], [0, 20, -2 ** 31, -2 ** 31 + 7]),
                                   ([20, 30, 10], [0, 20, 10, -5]), ([20, 30, 10], [0, 20, 61, 60]),
                                   ([2, 3, 1], [0, 2, 2 ** 31 - 1, -2 ** 31]), ([2, 3, 1], [0, 2, 1, -5]),
                                   ([2, 3, 1], [0, 2, 7, 6]), ([2, 3, 1], [0, 2, 6, 6]), ([20, 30, 10], [0, 20, 60, 60])])
def test_sequences_with_bad_offsets_are_left_out(qs, cu, fp8):
    """Offsets that fall, lie outside or give a sequence more tokens than max_q_len."""
    b = batch([200, 90, 70], qs, 16, 2, fp8, 97, 60, 4)
    w = b["w"]
    ref, ref_lse, tol, _ = reference(b)
    nt = w.num_tokens
    out = torch.full((nt, 16, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((nt, 16), 3.0, device=DEV)
    sk.sk_paged_window_attn(b["q"], b["kv"], b["bt"], b["lens"], torch.tensor(cu, dtype=torch.int32, device=DEV), out, lse,
                            **args_of(b))
    assert sk.sk_get_device_status(clear=True) == sk.SK_DEV_BAD_SEQ
    assert bool(((out.double() - ref).abs() <= tol + 1e-30)[:qs[0]].all())
    assert bool((out[qs[0]:] == 3).all()) and bool((lse[qs[0]:] == 3).all())


def test_offsets_that_give_the_same_tokens_to_many_sequences():
    """Falling offsets whose sequences' costs do not fit 32 bits in all: nothing is done, and the call ends."""
    bs, nt = 32767, 65536
    cu = torch.zeros(bs + 1, dtype=torch.int32, device=DEV)
    cu[1::2] = nt
    q = torch.zeros(nt, 8, 128, dtype=torch.bfloat16, device=DEV)
    kv = torch.zeros(16, 8, 16, 256, dtype=torch.bfloat16, device=DEV)
    bt = torch.zeros(bs, 4096, dtype=torch.int32, device=DEV)
    n = torch.full((bs,), 65536, dtype=torch.int32, device=DEV)
    out = torch.full_like(q, 3.0)
    sk.sk_paged_window_attn(q, kv, bt, n, cu, out, window=30000, max_q_len=nt, sm_scale=0.1)
    assert sk.sk_get_device_status(clear=True) == sk.SK_DEV_BAD_SEQ
    assert bool((out == 3).all())


@pytest.mark.parametrize("name", CALLS)
def test_rows_behind_the_last_sequence_are_left_as_they_were(name):
    b = made(name, False, 19)
    w = b["w"]
    nt, more = w.num_tokens, 37
    q = torch.cat([b["q"], torch.full((more, w.num_q_heads, 128), float("nan"), dtype=torch.bfloat16, device=DEV)])
    out = torch.full((nt + more, w.num_q_heads, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((nt + more, w.num_q_heads), 3.0, device=DEV)
    sk.sk_paged_window_attn(q, b["kv"], b["bt"], b["lens"], b["cu"], out, lse, **args_of(b))
    assert sk.sk_get_device_status(clear=True) == sk.SK_DEV_BAD_SEQ      # cu[bs] is not the number of tokens
    check(b, out[:nt], lse[:nt])
    assert bool((out[nt:] == 3).all()) and bool((lse[nt:] == 3).all())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,qs,hq,hkv", [([30000] * 6, [3] * 6, 16, 2), ([700, 130] * 60, [1, 2] * 60, 8, 2),
                                            ([20000, 9000, 300], [700, 1200, 300], 16, 2)])
def test_expired_waits_are_reported_and_leave_no_trace(lens, qs, hq, hkv, fp8):
    b = batch(lens, qs, hq, hkv, fp8, 71, 5000, 4)
    want = attend(b)
    assert sk.sk_get_device_status() == 0
    limit = sk.sk_set_wait_limit(0)
    try:
        for _ in range(3):                       # the calls return; nothing hangs
            attend(b)
        assert sk.sk_get_device_status(clear=True) & sk.SK_DEV_TIMEOUT
    finally:
        sk.sk_set_wait_limit(-1)
    assert limit > 0
    got = attend(b)
    assert sk.sk_get_device_status() == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bs,hkv,q,window", [(129, 1, 1, 40), (200, 2, 3, 129), (1000, 1, 1, 300), (700, 2, 30, 64)])
def test_many_sequences(bs, hkv, q, window, fp8):
    """More sequences than a warp holds at once, of lengths from nothing on."""
    r = random.Random(bs)
    qs = [r.randint(0, q) for _ in range(bs)]
    lens = [r.choice((0, r.randint(0, 20), r.randint(0, 400))) + n for n in qs]
    b = batch(lens, qs, 4 * hkv, hkv, fp8, 23, window, 5)
    out, lse = run(b)
    assert sk.sk_get_device_status() == 0
    check(b, out, lse)


@pytest.mark.parametrize("hq,hkv", [(3, 1), (5, 1), (12, 1), (24, 2), (48, 1), (64, 1), (65, 1), (96, 1), (160, 1), (256, 1),
                                    (6, 6), (257, 1)])
@pytest.mark.parametrize("qs", [[1, 1, 1], [2, 1, 3], [40, 7, 65]])
def test_groups(hq, hkv, qs):
    """Heads of a group that do and do not divide a tile's rows, on both sides of every bound of the step's rows."""
    b = batch([300, 150, 210], qs, hq, hkv, hq % 2 == 0, 29, 100, 3)
    out, lse = run(b)
    assert sk.sk_get_device_status() == 0
    check(b, out, lse)


@pytest.mark.parametrize("name", CALLS)
def test_outputs_and_queries_aligned_to_16_bytes_only(name):
    b = made(name, False, 37)
    w = b["w"]
    n = w.num_tokens * w.num_q_heads * 128
    q = torch.empty(n + 8, dtype=torch.bfloat16, device=DEV)[8:].view_as(b["q"])
    b["q"] = q.copy_(b["q"])
    flat = torch.full((n + 16,), 3.0, dtype=torch.bfloat16, device=DEV)
    out = flat[8:8 + n].view_as(q)
    assert out.data_ptr() % 32 == 16 and q.data_ptr() % 32 == 16
    sk.sk_paged_window_attn(q, b["kv"], b["bt"], b["lens"], b["cu"], out, **args_of(b))
    assert sk.sk_get_device_status() == 0
    ro, _, to, _ = reference(b)
    assert bool(((out.double() - ro).abs() <= to + 1e-30).all())
    assert bool((flat[:8] == 3).all()) and bool((flat[8 + n:] == 3).all())


@pytest.mark.parametrize("q", [1, 90])
def test_blocks_past_4_gb_and_2_to_the_31_elements(q):
    """The sequence's blocks lie at the far end of a cache of 9.7 GB."""
    b = batch([500, 333], [q, q], 8, 2, False, 41, 200, 4, forget=False)
    near = b["kv"]
    far = torch.empty((590000, *near.shape[1:]), dtype=near.dtype, device=DEV)
    far[-near.shape[0]:].copy_(near)
    shift = far.shape[0] - near.shape[0]
    ref = reference(b)
    b["kv"], b["bt"] = far, torch.where(b["bt"] >= 0, b["bt"] + shift, b["bt"])
    out, lse = run(b)
    assert sk.sk_get_device_status() == 0
    check(b, out, lse, ref)


@pytest.mark.parametrize("name", CALLS)
def test_infinities_and_nan_in_masked_places(name):
    """NaN and infinities in K and V of rows past the end, between sinks and window and in other blocks (as the helper has
    them); what a visible infinity in K does stays in its own head."""
    b = made(name, False, 43)
    kv = b["kv"]
    kv[torch.isnan(kv.float())] = float("inf")
    out, lse = run(b)
    assert sk.sk_get_device_status() == 0
    ref = reference(b)
    check(b, out, lse, ref)
    n = int(b["w"].seq_lens[0]) - 1
    kv[int(b["bt"][0, n // 16]), 1, n % 16, :128] = float("nan")         # a visible one, of head 1
    out, lse = run(b)
    assert sk.sk_get_device_status() == 0
    g, last = b["w"].group, int(b["w"].cu_q[1]) - 1
    assert torch.isnan(out[last, g:].float()).all() and torch.isnan(lse[last, g:]).all()
    ok = torch.ones(out.shape[:2], dtype=torch.bool, device=DEV)
    ok[:last + 1, g:] = False
    assert bool(((out.double() - ref[0]).abs() <= ref[2] + 1e-30)[ok].all())


def drawn(i):
    r = random.Random(1000 + i)
    hq, hkv = r.choice([(8, 1), (16, 2), (32, 2), (32, 8), (16, 16), (12, 4), (5, 1), (40, 8), (9, 3)])
    q = r.choice([1, 1, 2, 3, 4, 7, 20, 150, 600])
    bs = r.randint(1, 40 if q < 8 else 5)
    most = r.choice([20, 300, 3000, 9000 if bs < 9 else 1000])
    qs = [r.choice((q, r.randint(0, q))) for _ in range(bs)]
    lens = [max(0, r.choice((most, r.randint(0, most))) + n - r.choice((0, 0, 0, 1, 5))) for n in qs]
    window = int(2 ** r.uniform(0, 12))
    sinks = r.choice([0, 0, 1, 4, 16, 17, 64, 100, 1000])
    return lens, qs, hq, hkv, r.random() < 0.5, window, sinks


@pytest.mark.parametrize("i", range(80))
def test_drawn_batches(i):
    lens, qs, hq, hkv, fp8, window, sinks = drawn(i)
    if sum(qs) == 0:
        qs[0], lens[0] = 1, lens[0] + 1
    b = batch(lens, qs, hq, hkv, fp8, i, window, sinks)
    out, lse = run(b)
    assert sk.sk_get_device_status() == 0
    check(b, out, lse)


# ------------------------------------------------------------------------- the write and the attention, step after step
def turned(x, pos, freqs, axes, inter):
    """x [tokens, heads, 128] with its first pairs turned, in 64 bits; the bound of a bf16 result's distance."""
    x = x.double()
    n = freqs.numel()
    angle = pos[axes.long()].t().double() * freqs[None]                  # [tokens, pairs]
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if inter else (x[..., :n], x[..., n:2 * n])
    y = x.clone()
    ta, tb = a * c - b * s, b * c + a * s
    if inter:
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = ta, tb
    else:
        y[..., :n], y[..., n:2 * n] = ta, tb
    # half a step of bf16, and the angle's and the products' error in 32 bits (2^-20 of the pair's length)
    return y, 2.0 ** -8 * y.abs() + 2.0 ** -20 * x.abs().amax(-1, keepdim=True) * 2


@pytest.mark.parametrize("inter", [False, True])
def test_prompts_of_text_and_images_then_captured_steps(inter):
    """A server's turn: the prompts' rows turned and written, their attention, then steps whose write and attention are one
    captured graph; each result against the formulas, on the rows that the pages then hold."""
    hq, hkv, window, sinks, prompts, steps = 16, 2, 100, 4, [260, 33, 120], 5
    bs, g = len(prompts), torch.Generator(device=DEV).manual_seed(61)
    rows = [(n + steps + 15) // 16 for n in prompts]
    table = torch.full((bs, max(rows)), -1, dtype=torch.int32, device=DEV)
    perm = torch.randperm(sum(rows) + 3, generator=g, device=DEV).int()
    at = 0
    for s, n in enumerate(rows):
        table[s, :n], at = perm[at:at + n], at + n
    pages = torch.full((sum(rows) + 3, hkv, 16, 256), float("nan"), dtype=torch.bfloat16, device=DEV)
    axes = sk.sk_rope_axes(128, [16, 24, 24], cycled=False, device=DEV)
    freqs, _ = sk.sk_rope_frequencies(128, device=DEV)
    ws = {}

    def slots(s, first, n):
        r = torch.arange(first, first + n, device=DEV)
        return table[s].long()[r // 16] * 16 + r % 16

    def randn(n, h):
        return torch.randn(n, h, 128, generator=g, device=DEV).bfloat16()

    def write(q, k, v, pos, sl, q_out):
        sk.sk_rope_axes_and_cache(q, k, v, pos, freqs, axes, sl, pages, q_out, interleaved=inter)

    def written(q, k, v, pos, sl, q_out):
        y, tol = turned(q, pos, freqs, axes, inter)
        assert bool(((q_out.double() - y).abs() <= tol).all())
        y, tol = turned(k, pos, freqs, axes, inter)
        got = pages[sl // 16, :, sl % 16]
        assert bool(((got[..., :128].double() - y).abs() <= tol).all()) and torch.equal(got[..., 128:], v)

    def seen(lens, qs, q, out, lse):
        class W:
            num_tokens, num_q_heads, num_kv_heads, group, kv_dtype = sum(qs), hq, hkv, hq // hkv, si.KV_BF16
            seq_lens, q_lens, cu_q, sm_scale = lens, qs, [sum(qs[:i]) for i in range(bs + 1)], 0.088
        W.bs = bs
        check(dict(w=W, q=q, kv=pages, table=table, window=window, sinks=sinks), out, lse)

    # the prompts: text, then an image of 8 columns with a height and a width of its own
    pos = torch.cat([torch.stack([torch.arange(n), torch.where(torch.arange(n) < 20, torch.arange(n), 20 + (torch.arange(n) - 20) // 8),
                                  torch.where(torch.arange(n) < 20, torch.arange(n), 20 + (torch.arange(n) - 20) % 8)])
                     for n in prompts], 1).to(DEV)
    nt = sum(prompts)
    q, k, v, q_out = randn(nt, hq), randn(nt, hkv), randn(nt, hkv), torch.empty(nt, hq, 128, dtype=torch.bfloat16, device=DEV)
    sl = torch.cat([slots(s, 0, n) for s, n in enumerate(prompts)])
    write(q, k, v, pos, sl, q_out)
    lens = torch.tensor(prompts, dtype=torch.int32, device=DEV)
    cu = torch.tensor([sum(prompts[:i]) for i in range(bs + 1)], dtype=torch.int32, device=DEV)
    out, lse = sk.paged_window_attention(q_out, pages, table, lens, cu, window=window, sinks=sinks, max_q_len=max(prompts),
                                         sm_scale=0.088, workspace=ws)
    written(q, k, v, pos, sl, q_out)
    seen(prompts, prompts, q_out, out, lse)

    # the steps
    q, k, v, q_out = randn(bs, hq), randn(bs, hkv), randn(bs, hkv), torch.empty(bs, hq, 128, dtype=torch.bfloat16, device=DEV)
    pos, sl = torch.zeros(3, bs, dtype=torch.int64, device=DEV), torch.full((bs,), -1, dtype=torch.int64, device=DEV)
    cu = torch.arange(bs + 1, dtype=torch.int32, device=DEV)
    out, lse = torch.empty_like(q_out), torch.empty(bs, hq, device=DEV)

    def step():
        write(q, k, v, pos, sl, q_out)
        sk.sk_paged_window_attn(q_out, pages, table, lens, cu, out, lse, window=window, sinks=sinks, max_q_len=1,
                                sm_scale=0.088, workspace=ws)

    step()                                       # (slots of -1: nothing is written)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(steps):
        q.copy_(randn(bs, hq)), k.copy_(randn(bs, hkv)), v.copy_(randn(bs, hkv))
        pos.copy_((lens - 7).long().expand(3, bs))
        sl.copy_(torch.cat([slots(s, n + i, 1) for s, n in enumerate(prompts)]))
        lens += 1
        graph.replay()
        torch.cuda.synchronize()
        written(q, k, v, pos, sl, q_out)
        seen([n + i + 1 for n in prompts], [1] * bs, q_out, out, lse)
    assert sk.sk_get_device_status() == 0
