"""A cache bounded by eviction, step by step as a server runs it: rotate and write the new tokens, attend, gather the
weights, evict.  The calls of a step follow each other on the stream without a wait; each one's result is then compared
with the definition in 64 bits on what it read, with the tolerances of its own tests."""
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import paged_split_kv_gb300 as sk
import sk_inputs as si
from test_accum_gpu import check as check_weights
from test_evict_gpu import reference as evicted
from test_prefill_gpu import check as check_attention
from test_rope_gpu import bf16_bound, rotated

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
D, PAGE = 128, 16


class Server:
    """bs sequences over one pool of pages, `budget` rows each at the most between steps."""

    def __init__(self, bs, hq, hkv, budget, recent, fp8, rot, seed, room):
        self.g = torch.Generator(device=DEV).manual_seed(seed)
        self.bs, self.hq, self.hkv, self.budget, self.recent, self.fp8 = bs, hq, hkv, budget, recent, fp8
        npg = (budget + room + PAGE - 1) // PAGE
        perm = np.random.default_rng(seed).permutation(bs * npg + 3).astype(np.int32)
        self.bt_host = perm[:bs * npg].reshape(bs, npg)
        self.bt = torch.as_tensor(self.bt_host, device=DEV)
        nb = bs * npg + 3
        self.pages = torch.randn(nb, hkv, PAGE, 2 * D, generator=self.g, device=DEV).to(
            torch.float8_e4m3fn if fp8 else torch.bfloat16)
        self.acc = torch.full((nb, hkv, PAGE), 9.0, device=DEV)
        self.pos = torch.full((nb, hkv, PAGE), -9, dtype=torch.int32, device=DEV)
        self.freqs, self.factor = sk.sk_rope_frequencies(rot, 10000.0, device=DEV)
        self.lens = np.zeros(bs, np.int64)           # rows in the cache
        self.seen = np.zeros(bs, np.int64)           # tokens so far
        self.ks, self.vs = (0.5, 0.25) if fp8 else (1.0, 1.0)
        self.ws = {}
        self.sms = torch.cuda.get_device_properties(DEV).multi_processor_count

    def inputs(self, qs):
        """A step's tokens, with their positions and cache slots."""
        qs = np.asarray(qs)
        nt = int(qs.sum())
        qkv = torch.randn(nt, self.hq + 2 * self.hkv, D, generator=self.g, device=DEV).to(torch.bfloat16)
        pos, slots = [], []
        for s, q in enumerate(qs):
            r = self.lens[s] + np.arange(q)
            slots.append(self.bt_host[s, r // PAGE].astype(np.int64) * PAGE + r % PAGE)
            pos.append(self.seen[s] + np.arange(q))
        t = lambda x, dt: torch.as_tensor(np.asarray(x), device=DEV).to(dt)
        return SimpleNamespace(
            qs=qs, nt=nt, q=qkv[:, :self.hq], k=qkv[:, self.hq:self.hq + self.hkv], v=qkv[:, self.hq + self.hkv:],
            pos=t(np.concatenate(pos), torch.int64), slots=t(np.concatenate(slots), torch.int64),
            cu=t(np.concatenate([[0], np.cumsum(qs)]), torch.int32), lens=t(self.lens + qs, torch.int32),
            next_pos=t(self.seen + qs, torch.int32))

    def calls(self, x, keep=lambda name: None):
        """The five calls of a step; `keep(name)` after each."""
        qr = torch.empty(x.nt, self.hq, D, dtype=torch.bfloat16, device=DEV)
        sk.sk_rope_and_cache(x.q, x.k, x.v, x.pos, self.freqs, x.slots, self.pages, qr, attn_factor=self.factor,
                             k_scale=self.ks, v_scale=self.vs, acc_pages=self.acc, pos_pages=self.pos)
        keep("written")
        args = dict(max_q_len=int(x.qs.max()), sm_scale=D ** -0.5, k_scale=self.ks, v_scale=self.vs)
        if x.qs.max() == 1 and not self.fp8:
            out = torch.empty_like(qr)
            lse = torch.empty(x.nt, self.hq, device=DEV)
            sk.sk_paged_decode_attention_static(qr, self.pages, self.bt, x.lens, x.cu, out, lse,
                                                num_sms=self.sms, **args)
        else:
            out, lse = sk.paged_prefill_attention(qr, self.pages, self.bt, x.lens, x.cu, workspace=self.ws, **args)
        args.pop("v_scale")
        sk.sk_accum_attn_weights(qr, self.pages, self.bt, x.lens, x.cu, lse, self.acc, workspace=self.ws, **args)
        keep("gathered")
        new = sk.evict_rows(self.pages, self.acc, self.pos, self.bt, x.lens, x.next_pos, budget=self.budget,
                            recent=self.recent, workspace=self.ws)
        return qr, out, lse, new

    def step(self, qs):
        x = self.inputs(qs)
        was = {"before": (self.pages.clone(), self.acc.clone(), self.pos.clone())}
        qr, out, lse, new = self.calls(x, lambda name: was.__setitem__(
            name, (self.pages.clone(), self.acc.clone(), self.pos.clone())))
        assert sk.sk_get_device_status() == 0
        self.check_write(x, qr, was["before"], was["written"])
        w = SimpleNamespace(bs=self.bs, seq_lens=self.lens + x.qs, q_lens=x.qs, cu_q=x.cu.cpu().numpy(),
                            num_tokens=x.nt, num_q_heads=self.hq, num_kv_heads=self.hkv, group=self.hq // self.hkv,
                            kv_dtype=si.KV_FP8 if self.fp8 else si.KV_BF16, k_scale=self.ks, v_scale=self.vs,
                            sm_scale=D ** -0.5, causal=1)
        pages, acc, pos = was["gathered"]
        assert torch.equal(pages.view(torch.uint8), was["written"][0].view(torch.uint8))
        b = dict(w=w, q=qr, kv=pages.view(torch.uint8) if self.fp8 else pages, bt=self.bt, lens=x.lens, cu=x.cu)
        check_attention(b, out, lse)
        check_weights(b, lse, was["written"][1], acc)
        self.check_eviction(x, pages, acc, pos, new)
        self.lens = np.minimum(self.lens + x.qs, self.budget)
        self.seen = self.seen + x.qs

    def check_write(self, x, qr, before, after):
        kr, size = rotated(x.k, x.pos, self.freqs, False, self.factor)
        y, ysize = rotated(x.q, x.pos, self.freqs, False, self.factor)
        assert ((qr.double().cpu() - y).abs() <= bf16_bound(y, ysize)).all()
        blk, row = x.slots // PAGE, x.slots % PAGE
        got = after[0][blk, :, row].double().cpu()
        if self.fp8:
            kr, size = kr / self.ks, size / self.ks
            tol = torch.clamp(kr.abs() * 2.0 ** -4, min=2.0 ** -10) + size * 2.0 ** -21
        else:
            tol = bf16_bound(kr, size)
        assert ((got[..., :D] - kr).abs() <= tol).all()
        v = (x.v.float() / self.vs).to(self.pages.dtype)
        assert torch.equal(after[0][blk, :, row][..., D:].contiguous().view(torch.uint8), v.contiguous().view(torch.uint8))
        want_acc, want_pos = before[1].clone(), before[2].clone()
        want_acc[blk, :, row] = 0
        want_pos[blk, :, row] = x.pos.to(torch.int32)[:, None]
        assert torch.equal(after[1], want_acc) and torch.equal(after[2], want_pos)

    def check_eviction(self, x, pages, acc, pos, new):
        pages, acc, pos = (t.cpu() for t in (pages.view(torch.uint8), acc, pos))
        lens = [int(n) for n in self.lens + x.qs]
        for (s, h), (src, dst) in evicted(self.bt_host, acc.numpy(), pos.numpy(), lens, self.seen + x.qs, self.hkv,
                                          self.budget, self.recent).items():
            a, b = self.bt_host[s, src // PAGE], self.bt_host[s, dst // PAGE]
            for t in (pages, acc, pos):
                t[b, h, dst % PAGE] = t[a, h, src % PAGE]
        assert new.tolist() == [min(n, self.budget) for n in lens]
        assert torch.equal(pages, self.pages.view(torch.uint8).cpu())
        assert torch.equal(acc, self.acc.cpu()) and torch.equal(pos, self.pos.cpu())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv,budget,recent,rot,steps", [
    (8, 2, 48, 10, 128, [[37, 1, 60], [5, 20, 1], [1, 1, 1], [1, 1, 1], [0, 2, 90], [1, 1, 1]]),
    (16, 1, 300, 64, 64, [[290, 700, 33], [3, 3, 3], [1, 1, 1], [200, 1, 400], [1, 1, 1]]),
    (4, 4, 17, 0, 32, [[1, 1, 1]] * 4 + [[16, 15, 14], [1, 1, 1], [4, 4, 4]])])
def test_steps_of_a_bounded_cache(hq, hkv, budget, recent, rot, steps, fp8):
    room = max(max(s) for s in steps)
    server = Server(3, hq, hkv, budget, recent, fp8, rot, 7 + budget, room)
    for qs in steps:
        server.step(qs)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_captured_step_replayed_goes_on_as_the_calls_do(fp8):
    """A full cache takes one token a step with the same lengths every time: one graph, its inputs copied in."""
    servers = [Server(4, 8, 2, 64, 8, fp8, 128, 5, 100) for _ in range(2)]
    for server in servers:
        server.step([64, 64, 100, 70])
    eager, replayed = servers
    x = replayed.inputs([1, 1, 1, 1])
    held = SimpleNamespace(**{k: v.clone() if torch.is_tensor(v) else v for k, v in vars(x).items()})
    replayed.g.manual_seed(1)
    eager.g.manual_seed(1)
    saved = [t.clone() for t in (replayed.pages, replayed.acc, replayed.pos)]
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        qr, out, lse, new = replayed.calls(held)
    for t, s in zip((replayed.pages, replayed.acc, replayed.pos), saved):
        t.copy_(s)
    for _ in range(6):
        a, b = eager.inputs([1] * 4), replayed.inputs([1] * 4)
        for name, t in vars(b).items():
            if torch.is_tensor(t):
                getattr(held, name).copy_(t)
        graph.replay()
        want = eager.calls(a)
        for got, right in zip((qr, out, lse, new), want):
            assert torch.equal(got, right)
        for server in servers:
            server.seen += 1
    assert sk.sk_get_device_status() == 0
    assert torch.equal(eager.pages.view(torch.uint8), replayed.pages.view(torch.uint8))
    assert torch.equal(eager.acc, replayed.acc) and torch.equal(eager.pos, replayed.pos)


@pytest.mark.parametrize("fp8", [False, True])
def test_memory_of_calls_on_another_stream(fp8):
    """Calls on a stream of their own, without workspaces: what the caller's stream allocates next must not be memory that
    those calls, still waiting on their stream, will use."""
    qs = [64, 64, 100, 70]
    servers = [Server(4, 8, 2, 64, 8, fp8, 128, 6, 100) for _ in range(2)]
    want = servers[0].calls(servers[0].inputs(qs))
    server, x = servers[1], servers[1].inputs(qs)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    args = dict(max_q_len=100, sm_scale=D ** -0.5, k_scale=server.ks)
    qr = torch.empty(x.nt, 8, D, dtype=torch.bfloat16, device=DEV)
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    sk.sk_rope_and_cache(x.q, x.k, x.v, x.pos, server.freqs, x.slots, server.pages, qr, attn_factor=server.factor,
                         k_scale=server.ks, v_scale=server.vs, acc_pages=server.acc, pos_pages=server.pos, stream=side)
    out, lse = sk.paged_prefill_attention(qr, server.pages, server.bt, x.lens, x.cu, v_scale=server.vs, stream=side, **args)
    sk.sk_accum_attn_weights(qr, server.pages, server.bt, x.lens, x.cu, lse, server.acc, stream=side.cuda_stream, **args)
    new = sk.evict_rows(server.pages, server.acc, server.pos, server.bt, x.lens, x.next_pos, budget=64, recent=8,
                        stream=side)
    held = []
    for need in (sk.sk_prefill_workspace_bytes(x.nt, 8, int(fp8)), sk.sk_accum_workspace_bytes(x.nt, 8, 2, 100, int(fp8)),
                 4 * 2 * sk.sk_evict_capacity(64, server.bt.shape[1] * PAGE) * 4, 4 * 2 * 4):
        held += [torch.full((need,), 0xA5, dtype=torch.uint8, device=DEV) for _ in range(3)]
    torch.cuda.synchronize()
    assert sk.sk_get_device_status() == 0
    for got, right in zip((qr, out, lse, new), want):
        assert torch.equal(got, right)
    assert all(bool((t == 0xA5).all()) for t in held)
    assert torch.equal(server.pages.view(torch.uint8), servers[0].pages.view(torch.uint8))
    assert torch.equal(server.acc, servers[0].acc) and torch.equal(server.pos, servers[0].pos)
