"""Host-side checks of the rotary KV write and the eviction calls: refusals before anything touches CUDA, the
rotary frequencies against their formulas, and the binding's shape checks (CPU tensors: they come before the
device check)."""
import ctypes
import math

import numpy as np
import pytest
import torch

FAKE = ctypes.c_void_p(256)   # never dereferenced: validation runs first
ODD = ctypes.c_void_p(264)


@pytest.fixture(scope="module")
def sk():
    from paged_split_kv_gb300 import build as b
    b.build()
    import paged_split_kv_gb300 as sk
    sk.lib()
    return sk


def caller(f, base):
    return lambda **kw: f(*dict(base, **kw).values())


def test_rope_refusals(sk):
    call = caller(sk.lib().sk_rope_and_cache, dict(
        q=FAKE, k=FAKE, v=FAKE, qs=1024, ks=256, vs=256, pos=FAKE, fr=FAKE, rot=64, inter=0, f=1.0, sl=FAKE, nt=4,
        hq=8, hkv=2, d=128, qo=FAKE, pg=FAKE, dt=0, ksc=1.0, vsc=1.0, nb=8, page=16, acc=None, pp=None, st=None))
    assert call(d=64) == -3 and call(page=32) == -3
    for rot in (0, 8, 24, 144, -16):
        assert call(rot=rot) == -3, rot
    for kw in (dict(nt=-1), dict(hq=0), dict(hkv=0), dict(nb=0), dict(dt=2), dict(f=0.0), dict(f=float("nan")),
               dict(dt=1, ksc=0.0), dict(dt=1, vsc=float("inf")), dict(q=None), dict(sl=None), dict(fr=None),
               dict(qs=1023), dict(qs=1028), dict(ks=248), dict(vs=0), dict(q=ODD), dict(pg=ODD), dict(qo=ODD)):
        assert call(**kw) == -1, kw
    assert call(nt=0, q=None, k=None, v=None, pos=None, sl=None, qo=None, pg=None) == 0


def test_evict_refusals(sk):
    call = caller(sk.lib().sk_evict_select, dict(
        acc=FAKE, pos=FAKE, bt=FAKE, stride=10, nb=8, page=16, lens=FAKE, nxt=FAKE, bs=2, hkv=2, budget=32, recent=4,
        mx=160, cap=32, src=FAKE, dst=FAKE, cnt=FAKE, new=FAKE, st=None))
    for kw in (dict(bs=0), dict(bs=32768), dict(hkv=0), dict(nb=0), dict(stride=0), dict(budget=0), dict(recent=-1), dict(acc=ODD),
               dict(recent=33), dict(mx=-1), dict(acc=None), dict(nxt=None), dict(new=None)):
        assert call(**kw) == -1, kw
    assert call(page=8) == -3 and call(bs=32767, hkv=1 << 20) == -3
    assert call(cap=31) == -2 and call(mx=60, cap=27) == -2
    call = caller(sk.lib().sk_evict_move, dict(src=FAKE, dst=FAKE, cnt=FAKE, cap=4, bs=2, hkv=2, d=128, bt=FAKE,
                                               stride=10, nb=8, page=16, pg=FAKE, dt=0, acc=FAKE, pos=FAKE, st=None))
    for kw in (dict(bs=0), dict(cap=0), dict(dt=5), dict(src=None), dict(acc=None), dict(pos=None), dict(pg=ODD)):
        assert call(**kw) == -1, kw
    assert call(d=64) == -3 and call(page=32) == -3


def test_evict_capacity(sk):
    for budget in (1, 5, 100):
        for n in (0, 1, 5, 6, 99, 101, 150, 200, 201, 1000):
            assert sk.sk_evict_capacity(budget, n) == max(1, min(budget, n - budget))
    with pytest.raises(sk.SkError):
        sk.sk_evict_capacity(0, 5)


def test_rope_frequencies(sk):
    i = np.arange(32)
    w = 10000.0 ** (-2 * i / 64)
    f, a = sk.sk_rope_frequencies(64)
    np.testing.assert_allclose(f.numpy(), w, rtol=1e-14)
    assert a == 1.0 and f.dtype == torch.float64
    f, a = sk.sk_rope_frequencies(64, scaling="linear", factor=4.0)
    np.testing.assert_allclose(f.numpy(), w / 4, rtol=1e-14)
    f, a = sk.sk_rope_frequencies(64, scaling="base", factor=4.0)
    np.testing.assert_allclose(f.numpy(), (10000.0 * 4 ** (64 / 62)) ** (-2 * i / 64), rtol=1e-13)
    # the slowest frequency of a rescaled base turns `factor` times slower: positions reach that much further
    assert math.isclose(f[-1].item() * 4, w[-1], rel_tol=1e-12)
    f, a = sk.sk_rope_frequencies(64, scaling="bands", factor=8.0, original_len=4096, low=1, high=32)
    turns = 4096 * w / (2 * np.pi)
    keep = np.clip((turns - 1) / 31, 0, 1)
    np.testing.assert_allclose(f.numpy(), (1 - keep) * w / 8 + keep * w, rtol=1e-13)
    assert math.isclose(a, 0.1 * math.log(8) + 1)
    assert (f.numpy()[turns >= 32] == w[turns >= 32]).all() or np.allclose(f.numpy()[turns >= 32], w[turns >= 32], rtol=1e-14)
    for bad in (dict(rot_dim=63), dict(rot_dim=0), dict(rot_dim=64, base=1.0), dict(rot_dim=64, factor=0.5),
                dict(rot_dim=2, scaling="base"), dict(rot_dim=64, scaling="bands", original_len=0),
                dict(rot_dim=64, scaling="bands", original_len=10, low=4, high=4)):
        with pytest.raises(sk.SkError):
            sk.sk_rope_frequencies(**bad)
    with pytest.raises(ValueError):
        sk.sk_rope_frequencies(64, scaling="other")


def test_binding_checks_shapes_before_raw_pointers(sk):
    bf, i32, i64 = torch.bfloat16, torch.int32, torch.int64

    def rope(**kw):
        a = dict(q=torch.zeros(4, 8, 128, dtype=bf), k=torch.zeros(4, 2, 128, dtype=bf),
                 v=torch.zeros(4, 2, 128, dtype=bf), pos=torch.zeros(4, dtype=i64),
                 fr=torch.zeros(32, dtype=torch.float64), sl=torch.zeros(4, dtype=i64),
                 pg=torch.zeros(3, 2, 16, 256, dtype=bf), qo=torch.zeros(4, 8, 128, dtype=bf), acc=None, pp=None)
        a.update(kw)
        return sk.sk_rope_and_cache(a["q"], a["k"], a["v"], a["pos"], a["fr"], a["sl"], a["pg"], a["qo"],
                                    acc_pages=a["acc"], pos_pages=a["pp"])

    wide = torch.zeros(4, 8, 256, dtype=bf)
    for kw in (dict(q=torch.zeros(4, 8, 128)), dict(q=wide[..., ::2]), dict(q=wide[..., :128]),
               dict(k=torch.zeros(5, 2, 128, dtype=bf)), dict(v=torch.zeros(4, 3, 128, dtype=bf)),
               dict(pos=torch.zeros(4, dtype=i32)), dict(pos=torch.zeros(5, dtype=i64)),
               dict(sl=torch.zeros(3, dtype=i64)), dict(fr=torch.zeros(32)), dict(qo=torch.zeros(4, 8, 64, dtype=bf)),
               dict(pg=torch.zeros(3, 2, 16, 128, dtype=bf)), dict(pg=torch.zeros(3, 1, 16, 256, dtype=bf)),
               dict(acc=torch.zeros(3, 2, 8)), dict(acc=torch.zeros(3, 2, 16, dtype=i32)),
               dict(pp=torch.zeros(2, 2, 16, dtype=i32))):
        with pytest.raises(ValueError):
            rope(**kw)
    with pytest.raises(ValueError, match="CUDA"):
        rope()

    def select(**kw):
        a = dict(acc=torch.zeros(5, 2, 16), pos=torch.zeros(5, 2, 16, dtype=i32), bt=torch.zeros(3, 4, dtype=i32),
                 lens=torch.zeros(3, dtype=i32), nxt=torch.zeros(3, dtype=i32), src=torch.zeros(3, 2, 8, dtype=i32),
                 dst=torch.zeros(3, 2, 8, dtype=i32), cnt=torch.zeros(3, 2, dtype=i32), new=torch.zeros(3, dtype=i32))
        a.update(kw)
        return sk.sk_evict_select(*a.values(), budget=8)

    lens = torch.zeros(3, dtype=i32)
    for kw in (dict(pos=torch.zeros(5, 2, 8, dtype=i32)), dict(acc=torch.zeros(5, 2, 16, dtype=i32)),
               dict(bt=torch.zeros(2, 4, dtype=i32)), dict(nxt=torch.zeros(2, dtype=i32)),
               dict(src=torch.zeros(3, 1, 8, dtype=i32)), dict(dst=torch.zeros(3, 2, 7, dtype=i32)),
               dict(cnt=torch.zeros(3, 3, dtype=i32)), dict(new=torch.zeros(4, dtype=i32)), dict(lens=lens, new=lens)):
        with pytest.raises(ValueError):
            select(**kw)
    with pytest.raises(ValueError, match="CUDA"):
        select()

    def move(**kw):
        a = dict(src=torch.zeros(3, 2, 8, dtype=i32), dst=torch.zeros(3, 2, 8, dtype=i32),
                 cnt=torch.zeros(3, 2, dtype=i32), bt=torch.zeros(3, 4, dtype=i32),
                 pg=torch.zeros(5, 2, 16, 256, dtype=bf), acc=torch.zeros(5, 2, 16),
                 pos=torch.zeros(5, 2, 16, dtype=i32))
        a.update(kw)
        return sk.sk_evict_move(*a.values())

    for kw in (dict(dst=torch.zeros(3, 2, 9, dtype=i32)), dict(cnt=torch.zeros(2, 2, dtype=i32)),
               dict(bt=torch.zeros(2, 4, dtype=i32)), dict(pg=torch.zeros(5, 3, 16, 256, dtype=bf)),
               dict(acc=torch.zeros(4, 2, 16)), dict(acc=None), dict(pos=torch.zeros(5, 2, 16))):
        with pytest.raises(ValueError):
            move(**kw)
    with pytest.raises(ValueError, match="CUDA"):
        move()


def test_prefill_refusals(sk):
    call = caller(sk.lib().sk_paged_prefill_attn, dict(
        q=FAKE, kv=FAKE, dt=0, ks=1.0, vs=1.0, bt=FAKE, stride=10, nb=100, page=16, lens=FAKE, cu=FAKE, bs=4, nt=16,
        mq=4, hq=32, hkv=2, d=128, scale=0.088, causal=1, mx=160, ws=FAKE, wb=1 << 30, out=FAKE, lse=None, st=None))
    for kw in (dict(q=None), dict(out=None), dict(cu=None), dict(dt=3), dict(bs=0), dict(bs=32768), dict(nt=-1),
               dict(mq=0), dict(stride=0), dict(nb=0), dict(hq=31), dict(hkv=0), dict(mx=-1), dict(ws=ODD),
               dict(scale=0.0), dict(scale=float("inf")), dict(dt=1, ks=0.0), dict(dt=1, vs=float("nan")), dict(q=ODD),
               dict(kv=ODD), dict(out=ODD)):
        assert call(**kw) == -1, kw
    assert call(d=64) == -3 and call(page=32) == -3
    assert call(nb=1 << 30) == -3 and call(mq=1 << 30) == -3
    assert call(nt=0, mq=0) == 0


def test_accum_refusals(sk):
    call = caller(sk.lib().sk_accum_attn_weights, dict(
        q=FAKE, kv=FAKE, dt=0, ks=1.0, bt=FAKE, stride=10, nb=100, page=16, lens=FAKE, cu=FAKE, bs=4, nt=16, mq=4,
        hq=32, hkv=2, d=128, scale=0.088, causal=1, lse=FAKE, acc=FAKE, ws=None, wb=0, st=None))
    for kw in (dict(q=None), dict(lse=None), dict(acc=None), dict(dt=3), dict(bs=0), dict(mq=0), dict(hq=31),
               dict(scale=-1.0), dict(dt=1, ks=0.0), dict(kv=ODD), dict(ws=ODD)):
        assert call(**kw) == -1, kw
    assert call(d=64) == -3 and call(page=32) == -3 and call(nb=1 << 30) == -3
    need = sk.sk_accum_workspace_bytes(16, 32, 2, 4, 1)
    assert need == 16 * 32 * 260 and sk.sk_accum_workspace_bytes(16, 32, 2, 4, 0) == 0
    parts = sk.sk_accum_workspace_bytes(16, 32, 2, 5, 0)
    assert parts > 0 and sk.sk_accum_workspace_bytes(16, 32, 2, 5, 1) == need + parts
    assert call(mq=5, ws=FAKE, wb=parts - 1) == -2 and call(mq=5) == -2
    assert call(dt=1, ws=FAKE, wb=need - 1) == -2 and call(dt=1, ws=None, wb=need) == -2
    assert call(nt=0, mq=0) == 0
    with pytest.raises(sk.SkError):
        sk.sk_accum_workspace_bytes(16, 0, 2, 4, 1)


def test_binding_checks_attention_shapes(sk):
    bf, i32 = torch.bfloat16, torch.int32

    def base(**kw):
        a = dict(q=torch.zeros(8, 8, 128, dtype=bf), kv=torch.zeros(4, 2, 16, 256, dtype=bf),
                 bt=torch.zeros(2, 3, dtype=i32), lens=torch.zeros(2, dtype=i32), cu=torch.zeros(3, dtype=i32),
                 out=torch.zeros(8, 8, 128, dtype=bf), lse=torch.zeros(8, 8),
                 acc=torch.zeros(4, 2, 16))
        a.update(kw)
        return a

    def prefill(**kw):
        a = base(**kw)
        return sk.sk_paged_prefill_attn(a["q"], a["kv"], a["bt"], a["lens"], a["cu"], a["out"], a["lse"], max_q_len=4,
                                        sm_scale=0.1)

    def accum(**kw):
        a = base(**kw)
        return sk.sk_accum_attn_weights(a["q"], a["kv"], a["bt"], a["lens"], a["cu"], a["lse"], a["acc"], max_q_len=4,
                                        sm_scale=0.1)

    common = [dict(q=torch.zeros(8, 8, 128)), dict(q=torch.zeros(8, 8, 256, dtype=bf)[..., ::2]),
              dict(kv=torch.zeros(4, 3, 16, 256, dtype=bf)), dict(kv=torch.zeros(4, 2, 16, 128, dtype=bf)),
              dict(bt=torch.zeros(1, 3, dtype=i32)), dict(cu=torch.zeros(4, dtype=i32)), dict(lse=torch.zeros(7, 8))]
    for kw in common:
        for f in (prefill, accum):
            with pytest.raises(ValueError):
                f(**kw)
    for kw in (dict(out=torch.zeros(7, 8, 128, dtype=bf)), dict(out=torch.zeros(8, 8, 128)), dict(out=None)):
        with pytest.raises(ValueError):
            prefill(**kw)
    for kw in (dict(acc=torch.zeros(4, 2, 8)), dict(acc=None), dict(lse=None)):
        with pytest.raises(ValueError):
            accum(**kw)
    for f in (prefill, accum):
        with pytest.raises(ValueError, match="CUDA"):
            f()


def test_limits_of_row_numbers_and_pairs(sk):
    """Row numbers stay below 2^30 and (sequence, head) pairs at 2^24 or below, whatever the arrays hold."""
    lib = sk.lib()
    attn = dict(q=FAKE, kv=FAKE, dt=0, ks=1.0, vs=1.0, bt=FAKE, stride=10, nb=100, page=16, lens=FAKE, cu=FAKE, bs=4,
                nt=0, mq=0, hq=1024, hkv=1024, d=128, scale=0.088, causal=1, mx=160, ws=FAKE, wb=1 << 30, out=FAKE,
                lse=None, st=None)
    prefill = caller(lib.sk_paged_prefill_attn, attn)
    weights = {k: attn[k] for k in attn if k not in ("vs", "mx", "ws", "wb", "out", "lse", "st")}
    accum = caller(lib.sk_accum_attn_weights, dict(weights, lse=FAKE, acc=FAKE, ws=FAKE, wb=1 << 30, st=None))
    for call in (prefill, accum):
        assert call() == 0 and call(stride=1 << 26) == 0
        assert call(stride=(1 << 26) + 1) == -3 and call(bs=20000) == -3
    select = caller(lib.sk_evict_select, dict(
        acc=FAKE, pos=FAKE, bt=FAKE, stride=10, nb=100, page=16, lens=FAKE, nxt=FAKE, bs=4, hkv=2, budget=8, recent=0,
        mx=160, cap=8, src=FAKE, dst=FAKE, cnt=FAKE, new=FAKE, st=None))
    move = caller(lib.sk_evict_move, dict(
        src=FAKE, dst=FAKE, cnt=FAKE, cap=8, bs=4, hkv=2, d=128, bt=FAKE, stride=10, nb=100, page=16, kv=FAKE, dt=0,
        acc=FAKE, pos=FAKE, st=None))
    for call in (select, move):
        assert call(stride=(1 << 26) + 1) == -3 and call(bs=20000, hkv=1024) == -3
    assert select(mx=(1 << 30) + 1) == -3
