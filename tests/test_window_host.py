"""Host-side checks of windowed attention and of the rotary write with several axes: refusals before anything touches
CUDA, and the axes against their definition (CPU tensors: the shape checks come before the device check)."""
import ctypes

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


def test_window_refusals(sk):
    call = caller(sk.lib().sk_paged_window_attn, dict(
        q=FAKE, kv=FAKE, dt=0, ks=1.0, vs=1.0, bt=FAKE, stride=10, nb=8, page=16, lens=FAKE, cu=FAKE, bs=2, nt=4, mq=2,
        hq=8, hkv=2, d=128, scale=0.1, window=64, sinks=4, mx=160, ws=FAKE, wsb=1 << 40, out=FAKE, lse=None, st=None))
    for kw in (dict(window=0), dict(window=-1), dict(sinks=-1), dict(q=None), dict(kv=None), dict(bt=None),
               dict(lens=None), dict(cu=None), dict(out=None), dict(dt=2), dict(bs=0), dict(bs=32768), dict(nt=-1),
               dict(mq=0), dict(mq=-1), dict(stride=0), dict(nb=0), dict(hq=0), dict(hkv=0), dict(hq=7), dict(mx=-1),
               dict(scale=0.0), dict(scale=float("nan")), dict(dt=1, ks=0.0), dict(dt=1, vs=float("inf")),
               dict(q=ODD), dict(kv=ODD), dict(out=ODD), dict(ws=ODD)):
        assert call(**kw) == -1, kw
    assert call(d=64) == -3 and call(page=32) == -3
    assert call(nb=1 << 30) == -3 and call(stride=(1 << 26) + 1) == -3 and call(bs=32767, hq=1 << 20, hkv=1 << 20) == -3
    assert call(nt=0, mq=0, q=None, out=None) == 0


def test_window_workspace_refusals(sk):
    for bad in ((-1, 8, 2, 1, 0), (4, 0, 2, 1, 0), (4, 8, 0, 1, 0), (4, 7, 2, 1, 0), (4, 8, 2, -1, 0), (4, 8, 2, 1, 2)):
        with pytest.raises(sk.SkError):
            sk.sk_window_workspace_bytes(*bad)


def test_axes(sk):
    a = sk.sk_rope_axes(128, [16, 24, 24])
    assert a.dtype is torch.uint8 and a.tolist() == [0] * 16 + [1] * 24 + [2] * 24
    c = sk.sk_rope_axes(128, [24, 20, 20], cycled=True).tolist()
    assert c == [0, 1, 2] * 20 + [0] * 4 and [c.count(i) for i in range(3)] == [24, 20, 20]
    assert sk.sk_rope_axes(16, [8]).tolist() == [0] * 8 == sk.sk_rope_axes(16, [8], cycled=True).tolist()
    assert sk.sk_rope_axes(16, [0, 8, 0]).tolist() == [1] * 8
    # sections of different sizes: the axis that has run out leaves its turns to the first
    assert sk.sk_rope_axes(24, [6, 4, 2], cycled=True).tolist() == [0, 1, 2, 0, 1, 2, 0, 1, 0, 0, 1, 0]
    for rot, sec, cyc in ((15, [7], False), (0, [0], False), (16, [4, 3], False), (16, [9, -1], False), (16, [], False),
                          (16, [2, 2, 2, 1, 1], False), (16, [2, 3, 3], True), (16, [0, 8], True)):
        with pytest.raises(sk.SkError):
            sk.sk_rope_axes(rot, sec, cycled=cyc)


def test_axes_write_refusals(sk):
    call = caller(sk.lib().sk_rope_axes_and_cache, dict(
        q=FAKE, k=FAKE, v=FAKE, qs=1024, ks=256, vs=256, pos=FAKE, ps=4, na=3, fr=FAKE, ax=FAKE, rot=64, inter=0, f=1.0,
        sl=FAKE, nt=4, hq=8, hkv=2, d=128, qo=FAKE, pg=FAKE, dt=0, ksc=1.0, vsc=1.0, nb=8, page=16, acc=None, pp=None,
        st=None))
    assert call(d=64) == -3 and call(page=32) == -3 and call(rot=24) == -3 and call(rot=144) == -3
    for kw in (dict(na=0), dict(na=5), dict(ps=3), dict(ps=-4), dict(ax=None), dict(pos=None), dict(fr=None),
               dict(nt=-1), dict(hq=0), dict(dt=2), dict(f=0.0), dict(dt=1, ksc=0.0), dict(q=None), dict(sl=None),
               dict(qs=1023), dict(ks=248), dict(q=ODD), dict(pg=ODD), dict(qo=ODD)):
        assert call(**kw) == -1, kw
    assert call(nt=0, q=None, k=None, v=None, pos=None, sl=None, qo=None, pg=None) == 0


def test_axes_may_share_their_positions(sk):
    """A stride of 0 between the axes: one row of positions for all of them, as text has.  (The write refuses the heads
    after it has taken the positions' stride.)"""
    call = caller(sk.lib().sk_rope_axes_and_cache, dict(
        q=FAKE, k=FAKE, v=FAKE, qs=1024, ks=256, vs=256, pos=FAKE, ps=0, na=3, fr=FAKE, ax=FAKE, rot=64, inter=0, f=1.0,
        sl=FAKE, nt=4, hq=8, hkv=2, d=64, qo=FAKE, pg=FAKE, dt=0, ksc=1.0, vsc=1.0, nb=8, page=16, acc=None, pp=None,
        st=None))
    assert call() == -3
    for ps in (-1, 1, 2, 3):
        assert call(ps=ps) == -1, ps


def test_binding_checks_shapes_before_raw_pointers(sk):
    bf, i32, i64 = torch.bfloat16, torch.int32, torch.int64

    def axes(**kw):
        a = dict(q=torch.zeros(4, 8, 128, dtype=bf), k=torch.zeros(4, 2, 128, dtype=bf),
                 v=torch.zeros(4, 2, 128, dtype=bf), pos=torch.zeros(3, 4, dtype=i64),
                 fr=torch.zeros(32, dtype=torch.float64), ax=torch.zeros(32, dtype=torch.uint8),
                 sl=torch.zeros(4, dtype=i64), pg=torch.zeros(3, 2, 16, 256, dtype=bf),
                 qo=torch.zeros(4, 8, 128, dtype=bf), acc=None, pp=None)
        a.update(kw)
        return sk.sk_rope_axes_and_cache(a["q"], a["k"], a["v"], a["pos"], a["fr"], a["ax"], a["sl"], a["pg"], a["qo"],
                                         acc_pages=a["acc"], pos_pages=a["pp"])

    for kw in (dict(pos=torch.zeros(3, 5, dtype=i64)), dict(pos=torch.zeros(4, dtype=i64)),
               dict(pos=torch.zeros(3, 4, dtype=i32)), dict(pos=torch.zeros(3, 8, dtype=i64)[:, ::2]),
               dict(ax=torch.zeros(31, dtype=torch.uint8)), dict(ax=torch.zeros(32, dtype=i32)),
               dict(fr=torch.zeros(2, 16, dtype=torch.float64)), dict(q=torch.zeros(4, 8, 128)),
               dict(k=torch.zeros(5, 2, 128, dtype=bf)), dict(sl=torch.zeros(3, dtype=i64)),
               dict(qo=torch.zeros(4, 8, 64, dtype=bf)), dict(pg=torch.zeros(3, 1, 16, 256, dtype=bf)),
               dict(acc=torch.zeros(3, 2, 8)), dict(pp=torch.zeros(3, 2, 16)), dict()):
        with pytest.raises(ValueError):
            axes(**kw)

    def window(**kw):
        a = dict(q=torch.zeros(4, 8, 128, dtype=bf), pg=torch.zeros(3, 2, 16, 256, dtype=bf),
                 bt=torch.zeros(2, 5, dtype=i32), lens=torch.zeros(2, dtype=i32), cu=torch.zeros(3, dtype=i32), out=None,
                 lse=None)
        a.update(kw)
        return sk.paged_window_attention(a["q"], a["pg"], a["bt"], a["lens"], a["cu"], window=8, max_q_len=2,
                                         sm_scale=0.1, out=a["out"], lse=a["lse"])

    for kw in (dict(q=torch.zeros(4, 8, 128)), dict(q=torch.zeros(4, 8, 64, dtype=bf)),
               dict(pg=torch.zeros(3, 3, 16, 256, dtype=bf)), dict(bt=torch.zeros(1, 5, dtype=i32)),
               dict(bt=torch.zeros(2, 5, dtype=i64)), dict(lens=torch.zeros(2, dtype=i64)),
               dict(cu=torch.zeros(4, dtype=i32)), dict(out=torch.zeros(4, 8, 64, dtype=bf)),
               dict(lse=torch.zeros(4, 7)), dict()):
        with pytest.raises(ValueError):
            window(**kw)
