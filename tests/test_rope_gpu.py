"""sk_rope_and_cache against the rotation in 64 bits (complex multiplication), the KV write's own oracle for V,
and the rows that must stay as they were.

Tolerances.  The kernel's angle is off by at most 2^-24 of a half revolution's float plus sincospif's 2 ulp, and the
two products and their sum round in fp32: together under 2^-21 (|a| + |b|) f for a pair (a, b).  bf16 results add half
a step, 2^-8 of the value's binade; e4m3 codes add 2^-4, or 2^-10 in the subnormals' steps of 2^-9."""
import numpy as np
import pytest
import torch

import paged_split_kv_gb300 as sk
from helpers import KV_BF16, KV_FP8, to_bf16_bits
from oracle import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
D, PAGE = 128, 16


def rotated(x, pos, freqs, inter, f):
    """x [nt, heads, 128] turned in 64 bits, and the size |a| + |b| (times f) of each element's pair."""
    x = x.double().cpu()
    rot = 2 * freqs.numel()
    ang = pos.cpu().double()[:, None] * freqs.cpu()[None, :]
    turn = torch.polar(torch.full_like(ang, f), ang)[:, None, :]
    a = slice(0, rot, 2) if inter else slice(0, rot // 2)
    b = slice(1, rot, 2) if inter else slice(rot // 2, rot)
    z = torch.complex(x[..., a].contiguous(), x[..., b].contiguous()) * turn
    y, size = x.clone(), x.abs()
    y[..., a], y[..., b] = z.real, z.imag
    both = (x[..., a].abs() + x[..., b].abs()) * f
    size[..., a], size[..., b] = both, both
    return y, size


def bf16_bound(y, size):
    return y.abs() * 2.0 ** -8 + size * 2.0 ** -21 + 1e-38


def setup(nt, hq, hkv, rot, fp8, far, seed, fused=True, holes=True):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rng = np.random.default_rng(seed)
    if fused:
        qkv = torch.randn(nt, (hq + 2 * hkv) * D, generator=g, device=DEV).to(torch.bfloat16)
        q = qkv[:, :hq * D].view(nt, hq, D)
        k = qkv[:, hq * D:(hq + hkv) * D].view(nt, hkv, D)
        v = qkv[:, (hq + hkv) * D:].view(nt, hkv, D)
    else:
        q, k, v = (torch.randn(nt, h, D, generator=g, device=DEV).to(torch.bfloat16) for h in (hq, hkv, hkv))
    nb = nt // PAGE + 4
    slots = rng.permutation(nb * PAGE)[:nt].astype(np.int64)
    if holes and nt > 2:
        slots[rng.choice(nt, size=max(1, nt // 7), replace=False)] = -1
    pages0 = rng.integers(0, 256, size=(nb, hkv, PAGE, 2 * D), dtype=np.uint8) if fp8 else \
        rng.integers(0, 1 << 16, size=(nb, hkv, PAGE, 2 * D), dtype=np.uint16)
    pages = torch.as_tensor(pages0, device=DEV).view(torch.float8_e4m3fn) if fp8 else \
        torch.as_tensor(pages0.view(np.int16), device=DEV).view(torch.bfloat16)
    pos = torch.as_tensor(rng.integers(0, far + 1, size=nt).astype(np.int64), device=DEV)
    freqs, _ = sk.sk_rope_frequencies(rot, 10000.0, device=DEV)
    return q, k, v, torch.as_tensor(slots, device=DEV), pages0, pages, pos, freqs


def check(q, k, v, slots, pages0, pages, pos, freqs, q_out, inter, f, fp8, ks, vs):
    want, size = rotated(q, pos, freqs, inter, f)
    err = (q_out.double().cpu() - want).abs()
    assert bool((err <= bf16_bound(want, size)).all()), float((err / bf16_bound(want, size)).max())
    # V, and every row without a slot: the bits that the KV write gives
    bits = lambda t: t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
    dt = KV_FP8 if fp8 else KV_BF16
    base = oracle.reshape_and_cache(bits(k), bits(v), slots.cpu().numpy(), pages0.copy(), dt, ks, vs)
    got = pages.view(torch.uint8 if fp8 else torch.int16).cpu().numpy()
    got = got if fp8 else got.view(np.uint16)
    np.testing.assert_array_equal(got[..., D:], base[..., D:])
    sl = slots.cpu().numpy()
    written = np.zeros(got.shape[0] * PAGE, bool)
    written[sl[sl >= 0]] = True
    keep = ~written.reshape(-1, PAGE)
    np.testing.assert_array_equal(np.moveaxis(got, 1, 2)[keep], np.moveaxis(base, 1, 2)[keep])
    # K
    ok = sl >= 0
    want, size = rotated(k, pos, freqs, inter, f)
    want, size = want[ok] / ks, size[ok] / ks
    if not fp8:
        row = pages.double().cpu()[sl[ok] // PAGE, :, sl[ok] % PAGE, :D]
        assert bool(((row - want).abs() <= bf16_bound(want, size)).all())
    else:
        row = pages.float().double().cpu()[sl[ok] // PAGE, :, sl[ok] % PAGE, :D]
        want = want.clamp(-448, 448)
        bound = torch.clamp(want.abs() * 2.0 ** -4, min=2.0 ** -10) + size * 2.0 ** -21
        assert bool(((row - want).abs() <= bound).all())


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [16, 48, 64, 128])
@pytest.mark.parametrize("nt,hq,hkv,fp8", [(1, 1, 1, False), (37, 32, 8, False), (65, 5, 1, True), (300, 64, 16, True),
                                           (7, 96, 3, False)])
def test_turn_and_write(nt, hq, hkv, fp8, rot, inter):
    ks, vs = ((0.03, 0.25) if rot == 64 else (0.25, 0.5)) if fp8 else (1.0, 1.0)
    f = 1.0 if rot != 48 else 1.25
    q, k, v, slots, pages0, pages, pos, freqs = setup(nt, hq, hkv, rot, fp8, 3000000, nt + rot)
    q_out = torch.full((nt, hq, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    assert sk.sk_rope_and_cache(q, k, v, pos, freqs, slots, pages, q_out, interleaved=inter, attn_factor=f,
                                k_scale=ks, v_scale=vs) == sk.SK_OK
    assert sk.sk_get_device_status() == 0
    check(q, k, v, slots, pages0, pages, pos, freqs, q_out, inter, f, fp8, ks, vs)


def test_more_tokens_than_ctas_and_the_state_of_eviction():
    """2500 tokens: CTAs take several in turn.  Weights and positions of the written slots, and of no others."""
    q, k, v, slots, pages0, pages, pos, freqs = setup(2500, 8, 2, 64, False, 1000, 5, fused=False)
    nb = pages.shape[0]
    acc = torch.rand(nb, 2, PAGE, device=DEV) + 1
    pp = torch.full((nb, 2, PAGE), -5, dtype=torch.int32, device=DEV)
    acc0, pp0 = acc.clone(), pp.clone()
    q_out = torch.empty_like(q)
    sk.sk_rope_and_cache(q, k, v, pos, freqs, slots, pages, q_out, acc_pages=acc, pos_pages=pp)
    assert sk.sk_get_device_status() == 0
    check(q, k, v, slots, pages0, pages, pos, freqs, q_out, False, 1.0, False, 1.0, 1.0)
    ok = slots >= 0
    sl = slots[ok]
    acc0[sl // PAGE, :, sl % PAGE] = 0
    pp0[sl // PAGE, :, sl % PAGE] = pos[ok].to(torch.int32)[:, None]
    assert torch.equal(acc, acc0) and torch.equal(pp, pp0)


def test_in_place_negative_and_far_positions():
    """q_out is q itself; positions of either sign up to 2^31 keep their angle."""
    q, k, v, slots, pages0, pages, pos, freqs = setup(40, 4, 2, 128, False, 10, 6, fused=False)
    pos = torch.as_tensor(np.random.default_rng(3).integers(-2 ** 31, 2 ** 31, size=40), device=DEV)
    q0 = q.clone()
    sk.sk_rope_and_cache(q, k, v, pos, freqs, slots, pages, q)
    # the frequency in revolutions rounds twice, the test's product once, each by 2^-53 of the angle: 3 * 2^-22 at 2^31
    want, size = rotated(q0, pos, freqs, False, 1.0)
    err = (q.double().cpu() - want).abs()
    assert bool((err <= bf16_bound(want, size) + size * 3 * 2.0 ** -22).all())


def test_slots_past_the_end_and_no_tokens():
    q, k, v, slots, pages0, pages, pos, freqs = setup(20, 4, 2, 64, True, 100, 7, holes=False)
    slots[3] = pages.shape[0] * PAGE
    slots[9] = 2 ** 40
    q_out = torch.empty((20, 4, D), dtype=torch.bfloat16, device=DEV)
    sk.sk_get_device_status(clear=True)
    sk.sk_rope_and_cache(q, k, v, pos, freqs, slots, pages, q_out, k_scale=0.5, v_scale=0.5)
    assert sk.sk_get_device_status() == sk.SK_DEV_BAD_BLOCK
    slots[[3, 9]] = -1
    check(q, k, v, slots, pages0, pages, pos, freqs, q_out, False, 1.0, True, 0.5, 0.5)
    before = pages.view(torch.uint8).clone()
    assert sk.sk_rope_and_cache(q[:0], k[:0], v[:0], pos[:0], freqs, slots[:0], pages, q_out[:0]) == sk.SK_OK
    assert torch.equal(pages.view(torch.uint8), before)


def test_another_stream_and_a_graph():
    q, k, v, slots, pages0, pages, pos, freqs = setup(64, 32, 2, 128, False, 5000, 8)
    q_out = torch.zeros((64, 32, D), dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            sk.sk_rope_and_cache(q, k, v, pos, freqs, slots, pages, q_out)
    pos.add_(17)
    graph.replay()
    torch.cuda.synchronize()
    check(q, k, v, slots, pages0, pages, pos, freqs, q_out, False, 1.0, False, 1.0, 1.0)
