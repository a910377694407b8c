"""sk_rope_axes_and_cache against the rotation in 64 bits, each pair turned by its own axis's position.

Tolerances as for sk_rope_and_cache: the angle is off by at most 2^-24 of a half revolution's float plus sincospif's 2
ulp, the two products and their sum round in fp32: under 2^-21 (|a| + |b|) f for a pair (a, b); bf16 adds half a step,
2^-8, e4m3 2^-4 (2^-10 in the subnormals' steps of 2^-9)."""
import numpy as np
import pytest
import torch

import paged_split_kv_gb300 as sk
from test_rope_gpu import D, DEV, PAGE, bf16_bound, setup

pytestmark = pytest.mark.gpu


def turned(x, pos, axes, freqs, inter, f):
    """x [nt, heads, 128] turned in 64 bits, and the size |a| + |b| (times f) of each element's pair."""
    x = x.double().cpu()
    half = freqs.numel()
    ang = pos.cpu()[axes.cpu().long()].double().t() * freqs.cpu()[None, :]
    c, s = torch.cos(ang)[:, None, :] * f, torch.sin(ang)[:, None, :] * f
    a = slice(0, 2 * half, 2) if inter else slice(0, half)
    b = slice(1, 2 * half, 2) if inter else slice(half, 2 * half)
    y, size = x.clone(), x.abs()
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    both = (x[..., a].abs() + x[..., b].abs()) * f
    size[..., a], size[..., b] = both, both
    return y, size


def check(q, k, v, slots, pages0, pages, pos, axes, freqs, q_out, inter, f, fp8, ks, vs):
    want, size = turned(q, pos, axes, freqs, inter, f)
    err = (q_out.double().cpu() - want).abs()
    assert bool((err <= bf16_bound(want, size)).all()), float((err / bf16_bound(want, size)).max())
    sl = slots.cpu().numpy()
    ok = sl >= 0
    got = pages.double().cpu()[sl[ok] // PAGE, :, sl[ok] % PAGE]
    want, size = turned(k, pos, axes, freqs, inter, f)
    want, size = want[ok] / ks, size[ok] / ks
    val = v.double().cpu()[ok] / vs
    if fp8:
        want, val = want.clamp(-448, 448), val.clamp(-448, 448)
        step = lambda t: torch.clamp(t.abs() * 2.0 ** -4, min=2.0 ** -10)
        assert bool(((got[..., :D] - want).abs() <= step(want) + size * 2.0 ** -21).all())
        # the division rounds to fp32 before the code is chosen
        assert bool(((got[..., D:] - val).abs() <= step(val) + val.abs() * 2.0 ** -23).all())
    else:
        assert bool(((got[..., :D] - want).abs() <= bf16_bound(want, size)).all())
        assert torch.equal(got[..., D:], val)
    written = np.zeros(pages0.shape[0] * PAGE, bool)
    written[sl[ok]] = True
    keep = ~written.reshape(-1, PAGE)
    raw = pages.view(torch.uint8 if fp8 else torch.int16).cpu().numpy()
    raw = raw if fp8 else raw.view(np.uint16)
    np.testing.assert_array_equal(np.moveaxis(raw, 1, 2)[keep], np.moveaxis(pages0, 1, 2)[keep])


def positions(naxes, nt, far, seed, pad=0):
    p = torch.as_tensor(np.random.default_rng(seed).integers(0, far + 1, size=(naxes, nt + pad)), device=DEV)
    return p[:, :nt]


def sections_of(half, naxes):
    each = half // (naxes + 1)
    return [half - each * (naxes - 1)] + [each] * (naxes - 1)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("cycled", [False, True])
@pytest.mark.parametrize("naxes,rot", [(1, 64), (2, 16), (3, 128), (3, 48), (4, 128)])
@pytest.mark.parametrize("nt,hq,hkv,fp8", [(1, 1, 1, False), (37, 32, 8, False), (65, 5, 1, True), (300, 64, 16, True),
                                           (7, 96, 3, False)])
def test_turn_and_write(nt, hq, hkv, fp8, naxes, rot, cycled, inter):
    ks, vs = ((0.03, 0.25) if rot == 64 else (0.25, 0.5)) if fp8 else (1.0, 1.0)
    f = 1.0 if rot != 48 else 1.25
    q, k, v, slots, pages0, pages, _, freqs = setup(nt, hq, hkv, rot, fp8, 10, nt + rot)
    pos = positions(naxes, nt, 3000000, nt, pad=naxes)
    axes = sk.sk_rope_axes(rot, sections_of(rot // 2, naxes), cycled=cycled, device=DEV)
    q_out = torch.full((nt, hq, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    assert sk.sk_rope_axes_and_cache(q, k, v, pos, freqs, axes, slots, pages, q_out, interleaved=inter, attn_factor=f,
                                     k_scale=ks, v_scale=vs) == sk.SK_OK
    assert sk.sk_get_device_status() == 0
    check(q, k, v, slots, pages0, pages, pos, axes, freqs, q_out, inter, f, fp8, ks, vs)


@pytest.mark.parametrize("fp8", [False, True])
def test_equal_positions_are_the_single_axis_write(fp8):
    """Text: the same position on every axis gives the bits of sk_rope_and_cache."""
    q, k, v, slots, pages0, pages, pos, freqs = setup(70, 16, 2, 128, fp8, 50000, 3)
    axes = sk.sk_rope_axes(128, [16, 24, 24], device=DEV)
    other = torch.as_tensor(pages0 if fp8 else pages0.view(np.int16), device=DEV).view(pages.dtype)
    a, b = torch.empty_like(q.contiguous()), torch.empty_like(q.contiguous())
    sk.sk_rope_and_cache(q, k, v, pos, freqs, slots, pages, a, k_scale=0.5 if fp8 else 1.0)
    sk.sk_rope_axes_and_cache(q, k, v, pos.expand(3, 70).contiguous(), freqs, axes, slots, other, b,
                              k_scale=0.5 if fp8 else 1.0)
    assert torch.equal(a, b) and torch.equal(pages.view(torch.uint8), other.view(torch.uint8))
    assert sk.sk_get_device_status() == 0


@pytest.mark.parametrize("nt", [1, 70])
def test_one_row_of_positions_for_all_axes(nt):
    q, k, v, slots, pages0, pages, pos, freqs = setup(nt, 16, 2, 128, False, 50000, 4)
    axes = sk.sk_rope_axes(128, [16, 24, 24], device=DEV)
    other = pages.clone()
    a, b = torch.empty_like(q.contiguous()), torch.empty_like(q.contiguous())
    sk.sk_rope_axes_and_cache(q, k, v, pos.expand(3, nt).contiguous(), freqs, axes, slots, pages, a)
    sk.sk_rope_axes_and_cache(q, k, v, pos.expand(3, nt), freqs, axes, slots, other, b)
    assert torch.equal(a, b) and torch.equal(pages.view(torch.int16), other.view(torch.int16))
    check(q, k, v, slots, pages0, pages, pos.expand(3, nt), axes, freqs, a, False, 1.0, False, 1.0, 1.0)
    assert sk.sk_get_device_status() == 0


def test_more_tokens_than_ctas_and_the_state_of_eviction():
    q, k, v, slots, pages0, pages, _, freqs = setup(2500, 8, 2, 64, False, 1000, 5, fused=False)
    pos = positions(3, 2500, 40000, 5)
    axes = torch.as_tensor(np.random.default_rng(1).integers(0, 3, size=32).astype(np.uint8), device=DEV)
    nb = pages.shape[0]
    acc = torch.rand(nb, 2, PAGE, device=DEV) + 1
    pp = torch.full((nb, 2, PAGE), -5, dtype=torch.int32, device=DEV)
    acc0, pp0 = acc.clone(), pp.clone()
    q_out = torch.empty_like(q)
    sk.sk_rope_axes_and_cache(q, k, v, pos, freqs, axes, slots, pages, q_out, acc_pages=acc, pos_pages=pp)
    assert sk.sk_get_device_status() == 0
    check(q, k, v, slots, pages0, pages, pos, axes, freqs, q_out, False, 1.0, False, 1.0, 1.0)
    ok = slots >= 0
    sl = slots[ok]
    acc0[sl // PAGE, :, sl % PAGE] = 0
    pp0[sl // PAGE, :, sl % PAGE] = pos[0][ok].to(torch.int32)[:, None]
    assert torch.equal(acc, acc0) and torch.equal(pp, pp0)


def image_between_texts(words, side, more):
    """Positions [time, height, width] of text, a still image of side x side patches and text behind it."""
    text = lambda at, n: (at + torch.arange(n)).expand(3, n)
    cells = torch.stack([torch.zeros(side, side), *torch.meshgrid(torch.arange(side), torch.arange(side), indexing="ij")])
    return torch.cat([text(0, words), words + cells.reshape(3, -1).long(), text(words + side, more)], 1).to(DEV)


@pytest.mark.parametrize("cycled", [False, True])
def test_the_latest_rows_of_an_image_and_text_stay(cycled):
    """The token's place as an axis without pairs: the rotation is that of the other axes, and eviction keeps the last
    `recent` tokens, although an image of more patches than the budget has the same time throughout."""
    words, side, more, budget, recent, hkv = 100, 40, 200, 512, 256, 2
    grid = image_between_texts(words, side, more)
    n = grid.shape[1]
    q, k, v, slots, pages0, pages, _, freqs = setup(n, 4, hkv, 128, False, 10, 12, holes=False)
    place = torch.arange(n, device=DEV)
    axes = sk.sk_rope_axes(128, [24, 20, 20], cycled=cycled, device=DEV)
    blocks = torch.arange(-(-n // PAGE), device=DEV, dtype=torch.int32).flip(0)[None]
    at = blocks[0].long()[place // PAGE] * PAGE + place % PAGE
    state = [torch.zeros(pages.shape[:3], device=DEV), torch.full(pages.shape[:3], -7, dtype=torch.int32, device=DEV)]
    a, b = torch.empty((n, 4, D), dtype=torch.bfloat16, device=DEV), torch.empty((n, 4, D), dtype=torch.bfloat16, device=DEV)
    other = pages.clone()
    sk.sk_rope_axes_and_cache(q, k, v, grid, freqs, axes, at, other, a)
    sk.sk_rope_axes_and_cache(q, k, v, torch.cat([place[None], grid]), freqs, axes + 1, at, pages, b, acc_pages=state[0],
                              pos_pages=state[1])
    assert torch.equal(a, b) and torch.equal(pages.view(torch.int16), other.view(torch.int16))
    # the image weighs the most, the last text the least
    state[0].view(-1, PAGE)[:] = 1.0
    state[0][at[words:words + side * side] // PAGE, :, at[words:words + side * side] % PAGE] = 5.0
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    new = sk.evict_rows(pages, *state, blocks, lens, lens, budget=budget, recent=recent)
    assert new.tolist() == [budget] and sk.sk_get_device_status() == 0
    rows = torch.arange(budget, device=DEV)
    for h in range(hkv):
        kept = state[1][blocks[0].long()[rows // PAGE], h, rows % PAGE].sort().values
        # the last `recent`; of the others the heaviest, ties to the lower rows: the image's first patches
        assert torch.equal(kept, torch.cat([words + torch.arange(budget - recent), n - recent + torch.arange(recent)]).to(kept))
        keys = pages[blocks[0].long()[rows // PAGE], h, rows % PAGE]
        order = state[1][blocks[0].long()[rows // PAGE], h, rows % PAGE].long()
        assert torch.equal(keys, other[at[order] // PAGE, h, at[order] % PAGE])


def test_in_place_negative_and_far_positions():
    q, k, v, slots, pages0, pages, _, freqs = setup(40, 4, 2, 128, False, 10, 6, fused=False)
    pos = torch.as_tensor(np.random.default_rng(3).integers(-2 ** 31, 2 ** 31, size=(3, 40)), device=DEV)
    axes = sk.sk_rope_axes(128, [24, 20, 20], cycled=True, device=DEV)
    q0 = q.clone()
    sk.sk_rope_axes_and_cache(q, k, v, pos, freqs, axes, slots, pages, q)
    # the frequency in revolutions rounds twice, the test's product once, each by 2^-53 of the angle: 3 * 2^-22 at 2^31
    want, size = turned(q0, pos, axes, freqs, False, 1.0)
    err = (q.double().cpu() - want).abs()
    assert bool((err <= bf16_bound(want, size) + size * 3 * 2.0 ** -22).all())


def test_an_axis_that_is_none_does_not_turn():
    q, k, v, slots, pages0, pages, _, freqs = setup(20, 4, 2, 64, False, 100, 7)
    pos = positions(2, 20, 100, 7)
    axes = sk.sk_rope_axes(64, [16, 16], device=DEV)
    axes[3], axes[20] = 2, 255
    q_out = torch.empty((20, 4, D), dtype=torch.bfloat16, device=DEV)
    sk.sk_get_device_status(clear=True)
    sk.sk_rope_axes_and_cache(q, k, v, pos, freqs, axes, slots, pages, q_out)
    assert sk.sk_get_device_status() == sk.SK_DEV_BAD_SEQ
    still = torch.tensor([3, 20])
    f2 = freqs.clone()
    f2[still] = 0.0
    axes[still] = 0
    check(q, k, v, slots, pages0, pages, pos, axes, f2, q_out, False, 1.0, False, 1.0, 1.0)
    assert torch.equal(q_out[..., [3, 20, 35, 52]], q[..., [3, 20, 35, 52]])


def test_slots_past_the_end_and_no_tokens():
    q, k, v, slots, pages0, pages, _, freqs = setup(20, 4, 2, 64, True, 100, 7, holes=False)
    pos = positions(3, 20, 100, 8)
    axes = sk.sk_rope_axes(64, [12, 10, 10], cycled=True, device=DEV)
    slots[3], slots[9] = pages.shape[0] * PAGE, 2 ** 40
    q_out = torch.empty((20, 4, D), dtype=torch.bfloat16, device=DEV)
    sk.sk_get_device_status(clear=True)
    sk.sk_rope_axes_and_cache(q, k, v, pos, freqs, axes, slots, pages, q_out, k_scale=0.5, v_scale=0.5)
    assert sk.sk_get_device_status() == sk.SK_DEV_BAD_BLOCK
    slots[[3, 9]] = -1
    check(q, k, v, slots, pages0, pages, pos, axes, freqs, q_out, False, 1.0, True, 0.5, 0.5)
    before = pages.view(torch.uint8).clone()
    assert sk.sk_rope_axes_and_cache(q[:0], k[:0], v[:0], pos[:, :0], freqs, axes, slots[:0], pages, q_out[:0]) == sk.SK_OK
    assert torch.equal(pages.view(torch.uint8), before)


def test_another_stream_and_a_graph():
    q, k, v, slots, pages0, pages, _, freqs = setup(64, 32, 2, 128, False, 5000, 8)
    pos = positions(3, 64, 5000, 9)
    axes = sk.sk_rope_axes(128, [16, 24, 24], device=DEV)
    q_out = torch.zeros((64, 32, D), dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            sk.sk_rope_axes_and_cache(q, k, v, pos, freqs, axes, slots, pages, q_out)
    pos.add_(17)
    graph.replay()
    torch.cuda.synchronize()
    check(q, k, v, slots, pages0, pages, pos, axes, freqs, q_out, False, 1.0, False, 1.0, 1.0)


@pytest.mark.parametrize("fp8", [False, True])
def test_slots_past_4_gb_and_2_to_the_31_elements(fp8):
    """The same rows at the near and the far end of a cache."""
    q, k, v, slots, pages0, pages, _, freqs = setup(70, 8, 2, 128, fp8, 1000, 11)
    pos = positions(3, 70, 1000, 11)
    axes = sk.sk_rope_axes(128, [16, 24, 24], device=DEV)
    far = torch.empty((1200000 if fp8 else 600000, *pages.shape[1:]), dtype=pages.dtype, device=DEV)
    shift = far.shape[0] - pages.shape[0]
    far[shift:].copy_(pages)
    out = [torch.empty((70, 8, D), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    sk.sk_rope_axes_and_cache(q, k, v, pos, freqs, axes, slots, pages, out[0], k_scale=0.5, v_scale=0.5)
    sk.sk_rope_axes_and_cache(q, k, v, pos, freqs, axes, torch.where(slots >= 0, slots + shift * PAGE, slots), far, out[1],
                              k_scale=0.5, v_scale=0.5)
    assert sk.sk_get_device_status() == 0
    assert torch.equal(out[0], out[1])
    assert torch.equal(far[shift:].view(torch.uint8), pages.view(torch.uint8))
