"""Windowed attention where values are at the edge: keys whose scores are minus infinity, keys far above the rest, queries of
all sizes (bounds: window_helpers), and windows of any whole number."""
import math

import pytest
import torch

import paged_split_kv_gb300 as sk
from window_helpers import DEV, PAGE, batch, check, reference, run

pytestmark = pytest.mark.gpu
D = 128


@pytest.mark.parametrize("lens,qs,hq,hkv,window,sinks,gone", [
    ([100], [1], 4, 1, 90, 4, range(16)),                        # the sinks and the first keys of the window
    ([100], [20], 4, 1, 60, 4, range(48)),
    ([128, 90, 17], [3, 2, 1], 8, 2, 70, 0, range(60, 80)),
    ([1000, 700], [4, 3], 16, 2, 600, 4, range(380, 520)),       # of whole tiles
    ([1000, 700], [140, 33], 16, 2, 400, 16, range(450, 640)),
    ([1000], [3], 5, 1, 900, 3, [k for k in range(900) if k % 128 < 16 or k % 128 > 100]),
    ([20000], [1], 8, 1, 19000, 4, [k for k in range(19900) if k % 128 < 16]),      # in every part of a cluster's unit
    ([9000] * 20, [2] * 20, 16, 8, 8000, 4, range(1100, 5000)),  # and of the runs'
    ([20000], [33], 8, 1, 18000, 0, range(2100, 15000)),
    ([300, 300], [2, 200], 8, 2, 16, 0, range(280, 299)),        # all that some rows see
])
def test_scores_of_minus_infinity(lens, qs, hq, hkv, window, sinks, gone):
    """Keys with an element of minus infinity where the queries are positive weigh nothing, wherever they lie."""
    b = batch(lens, qs, hq, hkv, False, 91, window, sinks, forget=False)
    b["q"][..., 0] = b["q"][..., 0].abs() + 0.5
    at = torch.tensor(list(gone), device=DEV)
    for s, n in enumerate(lens):
        k = at[at < n]
        b["kv"][b["bt"][s].long()[k // PAGE], :, k % PAGE, 0] = -math.inf
    out, lse = run(b)
    assert sk.sk_get_device_status() == 0
    check(b, out, lse, reference(b, list(gone)))


@pytest.mark.parametrize("code,nats", [(36.0, 12.7), (44.0, 15.6), (52.0, 18.4), (56.0, 19.8)])
@pytest.mark.parametrize("lens,qs,hq,hkv", [([20000], [1], 8, 1), ([6000, 3000], [4, 2], 8, 2), ([3000] * 100, [1] * 100, 8, 2),
                                            ([6000, 3000], [200, 64], 8, 2)])
@pytest.mark.parametrize("back", [None, 400, 1])
def test_a_key_far_above_the_rest_on_e4m3_pages(lens, qs, hq, hkv, back, code, nats):
    """A sink, a key in the window or the last one lies `nats` above scores that are nearly equal, and its V is 0: the output
    is what the others give."""
    b = batch(lens, qs, hq, hkv, True, 92, 2500, 4, forget=False)
    b["q"] *= 0.125
    b["q"][..., 0] = 8.0
    kv = b["kv"].view(torch.float8_e4m3fn)
    for s, n in enumerate(lens):
        kv[b["bt"][s, :(n + PAGE - 1) // PAGE].long(), :, :, 0] = 0.0
        r = 0 if back is None else n - back
        kv[b["bt"][s, r // PAGE].long(), :, r % PAGE, 0] = code
        kv[b["bt"][s, r // PAGE].long(), :, r % PAGE, D:] = 0.0
    # (rows that no token sees have lost one of their NaN)
    assert abs(8 * code * b["w"].k_scale * b["w"].sm_scale - nats) < 0.1
    out, lse = run(b)
    assert sk.sk_get_device_status() == 0
    check(b, out, lse)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("qs", [[2, 1], [70, 40]])
def test_queries_of_all_sizes(qs, fp8):
    """Rows of zeros, tiny and large ones beside each other; elements of very different size in one."""
    b = batch([400, 300], qs, 8, 2, fp8, 93, 200, 4)
    size = 2.0 ** torch.linspace(-30, 1, 8, device=DEV).round()
    b["q"] = (b["q"].float() * size[None, :, None]).bfloat16()
    b["q"][0, 0] = 0.0
    b["q"][:, 7, ::2] *= 2.0 ** -7
    out, lse = run(b)
    assert sk.sk_get_device_status() == 0
    check(b, out, lse)


@pytest.mark.parametrize("qs", [[1, 1], [50, 3]])
def test_windows_and_sinks_of_any_whole_number(qs):
    b = batch([300, 77], qs, 8, 2, False, 94, 2 ** 31 - 1, 0)
    want = run(b)
    check(b, *want)
    for kw in (dict(window=2 ** 31), dict(window=2 ** 32 + 5), dict(window=2 ** 63 - 1), dict(window=1, sinks=2 ** 40),
               dict(window=300, sinks=300)):
        out, lse = run(b, **kw)
        check(b, out, lse)
    for kw in (dict(window=0), dict(window=-2 ** 33 + 5), dict(sinks=-1)):
        with pytest.raises((sk.SkError, ValueError)):
            run(b, **kw)
    assert sk.sk_get_device_status() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,qs,hq,hkv,window,sinks", [
    ([9000], [300], 8, 2, 5000, 4), ([7000, 9001, 6500], [33, 260, 1], 16, 2, 4000, 70), ([12000], [130], 5, 1, 9000, 0),
    ([6200], [6200], 4, 1, 5000, 17), ([20001, 300], [70, 300], 12, 4, 6000, 4)])
@pytest.mark.parametrize("rising", [False, True])
def test_long_units(lens, qs, hq, hkv, window, sinks, rising, fp8):
    """Units of many key tiles, which take a tile in one go where all rows see it; scores that grow by far along the keys move
    the references again and again."""
    b = batch(lens, qs, hq, hkv, fp8, 95, window, sinks, gain=6.0 if rising else 1.0, forget=not rising)
    if rising:
        for s, n in enumerate(lens):
            for i in range(0, (n + PAGE - 1) // PAGE):
                blk = int(b["table"][s, i])
                k = b["kv"].view(torch.float8_e4m3fn)[blk, :, :, :D] if fp8 else b["kv"][blk, :, :, :D]
                k.copy_((k.float() * (0.05 + 2.0 * i * PAGE / n)).to(k.dtype))
    out, lse = run(b)
    assert sk.sk_get_device_status() == 0
    check(b, out, lse)
