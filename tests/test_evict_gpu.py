"""Eviction: the rows that stay against a sort in NumPy, the moves against an index copy; whole numbers and copied
bytes, so everything is compared for equality."""
import numpy as np
import pytest
import torch

import paged_split_kv_gb300 as sk

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
PAGE = 16


def cache(lens, hkv, seed, fp8=False, weights=None, stride_extra=0, positions=True):
    """A cache of given lengths: pages of random bytes, weights, positions in no order, block table."""
    rng = np.random.default_rng(seed)
    npg = [(n + PAGE - 1) // PAGE for n in lens]
    nb = sum(npg) + 3
    perm = rng.permutation(nb).astype(np.int32)
    bt = np.full((len(lens), max(1, max(npg)) + stride_extra), -1, np.int32)
    k = 0
    for s, n in enumerate(npg):
        bt[s, :n] = perm[k:k + n]
        k += n
    acc = (weights(rng, (nb, hkv, PAGE)) if weights else np.exp(rng.normal(0, 2, (nb, hkv, PAGE)))).astype(np.float32)
    pos = np.full((nb, hkv, PAGE), -1, np.int32)
    for s, n in enumerate(lens):
        r = np.arange(n)
        for h in range(hkv):
            pos[bt[s, r // PAGE], h, r % PAGE] = rng.permutation(n) if positions else r
    pages = rng.integers(0, 256, size=(nb, hkv, PAGE, 256 * (1 if fp8 else 2)), dtype=np.uint8)
    return bt, acc, pos, pages


def reference(bt, acc, pos, lens, next_pos, hkv, budget, recent):
    """[(s, h)] -> (source rows, destination rows)."""
    out = {}
    for s, n in enumerate(lens):
        r = np.arange(n)
        for h in range(hkv):
            if n <= budget:
                out[s, h] = (np.zeros(0, int), np.zeros(0, int))
                continue
            w = acc[bt[s, r // PAGE], h, r % PAGE].astype(np.float64)
            w[np.isnan(w)] = -np.inf
            near = pos[bt[s, r // PAGE], h, r % PAGE] >= next_pos[s] - recent
            others = r[~near]
            order = np.concatenate([r[near], others[np.lexsort((others, -w[others]))]])
            stays = np.zeros(n, bool)
            stays[order[:budget]] = True
            out[s, h] = (r[stays & (r >= budget)], r[~stays & (r < budget)])
    return out


def dev(x, dt=None):
    return torch.as_tensor(x, device=DEV) if dt is None else torch.as_tensor(x, dtype=dt, device=DEV)


def run_select(bt, acc, pos, lens, next_pos, hkv, budget, recent, max_len=None, cap=None):
    bs = len(lens)
    m = max_len if max_len is not None else bt.shape[1] * PAGE
    cap = cap or sk.sk_evict_capacity(budget, m)
    src = torch.full((bs, hkv, cap), -9, dtype=torch.int32, device=DEV)
    dst = torch.full((bs, hkv, cap), -9, dtype=torch.int32, device=DEV)
    counts = torch.full((bs, hkv), -9, dtype=torch.int32, device=DEV)
    new = torch.full((bs,), -9, dtype=torch.int32, device=DEV)
    sk.sk_evict_select(dev(acc), dev(pos), dev(bt), dev(lens, torch.int32), dev(next_pos, torch.int32), src, dst,
                       counts, new, budget=budget, recent=recent, max_seq_len=max_len)
    return src, dst, counts, new


def check_select(got, want, lens, hkv, budget):
    src, dst, counts, new = (t.cpu().numpy() for t in got)
    np.testing.assert_array_equal(new, np.minimum(lens, budget))
    for (s, h), (a, b) in want.items():
        n = counts[s, h]
        assert n == len(a) == len(b), (s, h, n, len(a))
        np.testing.assert_array_equal(src[s, h, :n], a)
        np.testing.assert_array_equal(dst[s, h, :n], b)
        assert (src[s, h, n:] == -9).all() and (dst[s, h, n:] == -9).all()     # left as they were


def flat(rng, shape):
    return np.full(shape, 0.25)


def coarse(rng, shape):
    return rng.integers(0, 3, size=shape)


def odd(rng, shape):
    x = rng.normal(0, 1, shape)
    x.reshape(-1)[::7] = np.nan
    x.reshape(-1)[1::11] = np.inf
    x.reshape(-1)[2::13] = -np.inf
    x.reshape(-1)[3::5] = 0.0
    x.reshape(-1)[4::17] = -0.0
    return x


@pytest.mark.parametrize("weights", [None, flat, coarse, odd])
@pytest.mark.parametrize("lens,hkv,budget,recent", [
    ([1], 1, 1, 0), ([2], 2, 1, 1), ([17, 0, 1, 16, 300], 2, 16, 4), ([2049, 2050, 2048, 7], 2, 2048, 100),
    ([1023, 1024, 1025, 3000], 3, 1000, 0), ([5000], 1, 4999, 4999), ([5000, 40], 5, 33, 33)])
def test_select_against_a_sort(lens, hkv, budget, recent, weights):
    bt, acc, pos, _ = cache(lens, hkv, sum(lens) + budget, weights=weights)
    next_pos = np.asarray(lens)
    got = run_select(bt, acc, pos, lens, next_pos, hkv, budget, recent)
    assert sk.sk_get_device_status() == 0
    check_select(got, reference(bt, acc, pos, lens, next_pos, hkv, budget, recent), lens, hkv, budget)


@pytest.mark.parametrize("length,budget,recent", [(24577, 24576, 64), (60000, 8192, 512), (100001, 60000, 3),
                                                  (248000, 1, 0), (400000, 1000, 999), (786432, 700000, 5000),
                                                  (1000001, 300000, 7)])
def test_select_over_clusters(length, budget, recent):
    """Lengths around and past what one CTA, and a cluster, keeps in shared memory."""
    lens = [length, length // 3]
    bt, acc, pos, _ = cache(lens, 1, length, weights=coarse if length == 60000 else None)
    got = run_select(bt, acc, pos, lens, np.asarray(lens), 1, budget, recent)
    assert sk.sk_get_device_status() == 0
    check_select(got, reference(bt, acc, pos, lens, np.asarray(lens), 1, budget, recent), lens, 1, budget)


def test_many_long_rows():
    """More pairs than SMs for clusters: a CTA each, most of whose rows are past what it keeps."""
    lens = [60001] * 19 + [150000]
    bt, acc, pos, _ = cache(lens, 8, 5, weights=coarse)
    got = run_select(bt, acc, pos, lens, np.asarray(lens), 8, 40000, 300)
    assert sk.sk_get_device_status() == 0
    check_select(got, reference(bt, acc, pos, lens, np.asarray(lens), 8, 40000, 300), lens, 8, 40000)


def test_more_recent_rows_than_the_budget():
    """Positions that repeat can leave more recent rows than fit: the lower ones stay."""
    bt, acc, pos, _ = cache([200], 1, 3)
    pos[:] = 7
    got = run_select(bt, acc, pos, [200], [8], 1, 50, 1)
    check_select(got, {(0, 0): (np.zeros(0, int), np.zeros(0, int))}, [200], 1, 50)


def test_bad_lengths_and_blocks_are_reported():
    lens = [100, 100, 300, 40]
    bt, acc, pos, _ = cache(lens, 2, 4)
    sk.sk_get_device_status(clear=True)
    src, dst, counts, new = run_select(bt, acc, pos, lens, lens, 2, 32, 0, max_len=250)
    assert sk.sk_get_device_status() == sk.SK_DEV_BAD_SEQ
    assert counts.cpu().numpy()[2].tolist() == [0, 0] and new.cpu().tolist() == [32, 32, 300, 32]
    lens[2] = -1
    got = run_select(bt, acc, pos, lens, lens, 2, 32, 0)
    assert sk.sk_get_device_status() == sk.SK_DEV_BAD_SEQ
    assert got[2].cpu().numpy()[2].tolist() == [0, 0] and got[3].cpu().tolist()[2] == -1
    lens[2] = 300
    bad = bt.copy()
    bad[0, 2], bad[1, 0] = 10 ** 6, -1          # rows 32..47 of sequence 0 and 0..15 of sequence 1
    got = run_select(bad, acc, pos, lens, lens, 2, 32, 0)
    assert sk.sk_get_device_status() == sk.SK_DEV_BAD_BLOCK
    nb = acc.shape[0]
    acc2 = np.concatenate([acc, np.full((1, 2, PAGE), -np.inf, np.float32)])
    pos2 = np.concatenate([pos, np.full((1, 2, PAGE), -1, np.int32)])
    bad[0, 2] = bad[1, 0] = nb
    check_select(got, reference(bad, acc2, pos2, lens, lens, 2, 32, 0), lens, 2, 32)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,hkv,budget,recent", [([20], 1, 19, 0), ([2049, 100, 0, 2060], 2, 2048, 32),
                                                    ([700, 5000, 1], 4, 640, 64), ([9000] * 9, 8, 4000, 0)])
def test_evict_rows_moves_pages_weights_and_positions(fp8, lens, hkv, budget, recent):
    bt, acc, pos, pages = cache(lens, hkv, 11 + budget, fp8=fp8)
    want = reference(bt, acc, pos, lens, lens, hkv, budget, recent)
    pg = dev(pages).view(torch.uint8 if fp8 else torch.bfloat16)
    a, p = dev(acc), dev(pos)
    new = sk.evict_rows(pg, a, p, dev(bt), dev(lens, torch.int32), dev(lens, torch.int32), budget=budget,
                        recent=recent)
    assert sk.sk_get_device_status() == 0
    assert new.cpu().tolist() == [min(n, budget) for n in lens]
    for (s, h), (x, y) in want.items():
        for t in (pages, acc, pos):
            t[bt[s, y // PAGE], h, y % PAGE] = t[bt[s, x // PAGE], h, x % PAGE]
    np.testing.assert_array_equal(pg.view(torch.uint8).cpu().numpy(), pages)
    np.testing.assert_array_equal(a.cpu().numpy(), acc)
    np.testing.assert_array_equal(p.cpu().numpy(), pos)


def test_moves_out_of_range_are_skipped_and_reported():
    bt, acc, pos, pages = cache([64, 64], 1, 12)
    bt[1, 3] = -1
    src = dev([[[40, 64 * 9, -1, 41]], [[50, 20, 21, 22]]], torch.int32)
    dst = dev([[[0, 1, 2, 99999]], [[3, 4, 5, 6]]], torch.int32)
    counts = dev([[4], [9]], torch.int32)       # the second count is past the capacity
    pg, a, p = dev(pages).view(torch.bfloat16), dev(acc), dev(pos)
    sk.sk_get_device_status(clear=True)
    sk.sk_evict_move(src, dst, counts, dev(bt), pg, a, p)
    assert sk.sk_get_device_status() == sk.SK_DEV_BAD_SEQ | sk.SK_DEV_BAD_BLOCK
    for s, x, y in ((0, 40, 0), (1, 20, 4), (1, 21, 5), (1, 22, 6)):
        for t in (pages, acc, pos):
            t[bt[s, y // PAGE], 0, y % PAGE] = t[bt[s, x // PAGE], 0, x % PAGE]
    np.testing.assert_array_equal(pg.view(torch.uint8).cpu().numpy(), pages)
    np.testing.assert_array_equal(a.cpu().numpy(), acc)
    np.testing.assert_array_equal(p.cpu().numpy(), pos)


def test_a_captured_eviction_follows_its_inputs():
    lens, hkv = [500, 900], 2
    bt, acc, pos, pages = cache(lens, hkv, 13)
    pg, a, p = dev(pages).view(torch.bfloat16), dev(acc), dev(pos)
    tl, tb = dev(lens, torch.int32), dev(bt)
    ws = {}
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        new = sk.evict_rows(pg, a, p, tb, tl, tl, budget=300, recent=10, workspace=ws)
    acc = np.random.default_rng(1).random(acc.shape, dtype=np.float32)
    a.copy_(dev(acc))
    tl.copy_(dev([400, 899], torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    want = reference(bt, acc, pos, [400, 899], [400, 899], hkv, 300, 10)
    for (s, h), (x, y) in want.items():
        for t in (pages, acc, pos):
            t[bt[s, y // PAGE], h, y % PAGE] = t[bt[s, x // PAGE], h, x % PAGE]
    np.testing.assert_array_equal(pg.view(torch.uint8).cpu().numpy(), pages)
    np.testing.assert_array_equal(p.cpu().numpy(), pos)
    assert new.cpu().tolist() == [300, 300]
