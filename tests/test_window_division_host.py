"""The division of a windowed chunk call among its CTAs, on the CPU: the kernel's own arithmetic, compiled for the host.

Bound.  A run has an equal share of the batch's price.  A unit's price is its keys and 224, with a full window 288, rounded up
by 32 at most (two steps of 16); its tiles are its keys rounded up by less than 128.  So a share is at most the average of
key tiles and 2.5 for each unit of a run on average, and a cut moves by less than 4 tiles (512 keys) at either end.  Runs of
whole units are taken where the longest is then at most 1.1 times as long as the share and 6.25 tiles (800 keys) more.  Units
are dealt in turn where the dearest costs at most 1.4 times the average, and those left over are shared with 4 tiles more at
either end."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def library(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("division") / "division.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "paged_split_kv_gb300", "csrc"), "-o", so,
                    os.path.join(ROOT, "tests", "window_division.cpp")], check=True)
    return ctypes.CDLL(so)


@pytest.fixture(scope="module")
def longest_run(library):
    f = library.window_division

    def call(lens, qs, hq, hkv, window, count=152, deal=False):
        """Key tiles of the longest run, and the most that it may have."""
        n, units = len(lens), ctypes.c_int()
        tiles = (ctypes.c_int * count)()
        total = f(n, (ctypes.c_int * n)(*lens), (ctypes.c_int * n)(*qs), hq, hkv, window, 4, (max(lens) + 15) // 16, count,
                  int(deal), tiles, ctypes.byref(units))
        assert total >= 0 and sum(tiles) == total              # every unit is covered, in order
        return max(tiles), (1.4 if deal else 1.1) * (total + 2.5 * units.value) / count + 8

    return call


@pytest.mark.parametrize("deal", [False, True])
@pytest.mark.parametrize("group", [1, 3, 8, 9, 12, 16, 24, 32, 48, 71, 128, 129, 160, 300])
def test_the_longest_run_is_near_the_average(longest_run, group, deal):
    for window in (128, 1000, 4096):
        for hkv, tokens, cached in ((1, 2000, 0), (1, 4000, 0), (2, 2000, 100), (1, 3000, 2500), (4, 777, 0)):
            longest, most = longest_run([cached + tokens], [tokens], group * hkv, hkv, window, deal=deal)
            assert longest <= most, (window, hkv, tokens, cached)


@pytest.mark.parametrize("count", [1, 7, 152])
@pytest.mark.parametrize("group", [5, 8, 32, 200])
def test_many_sequences(longest_run, group, count):
    qs = [83 * (i + 1) for i in range(24)] + [1, 2, 0, 40]
    lens = [q + 57 * (i % 5) for i, q in enumerate(qs)]
    longest, most = longest_run(lens, qs, group, 1, 512, count=count)
    assert longest <= most


@pytest.mark.parametrize("group", [1, 8, 32, 48, 71, 128, 160, 300])
def test_a_window_of_more_rows_than_the_table_has(longest_run, group):
    for hkv, tokens, cached in ((1, 2000, 0), (2, 4000, 0), (2, 2000, 100), (1, 3000, 2500), (4, 777, 0), (1, 120000, 0)):
        longest, most = longest_run([cached + tokens], [tokens], group * hkv, hkv, 2 ** 31 - 1)
        assert longest <= most, (hkv, tokens, cached)


@pytest.mark.parametrize("group", [8, 32, 128])
def test_costs_past_32_bits_are_counted_in_coarser_steps(longest_run, group):
    longest, most = longest_run([120000], [120000], group, 1, 120000)
    assert longest <= most


@pytest.mark.parametrize("hkv", [1, 2, 8])
def test_a_step_whose_units_may_be_short_is_not_left_to_long_clusters(library, hkv):
    """One sequence of a full window among short ones: its units' CTAs walk at most 40 key tiles each, whatever the window, or
    the batch is divided into runs."""
    fit = (ctypes.c_int * 9)(0, 0, 76, 50, 36, 28, 24, 20, 16)
    f = library.window_step_cluster
    f.argtypes = [ctypes.c_longlong, ctypes.c_longlong, ctypes.c_int, ctypes.POINTER(ctypes.c_int)]
    for bs in range(1, 153):
        for tiles in (0, 1, 2, 5, 9, 17, 33, 40, 41, 49, 65, 129, 400, 10 ** 6):
            split = f(bs * hkv, tiles, 152, fit)
            assert 0 <= split <= 8 and (split < 2 or fit[split] >= bs * hkv) and split <= max(1, tiles)
            assert split == 0 or (tiles + split - 1) // split <= 40
            # (no more CTAs than SMs, each with a place in the workspace)
            assert bs * hkv * split <= 152


def test_answers_are_kept_per_device_and_failures_are_not(library):
    calls = [(0, -1), (0, 7), (0, 9), (1, 3), (0, 1), (63, 0), (63, 5), (64, 2), (64, 4), (1, -1)]
    n = len(calls)
    got = (ctypes.c_int * n)()
    asked = library.per_device(n, (ctypes.c_int * n)(*[d for d, _ in calls]), (ctypes.c_int * n)(*[a for _, a in calls]), got)
    assert list(got) == [-1, 7, 7, 3, 7, 0, 0, 2, 4, 3] and asked == 6
