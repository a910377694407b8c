// The division of a windowed chunk call's cost among its CTAs, run for run, on the host (the kernel's arithmetic).
#include "sk_window_cost.cuh"

#include <algorithm>
#include <vector>

using namespace sk;

namespace {
struct Unit {
    int tiles, start, cost;
};
int tiles_of(int L, int q, int last, int first, int window, int sink_pages)
{
    const int seen = std::max(0, L - q + std::min(last, q - 1) + 1);
    const int lo = std::max(0, std::max(0, L - q + first + 1) - window);
    const int gap = std::max(0, lo / 16 - sink_pages);
    return (seen - gap * 16 + kChunkKeys - 1) / kChunkKeys;
}
}  // namespace

// Key tiles of each of `count` runs, for a block table of `stride` pages a sequence; returns the batch's, or -1 where the runs
// do not cover each unit in order.
extern "C" int window_division(int bs, const int *lens, const int *qs, int hq, int hkv, int window, int sinks, int stride,
                               int count, int may_deal, int *tiles, int *num_units)
{
    window = rows_in_table(window, stride, 16);
    sinks = rows_in_table(sinks, stride, 16);
    const ChunkShape c = chunk_shape(hq / hkv);
    const int sink_pages = (sinks + 15) / 16;
    long long all = 0;
    for (int s = 0; s < bs; ++s)
        all += (long long)(((qs[s] + c.tpb - 1) / c.tpb * c.nsub + 1) / 2) * hkv;
    const int shift = cost_shift(all, (long long)sink_pages * 16 + window + 2 * c.tpb);
    std::vector<Unit> units;
    int total = 0, largest = 0, sum = 0;
    for (int s = 0; s < bs; ++s) {
        const UnitCosts uc = unit_costs(std::max(0, lens[s] - qs[s]), sink_pages, 16, window, c.tpb, c.slope, shift);
        const int n = ((qs[s] + c.tpb - 1) / c.tpb * c.nsub + 1) / 2;
        for (int h = 0; h < hkv; ++h)
            for (int i = 0; i < n; ++i) {
                const int first = 2 * i / c.nsub * c.tpb, last = (2 * i + 1) / c.nsub * c.tpb + c.tpb - 1;
                units.push_back({tiles_of(lens[s], qs[s], last, first, window, sink_pages), total,
                                 cost_of(i, uc, c.slope, shift)});
                if (units.back().cost < 1)
                    return -1;
                total += units.back().cost;
                sum += units.back().tiles;
                largest = std::max(largest, units.back().cost);
            }
    }
    const Division d = divide(total, (int)all, largest, count, may_deal != 0, shift);
    std::vector<int> upto(units.size(), 0);              // tiles of each unit that the runs so far have
    for (int r = 0; r < count; ++r) {
        tiles[r] = 0;
        const int dealt = d.deal ? (int)all / count * count : 0;
        for (int u = r; u < dealt; u += count)
            tiles[r] += upto[u] = units[u].tiles;
        const int left = (int)all - dealt;
        const long long lo = d.deal ? (long long)left * r : std::min<long long>(total, (long long)d.each * r);
        const long long hi = d.deal ? lo + left : std::min<long long>(total, (long long)d.each * (r + 1));
        for (int u = dealt; u < (int)all; ++u) {
            const long long start = d.deal ? (long long)(u - dealt) * count : units[u].start;
            const int cost = d.deal ? count : units[u].cost;
            if (start + cost <= lo || start >= hi)
                continue;
            const int a = cut_tile((int)(std::max(lo, start) - start), cost, units[u].tiles, d.uncut);
            const int b = cut_tile((int)(std::min<long long>(hi, start + cost) - start), cost, units[u].tiles, d.uncut);
            if (a != upto[u] || b < a)
                return -1;
            upto[u] = b;
            tiles[r] += b - a;
        }
    }
    for (size_t u = 0; u < units.size(); ++u)
        if (upto[u] != units[u].tiles)
            return -1;
    *num_units = (int)all;
    return sum;
}

// What PerDevice answers to calls on devices[i] where the query gives answers[i]; returns how often it asked.
extern "C" int per_device(int n, const int *devices, const int *answers, int *got)
{
    PerDevice kept;
    int asked = 0;
    for (int i = 0; i < n; ++i)
        got[i] = kept.get(devices[i], [&] { return ++asked, answers[i]; });
    return asked;
}

extern "C" int window_step_cluster(long long units, long long tiles, int num_sms, const int *fit)
{
    return step_cluster(units, tiles, num_sms, fit);
}
