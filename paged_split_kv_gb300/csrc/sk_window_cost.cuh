// Windowed attention: how a call's work is shared among the CTAs.  Chunks: what a unit of work costs, and where the batch's
// cost is cut into the CTAs' runs; steps: clusters or runs.  Plain arithmetic, for the host as well.
#pragma once
#include <stdint.h>

#include <atomic>

#ifdef __CUDACC__
#define SK_COST_FN __device__ __forceinline__
#define SK_COST_DIV(a, b) __fdividef(a, b)
#else
#define SK_COST_FN inline
#define SK_COST_DIV(a, b) ((a) / (b))
#endif

namespace sk {

constexpr int kChunkKeys = 128;                      // keys of a tile
constexpr int kChunkRows = 128;                      // rows of a row tile
// Cost of starting and finishing a unit, in keys, next to other units, which hide part of it, and of its last key tile, which
// is filled in part; and what a unit of a full window costs more, whose first tile is masked too.  Geometric means over 94
// calls (one to 24 prompts and chunks, groups of 4 to 160 heads, windows of 128 to 4096 and of all; bf16 and e4m3 pages), us:
//   128 and 0    112.3      160 and 32   110.2      192 and 64   108.9      224 and 0    108.6      224 and 64   108.4
//   256 and 64   108.4      224 and 128  108.9      224 and 192  109.8      224 and 320  112.5      160 and 96   111.1
// Single long prompts gain, whose first CTAs have nothing but small units: with 128 and 0, and with 224 and 64, 8000 tokens
// of 16/2 heads over 4096 take 158 and 151, 4000 of 48/2 heads 203 and 174.  Batches differ by where their cuts fall: eight
// prompts of up to 4000 over 4096 177 and 176, six of 24 prompts over 512 98 to 120, and 100 to 120, ten of up to 3000 over
// 1024 167 to 217, and 165 to 216.
constexpr int kChunkFixed = 224;
constexpr int kChunkEdge = 64;
// A cut costs a piece's start and end, and the join of the unit: it moves to the unit's start or end where that is no further
// than this (106 calls, the geometric mean: 98.7 us with 256, 98.6 with 384, 98.6 with 512, 99.2 with 640, 99.9 with 768).
constexpr int kCutFixed = 512;
// Where units cost alike, none is cut if the longest run is then longer by this or less than if they were: 122 units over a
// window of 2048 take 39.4 us, and 44.4 cut (e4m3 pages 41.3 and 46.2), 100 over 1024 26.5 and 29.6; 168 over 1024 on the 152
// SMs take 38.4 cut, and 42.6 whole.  The mean of the 106 calls: 99.4 us with 0, 99.3 with 400, 98.6 with 800, 99.1 with 1600.
constexpr int kJoinCost = 800;

// A row tile is `tpb` query tokens times `gb` heads of the group, or one of the `nsub` tiles of a token whose group has more
// than 128 heads; a unit is two row tiles.  `slope`: what a unit sees more than the one before, in 2^-kSlopeBits keys (a
// unit of 2 tpb tokens, or of 2 / nsub of one).
constexpr int kSlopeBits = 8;
struct ChunkShape {
    int gb, nsub, tpb;
    uint32_t slope;
};
inline ChunkShape chunk_shape(int G)
{
    ChunkShape c;
    c.gb = G < kChunkRows ? G : kChunkRows;
    c.nsub = (G + c.gb - 1) / c.gb;
    c.tpb = kChunkRows / c.gb;
    c.slope = (uint32_t)((2 * c.tpb << kSlopeBits) / c.nsub);
    return c;
}

// A window or sinks of more rows than the block table has are all of a sequence.  (The steps that costs are counted in go by
// the window: with one of 2^30 rows they were so coarse that a unit's price said little of its keys: 8000 tokens of 16/2 heads
// over a window of all took 194 us, 184 so, 2000 of 71/1 heads 152 and 123.)
inline int rows_in_table(int rows, int stride, int page)
{
    return rows / page < stride ? rows : stride * page;
}

// Costs are counted in 2^shift keys, so that those of `units` units of `most` keys or less come to less than 2^30.
inline int cost_shift(long long units, long long most)
{
    int shift = 4;
    while ((units * (kChunkFixed + kChunkEdge + most) >> shift) >> 30)
        ++shift;
    return shift;
}

// The units of one (sequence, KV head): unit i costs what its last tokens see, base + slope (i + 1), below `rising`, then
// `top`, a full window and its edge.  Sums keep the slope's fraction of 2^shift keys: with a slope of whole steps, 8 tokens a
// unit and shift 4, all units cost alike, the longest run of 4000 tokens of 32/1 heads over a window of 4096 had 125 key tiles
// where the average is 53, and the call took 214 us; it takes 114 so (48/2 heads: 319 and 174; 5000 tokens of 24/2 heads: 145
// and 136).
struct UnitCosts {
    int base, top, rising;
};
SK_COST_FN UnitCosts unit_costs(int cached, int sink_pages, int page, int window, int tpb, uint32_t slope, int shift)
{
    UnitCosts c;
    c.base = ((kChunkFixed + cached) >> shift) + 1;
    c.top = (int)((kChunkFixed + (long long)sink_pages * page + window + 2 * tpb) >> shift) + 1;
    const float rise = (float)(c.top - c.base) * (float)(1 << kSlopeBits) * (float)(1 << shift);
    const float steps = slope == 0 ? 2e9f : SK_COST_DIV(rise, (float)slope);
    c.rising = c.base >= c.top ? 0 : (int)(steps < 2e9f ? steps : 2e9f);
    c.top += kChunkEdge >> shift;
    return c;
}
// Cost of the units before unit i.  (slope n / 2^kSlopeBits is below 2^32 for n up to `rising`, and n below 2^24.)
SK_COST_FN int cost_before(int i, UnitCosts c, uint32_t slope, int shift)
{
    const int n = i < c.rising ? i : c.rising;
    const uint64_t rise = (uint64_t)(uint32_t)n * (uint32_t)(n + 1) * slope >> (kSlopeBits + 1 + shift);
    return n * c.base + (int)rise + (i - n) * c.top;
}
// Cost of unit i.
SK_COST_FN int cost_of(int i, UnitCosts c, uint32_t slope, int shift)
{
    return cost_before(i + 1, c, slope, shift) - cost_before(i, c, slope, shift);
}

// How `count` runs share `all` units that cost `total`, the dearest of them `largest`: with `may_deal`, whole units in turn
// where they cost alike or little beside a share; else equal shares of the cost, cut within units or, `uncut`, between them.
struct Division {
    bool deal, uncut;
    int each;
};
SK_COST_FN Division divide(int total, int all, int largest, int count, bool may_deal, int shift)
{
    Division d;
    d.deal = may_deal && ((float)largest * (float)all <= 1.4f * (float)total ||
                          (float)largest * (float)count * 8.f <= (float)total);
    d.each = total / count + 1;
    const int most = (all + count - 1) / count;      // units of a run, if none is cut
    d.uncut = !d.deal && (float)largest * (float)all <= 1.1f * (float)total &&
              (float)largest * (float)(most * count - all) <= (float)(kJoinCost >> shift) * (float)count;
    return d;
}
// Key tile at which a run's bound cuts a unit of t tiles, `at` of `cost` in.
SK_COST_FN int cut_tile(int at, int cost, int t, bool uncut)
{
    const float f = SK_COST_DIV((float)at, (float)cost);
    const float g = uncut ? 0.5f : SK_COST_DIV((float)kCutFixed, (float)(kCutFixed + t * kChunkKeys));
    const int tile = (int)((float)t * f);
    return at >= cost ? t : f <= g ? 0 : f >= 1.f - g ? t : tile < t ? tile : t;
}

// ------------------------------------------------------------------ steps
constexpr int kMaxSplit = 8;                         // CTAs of a cluster
// What the join kernel costs, in key tiles of a CTA: 96 units of 9 tiles take 11.9 us as clusters (of one) and 15.2 as runs, of
// 17 tiles 20.1 and 21.2.
constexpr int kJoinTiles = 7;
// Key tiles of a cluster's CTA up to which clusters are taken.  `tiles` is a bound on the units: where sequences are shorter,
// runs share what there is, while a cluster still walks its own unit, so that what clusters can lose grows with their tiles,
// and what they gain, the join and the cuts, does not.  Clusters and runs of 19 sequences of 32/8 heads (clusters of one), us:
//   window (tiles)    all full       0.1 to 1 of it    one full, 18 of 300
//   4096 (33)         50.9, 53.4     37.1, 36.8        31.7, 16.8     (e4m3 pages 34.3, 36.8;  34.1, 29.3;  33.7, 17.8)
//   6144 (49)         72.8, 75.0     52.2, 49.1        43.2, 18.3     (47.6, 50.0;  47.3, 37.3;  47.0, 20.9)
//   16384 (129)       180, 182       127, 109          99.9, 25.6     (114, 116;  113, 73.7;  114, 27.9)
// and of 9 sequences (clusters of two) over 12288: 70.2, 75.1; 51.5, 46.4; 43.3, 20.3 (48.9, 50.9; 48.4, 34.5; 48.1, 22.2).
constexpr int kClusterTiles = 40;

// Runs of a step's call: one per SM, and no more than there are key tiles.
inline long long step_runs(long long units, long long tiles, int num_sms)
{
    const long long most = units * (tiles < 1 ? 1 : tiles);
    return most < num_sms ? most : num_sms;
}
// CTAs of each unit's cluster; 0: the batch is divided into equal runs.  Units that fit at once have a cluster each, as large
// as fits (fit[c] clusters of c CTAs run at the same time) and as they have tiles, where units of `tiles` key tiles take no
// longer than equal runs and their join, and shorter ones not much longer.
inline int step_cluster(long long units, long long tiles, int num_sms, const int *fit)
{
    const long long runs = step_runs(units, tiles, num_sms);
    if (units > runs)
        return 0;
    int split = 1;
    for (int c = 2; c <= kMaxSplit && c <= tiles; ++c)
        if (fit[c] >= units)
            split = c;
    const long long own = (tiles + split - 1) / split;
    return own > units * tiles / runs + kJoinTiles || own > kClusterTiles ? 0 : split;
}

// Answers of a query about a device, asked once for each: ask() gives one of at least 0, or a negative value where it fails.
// A failure is not kept: the next call asks again.
struct PerDevice {
    static constexpr int kDevices = 64;
    std::atomic<int> kept[kDevices] = {};            // the answer and 1
    template <typename Ask>
    int get(int device, Ask ask)
    {
        if (device < 0 || device >= kDevices)
            return ask();
        int x = kept[device].load() - 1;
        if (x < 0) {
            x = ask();
            if (x >= 0)
                kept[device].store(x + 1);
        }
        return x;
    }
};

}  // namespace sk
