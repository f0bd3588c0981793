// row_plan.h -- how the launches over row tiles (row_tiles.h) split their work:
// host code, apart from the kernels so that it can be built and checked alone.
// Internal to the library.
#pragma once

#include "qmm_internal.h"

namespace qmm {

constexpr int kImageBytes = 192;       // activation parts of one token and 32-block
constexpr int kScaleLds = 16 * 80;     // a wave's LDS for the scales of its rows
constexpr int kLdsMost = 160 * 1024;   // of one workgroup

struct RowPlan {
    int half;        // tiles of eight rows (HALF)
    int s_log2;      // log2 of the waves that share a tile
    int waves;       // per workgroup
    int steps;       // units (HALF: pairs of units) per row
    int step_bytes;  // image bytes per step and token
    int image;       // LDS bytes for the image
};

// units: 64-byte units per row, mf: blocks per unit; tiles: tiles of the
// launch; half_tiles: their number with eight rows each (0: not available);
// tokens: the most tokens one image holds at once; likely: how many it will hold
// as a rule.
//
// The memory streams at its rate with about sixteen waves on every CU and four
// or more units of each in flight, so waves share tiles until there are that
// many (tile, wave) tasks or four units left to a wave (three Q8_0 tokens
// choosing four of sixteen experts of 1408 x 2048: 25.2 us with four waves a
// tile, 27.0 with two, 29.4 with one).  With two token groups a unit is twice
// the work and two units will do (5632 x 2048 for eight tokens: 6.0 us with
// eight waves a tile, 6.8 with four), and so they will with several tokens and
// no more tiles than CUs (256 tiles of 5632 for two tokens: 5.7 us with
// sixteen waves a tile, 7.2 with eight).  Where a launch has so few tiles that most
// of the chip idles even so, tiles of eight rows and pairs of units double
// them (2048 x 5632 for one token: 4.4 us against 4.9; 5632 x 2048, whose 352
// tiles are enough, 5.0 against 4.4).  Workgroups are small (four waves) while
// their image is, so that several share a CU and one's loads run beside
// another's setup; with more tokens a larger workgroup shares one image, and so
// it does where a larger one's image then holds all of K (11008 x 4096 for four
// tokens: 9.4 us with sixteen waves, 13.4 with eight and two passes).
constexpr int kImageMost = 112 * 1024;
inline RowPlan plan_rows(int64_t units, int mf, int64_t tiles, int64_t half_tiles, int tokens, int likely)
{
    const int64_t cus = device_cus();
    RowPlan p = {0, 0, 4, 0, 0, 0};
    auto steps_of = [&](int half) { return (units + half) / (1 + half); };
    auto share = [&](int64_t t, int64_t steps, int least) {
        int s = 0;
        while (s < 4 && t << s < 16 * cus && steps >> (s + 1) >= least) ++s;
        return s;
    };
    p.s_log2 = share(tiles, steps_of(0), tokens > 4 || (tokens > 1 && tiles <= cus) ? 2 : 4);
    if (half_tiles && tokens <= 4 && tiles << p.s_log2 < 5 * cus) {
        p.half = 1;
        p.s_log2 = share(half_tiles, steps_of(1), 2);
    }
    p.waves = likely <= 2 ? 4 : likely <= 4 ? 8 : 16;
    if (p.waves < 1 << p.s_log2) p.waves = 1 << p.s_log2;
    auto budget = [&] { return p.waves <= 4 ? 32 * 1024 : p.waves <= 8 ? 64 * 1024 : kImageMost; };
    const int64_t whole = (int64_t)steps_of(p.half) * (1 + p.half) * mf * kImageBytes * tokens;
    if (likely == tokens && whole > budget() && whole <= kImageMost)
        while (whole > budget()) p.waves *= 2;
    // one step of every wave of a tile has to fit the image
    for (;;) {
        p.step_bytes = (1 + p.half) * mf * kImageBytes;
        if (((int64_t)p.step_bytes * tokens << p.s_log2) <= budget()) break;
        if (p.waves < 16) p.waves *= 2;
        else --p.s_log2;
    }
    p.steps = (int)steps_of(p.half);
    const int64_t all = (int64_t)p.steps * p.step_bytes * tokens;
    p.image = (int)(all < budget() ? all : budget());
    return p;
}
// Steps per pass over K of an image for `tokens` tokens: all of them, or a
// multiple of the waves per tile.
__host__ __device__ inline int pass_steps(int image, int step_bytes, int tokens, int s_log2, int steps)
{
    const int n = image / (step_bytes * tokens);
    return n < steps ? n >> s_log2 << s_log2 : steps > 0 ? steps : 1;
}


// A launch of gemv_mx_kernel.
struct MxPlan {
    RowPlan rows;
    int parts;       // workgroups among which each item's tokens are divided
    int64_t N;       // tokens of one of them (the last may have fewer)
    int tile_rows;   // weight rows per tile
    int T;           // tiles per workgroup
    int tg;          // token groups
    int pass;        // steps per pass over K
    int depth;       // units of a wave in flight
    int lds;         // bytes
    int64_t groups;  // tile groups of all items
    int64_t cap;     // workgroups the chip holds at once
};

// The depths gemv_mx_kernel and moe_up_kernel are built for, by the units of one
// wave and pass over K (with one or two there is nothing to load ahead).
inline int mx_depth(int units, bool half) { return units <= 1 ? 1 : units == 2 ? 2 : units > 4 && !half ? 8 : 4; }
inline int moe_depth(int units) { return units > 4 ? 8 : units > 2 ? 4 : 2; }

// count items of M[i] rows (not all zero) with K weights, N >= 1 tokens; pair: one
// gate / up pair of M[0] rows each.
inline MxPlan plan_mx(const int64_t *M, int count, int64_t K, int64_t N, bool pair)
{
    int64_t full = 0, half = 0;
    for (int i = 0; i < count; ++i) {
        full += (M[i] + 15) / 16;
        half += (M[i] + 7) / 8;
    }
    MxPlan m = {};
    // With tiles for no more than half the CUs, every workgroup's reading and
    // splitting of all the activations is what takes the time, and half the
    // tokens each in twice the workgroups is faster although the weights are
    // read twice, once from the caches (us, whole and halved: 2047 x 5632, eight
    // tokens 11.0, 7.9; 2048 x 2048, eight 5.8, 4.3; 2048 x 5632, four 8.1, 5.7,
    // two 5.9, 5.1; but 32000 x 2048, eight 11.3, 13.8).
    // The same where the image of half the tokens holds all of K and that of all
    // of them does not, since every tile group would build it again for each
    // pass (11008 x 4096, eight tokens 18.9, 11.3; 32000 x 4096 25.7, 20.2).
    const int64_t token = (K + 127) / 128 * 4 * kImageBytes;
    const bool few = 2 * (pair ? half : full) <= device_cus(), fits = N * token > kImageMost && (N + 1) / 2 * token <= kImageMost;
    const bool halve = N > 1 && (few || fits) && 2 * count <= QMM_GEMV_BATCH_MAX;
    m.parts = halve ? 2 : 1;
    m.N = (N + m.parts - 1) / m.parts;
    full *= m.parts;
    half *= m.parts;
    RowPlan &p = m.rows;
    p = plan_rows((K + 127) / 128, 4, pair ? half : full, pair ? 0 : half, (int)m.N, (int)m.N);
    // One more split of the tiles where the workgroups' last round is mostly
    // empty otherwise (11008 x 4096 for eight tokens in two halves: 344 groups of
    // four tiles on 256 CUs 13.9 us, 688 of two 11.3).
    auto busy = [&](int s_log2) {
        const int64_t held = 16 / p.waves * (int64_t)device_cus(), tiles = p.half ? half : pair ? half : full;
        const int64_t groups = (tiles * (1 << s_log2) + p.waves - 1) / p.waves;
        return (double)groups / (double)((groups + held - 1) / held * held);
    };
    const bool one_pass = p.image >= (int64_t)p.steps * p.step_bytes * m.N;
    if (one_pass && 2 << p.s_log2 <= p.waves && p.steps >> (p.s_log2 + 1) >= 4 && busy(p.s_log2 + 1) > 1.2 * busy(p.s_log2))
        ++p.s_log2;
    m.tile_rows = pair || p.half ? 8 : 16;
    m.T = p.waves >> p.s_log2;
    m.tg = m.N > 4 ? 2 : 1;
    m.pass = pass_steps(p.image, p.step_bytes, (int)m.N, p.s_log2, p.steps);
    m.depth = mx_depth((m.pass + (1 << p.s_log2) - 1) >> p.s_log2, p.half);
    m.lds = p.waves * (2 * m.tg * 64 * 4 + kScaleLds) + p.image;
    // as many workgroups as the CUs hold at once stream the tiles between them
    m.cap = (int64_t)(16 / p.waves) * device_cus();
    for (int i = 0; i < count; ++i) m.groups += m.parts * (((M[i] + m.tile_rows - 1) / m.tile_rows + m.T - 1) / m.T);
    return m;
}

// A launch of moe_up_kernel: N tokens that choose k of E experts of F rows.
inline RowPlan plan_moe(int64_t E, int64_t k, int64_t N, int64_t F, int64_t units, int mf)
{
    // About how many entries the tokens make: a token chooses k of E experts, so
    // an expert has c pairs of N trials with chance k / E each, and ceil(c / 2)
    // entries: the mean of c plus the chance that it is odd, halved.
    const double chance = k < E ? (double)k / (double)E : 1.0;
    double even = 1.0;
    for (int64_t n = 0; n < N; ++n) even *= 1.0 - 2.0 * chance;
    const double mean = (double)E * ((double)N * chance + (1.0 - even) / 2.0) / 2.0;
    const int64_t entries = mean < 1.0 ? 1 : (int64_t)(mean + 0.5);
    return plan_rows(units, mf, (F + 7) / 8 * entries, 0, (int)(N * k < 2 ? 1 : 2), 1);
}
inline int moe_lds(const RowPlan &p) { return p.waves * (64 * 4 + kScaleLds) + p.image; }

}  // namespace qmm
