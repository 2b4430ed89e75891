// Planner of scored attention: how the shared positions and the sequences' own spans are cut into
// items. Pure host code, no CUDA calls.
//
// The kernel is persistent, one CTA an SM; item i of a round goes to CTA i, every other round
// from the last CTA to the first, the shared items before the others and those by size (ScoredOrder). The planner
// scores candidates by that assignment, in units of a sixteenth of the time that a K and a V
// tile take from memory at one SM's share of the rate, and keeps the cheapest.
#include <algorithm>
#include <cstdint>
#include <vector>

#include "scored.h"

namespace skv {

namespace {

constexpr int64_t kUnit = 16;
constexpr int64_t kMaxItems = 1 << 22;
constexpr int64_t kSimulated = 1 << 14; // items whose assignment is followed

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

} // namespace

void scored_order(const int32_t *tiles, const int32_t *chunk, int batch, uint8_t *order)
{
    for (int b = 0; b < batch; ++b) order[b] = (uint8_t)b;
    std::stable_sort(order, order + batch, [&](uint8_t x, uint8_t y) {
        return std::min(tiles[x], chunk[x]) > std::min(tiles[y], chunk[y]);
    });
}

// a shared tile: its softmax and MMAs take 0.38 of its time from memory for each term of q and of the
// weights and 128 rows
static int64_t shared_tile_cost(int units, int terms)
{
    return std::max<int64_t>(kUnit, kUnit * units * terms * 5 / 13);
}
// of an item beside its tiles: q, the first tile's latency and the epilogue, in which copies of more
// than 16 rows are joined in several passes; and the partials that it writes and the combine reads
static int64_t item_cost(int tile, int head_dim, int rows)
{
    const int64_t fixed = (rows > 16 && rows <= 64 ? 4 : 2) * kUnit * 128 / tile;
    return fixed + (int64_t)rows * head_dim * 8 * kUnit / ((int64_t)tile * head_dim * 4);
}

int scored_lead(const ScoredWork &w, int shared, int64_t own)
{
    if (own < 1) return 1;
    int64_t tiles = 0;
    for (int b = 0; b < w.batch; ++b) tiles += (int64_t)w.tiles[b] * w.hkv * w.row_groups;
    const int64_t each = item_cost(w.tile, w.head_dim, w.own_rows) + kUnit * tiles / own;
    const int64_t all = item_cost(w.tile, w.head_dim, w.shared_rows) +
                        shared_tile_cost(w.units, w.q_terms + w.p_terms) * shared;
    return (int)std::max<int64_t>(1, std::min<int64_t>((all + each / 2) / each, 1024));
}

int plan_scored(const ScoredWork &w, ScoredSplit *out)
{
    const int64_t shared_tile = shared_tile_cost(w.units, w.q_terms + w.p_terms);

    struct Candidate {
        std::vector<int32_t> chunk;
        int32_t shared;
    };
    std::vector<Candidate> cand;
    int32_t most = w.shared_tiles;
    int64_t total = (int64_t)w.shared_tiles * w.row_tiles * w.hkv;
    for (int b = 0; b < w.batch; ++b) {
        most = std::max(most, w.tiles[b]);
        total += (int64_t)w.tiles[b] * w.hkv * w.row_groups;
    }
    // chunks of n splits of about one size, of `most` tiles at most
    auto even = [](int tiles, int64_t n, int most) {
        if (!tiles) return (int32_t)1;
        n = std::max(n, ceil_div(tiles, most));
        return (int32_t)ceil_div(tiles, std::min<int64_t>(n, tiles));
    };
    if (w.force_splits > 0) {
        Candidate c;
        for (int b = 0; b < w.batch; ++b) c.chunk.push_back(even(w.tiles[b], w.force_splits, w.own_max));
        c.shared = even(w.shared_tiles, w.force_splits, w.shared_max);
        cand.push_back(c);
    } else {
        // targets: the even share of a number of rounds, and steps of a quarter octave
        std::vector<double> targets;
        for (int r = 1; r <= 12; ++r) targets.push_back((double)total / ((double)r * w.slots));
        for (double t = std::max(1.0, (double)total / (24.0 * w.slots));; t *= 1.19) {
            targets.push_back(t);
            if (t > most) break;
        }
        for (double t : targets) {
            if (t < 0.25) continue;
            for (int round = 0; round < 2; ++round) {
                Candidate c;
                // (a) splits of at most t tiles, (b) of about t
                auto splits = [&](int tiles, double share) {
                    const double n = tiles / share;
                    return (int64_t)(round ? n + 0.5 : n + 0.999);
                };
                for (int b = 0; b < w.batch; ++b)
                    c.chunk.push_back(even(w.tiles[b], splits(w.tiles[b], t), w.own_max));
                c.shared = even(w.shared_tiles, splits(w.shared_tiles, t * kUnit / shared_tile),
                                w.shared_max);
                cand.push_back(c);
            }
        }
    }

    int64_t best = -1;
    std::vector<int64_t> load;
    std::vector<uint8_t> order((size_t)w.batch);
    for (const Candidate &c : cand) {
        const int64_t ss = w.shared_tiles ? ceil_div(w.shared_tiles, c.shared) : 0;
        int64_t items = ss * w.hkv * w.row_tiles;
        const int64_t all = items; // of the shared positions
        int64_t most_splits = 1;
        for (int b = 0; b < w.batch; ++b) {
            const int64_t n = std::max<int64_t>(1, ceil_div(w.tiles[b], c.chunk[b]));
            items += n * w.hkv * w.row_groups;
            most_splits = std::max(most_splits, n + ss);
        }
        if (items > kMaxItems) continue;
        // (candidates of very many items: the mean load instead of the largest)
        const int64_t grid = std::min<int64_t>(items, w.slots);
        const bool exact = items <= kSimulated;
        int64_t cost = 0, sum = 0, i = 0;
        load.assign((size_t)grid, 0);
        const int lead = scored_lead(w, c.shared, items - all);
        const ScoredOrder order_of = {(int32_t)grid, (int32_t)all, lead};
        auto add = [&](int64_t n, int64_t each) {
            sum += n * each;
            for (int64_t k = 0; exact && k < n; ++k, ++i) load[(size_t)order_of.cta((int32_t)i)] += each;
        };
        const int64_t per = (int64_t)w.hkv * w.row_tiles;
        for (int64_t s = 0; s < ss; ++s)
            add(per, item_cost(w.tile, w.head_dim, w.shared_rows) +
                         shared_tile * std::min<int64_t>(c.shared, w.shared_tiles - s * c.shared));
        scored_order(w.tiles, c.chunk.data(), w.batch, order.data());
        for (int b : order) {
            const int64_t n = std::max<int64_t>(1, ceil_div(w.tiles[b], c.chunk[b]));
            const int64_t each = item_cost(w.tile, w.head_dim, w.own_rows);
            // (all splits but the last are of one size)
            add((n - 1) * w.hkv * w.row_groups, each + kUnit * c.chunk[b]);
            add((int64_t)w.hkv * w.row_groups,
                each + kUnit * (w.tiles[b] - (n - 1) * c.chunk[b]));
        }
        cost = exact ? *std::max_element(load.begin(), load.end()) : sum / grid;
        if (most_splits > 1) cost += 2 * kUnit * 128 / w.tile; // the combine's launch
        if (best < 0 || cost < best) {
            best = cost;
            for (int b = 0; b < w.batch; ++b) {
                out->chunk[b] = c.chunk[b];
                out->n_splits[b] = (int32_t)std::max<int64_t>(1, ceil_div(w.tiles[b], c.chunk[b]));
            }
            out->shared_chunk = c.shared;
            out->shared_splits = (int32_t)ss;
            out->items = items;
            out->cost = cost;
        }
    }
    return best < 0 ? 1 : 0;
}

} // namespace skv
