// Planner entry used by the C ABI (pure host code).
#pragma once
#include <cstdint>

#include "split_kv_decode.h"

namespace skv {

struct PlanOut {
    int32_t chunk[DA_MAX_BATCH];
    int32_t n_splits[DA_MAX_BATCH];
    int32_t n_items;
    int32_t grid;
    int64_t est_cost;
};

// How the split kernel hands out its items, and what an item costs beside its positions.
struct PlanRule {
    int64_t overhead; // per item, in positions
    // false: sequences as they stand, item i to CTA i % grid. true: sequences in the order
    // of order_by_size, every other round of grid items from the last CTA to the first.
    bool by_size;
    int64_t combine; // what a combine costs where some sequence has several splits, in positions
};

// The sequences by the length of their items, the longest first (equal ones as they stand).
void order_by_size(const int32_t *lens, const int32_t *chunk, int batch, uint8_t *order);

// Returns 0 on success, 1 for invalid input, 2 if no split fits max_items.
int plan_splits(const int32_t *lens, int batch, int hkv, int tile, int slots, int force_splits,
                int max_items, const PlanRule &rule, PlanOut *out);

} // namespace skv
