// Scored attention (decode_attn_splitk_scored): what the host and the kernel share.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "internal.h"

namespace skv {

// positions of a tile, accumulators (two softmax warpgroups take tiles in turn; TMEM has room for an
// accumulator each at 128 columns), and 16-bit terms of a weight
__host__ __device__ constexpr int scored_tile(int D, int terms)
{
    return D == 128 && terms == 2 ? 128 : 64;
}
__host__ __device__ constexpr int scored_accs(int D) { return D == 128 ? 2 : 1; }
// 256 columns, two terms: TMEM has room for a term of Q beside O and the scores
__host__ __device__ constexpr bool scored_q_in_tmem(int D, int terms) { return D == 256 && terms == 2; }
// terms of a weight (and of an f32 q): f16 carries 11 bits a term, bf16 8
constexpr int scored_terms(int kv_dtype, int out_dtype)
{
    return kv_dtype == DA_BF16 && out_dtype == DA_F32 ? 3 : 2;
}
constexpr int kScoredMaxSlots = 8;
// barriers, exchange of (m, l), row scales (at 256 columns beside 128 rows of two terms and five tiles
// of the ring)
__host__ __device__ constexpr int scored_misc(int D) { return D == 128 ? 4096 : 2048; }
constexpr int kScoredRowBytes = 512; // of the place where copies are joined: a row's factor and place
constexpr int kScoredSmemMax = 232448;

// Shared memory: the terms of Q that TMEM does not hold, [row tile][term][64-column chunk][rpad rows
// of 128 bytes], then a ring of K and V tiles, then the place where the copies of an item's rows are
// joined, then the rest.
struct ScoredGeometry {
    int kind;
    int q_terms;   // 1: q is of the cache's type
    int tile_rows; // query rows of an item, at most (256: two row tiles that share K and V tiles)
    int rpad;      // rows of a Q chunk
    int q_bytes;
    int slots;     // of the ring
    int join_bytes;
    int smem;
};

// Kernels by what their items are, so that each has the code of its own tiles only (the softmax warps
// run straight code, and wait for instructions as long as they compute: with both forms in one
// kernel a tile of packed rows took 1.25 us, without the other 0.98): sequences' items whose few
// rows' terms lie in the lanes of a warp, other items of sequences, items of shared positions and of
// sequences.
enum : int { kScoredPacked = 0, kScoredOwn = 1, kScoredShared = 2 };
// Rows up to which items are packed.
constexpr int scored_packed(int p_terms) { return p_terms == 2 ? 16 : 8; }

// own_rows: a sequence's query rows of a KV head; shared_rows: those of the batch, or 0
inline ScoredGeometry scored_geometry(int D, int q_terms, int p_terms, int own_rows,
                                      int64_t shared_rows)
{
    ScoredGeometry g;
    const int slot = scored_tile(D, p_terms) * D * 2;
    const int64_t most = shared_rows > own_rows ? shared_rows : own_rows;
    g.q_terms = q_terms;
    g.kind = shared_rows > 0                      ? kScoredShared
             : own_rows <= scored_packed(p_terms) ? kScoredPacked
                                                  : kScoredOwn;
    const bool tm = scored_q_in_tmem(D, p_terms);
    const int held = (g.kind == kScoredPacked ? 1 : q_terms) - (tm ? 1 : 0); // in shared memory
    // (two row tiles only for a q of one term: with more terms the ring would be too short)
    for (g.tile_rows = scored_accs(D) == 2 && q_terms == 1 ? 256 : 128;; g.tile_rows /= 2) {
        const int rows = (int)(most < g.tile_rows ? most : g.tile_rows);
        // 128 lanes, with copies of few rows, where that leaves a ring of two tiles; a ring
        // shorter than a tile and a half takes smaller items
        for (g.rpad = 128;; g.rpad /= 2) {
            g.q_bytes = (rows > 128 ? 2 : 1) * held * g.rpad * D * 2;
            // copies of up to 64 rows are joined at least 16 columns at a time
            auto narrow = [&](int64_t all) { // has an item of up to 64 rows
                const int64_t rest = all % g.tile_rows;
                return all > 0 && (all <= 64 || g.tile_rows == 64 || (rest > 0 && rest <= 64));
            };
            g.join_bytes = narrow(own_rows) || narrow(shared_rows) ? kScoredRowBytes + g.rpad * 128 : 0;
            g.slots = (kScoredSmemMax - 1024 - scored_misc(D) - g.q_bytes - g.join_bytes) / slot;
            if (g.slots >= 4 || g.rpad / 2 < rows || g.rpad == 32) break;
        }
        if (g.slots >= 3 || g.tile_rows == 64) break;
    }
    if (g.slots > kScoredMaxSlots) g.slots = kScoredMaxSlots;
    // the 128-row MMA reads 128 rows from every Q chunk: past the last one, into the ring
    g.smem = 1024 + g.q_bytes + g.slots * slot + g.join_bytes + scored_misc(D);
    return g;
}

// Tiles of an item at most. An MMA's sums are cut off at their 24th bit, so that a lane's accumulator
// loses up to 2^-24 of itself at every addition of a term of 16 positions (measured, 1024
// additions: 6e-5 of values of one sign, 2e-5 of N(0, 1) ones). f32 outputs start a partial after at
// most 48 additions, which the combine adds in f32; f16 ones after 1024 and bf16 ones after 8192, a
// quarter of the output's half step. (131072 positions of 96 rows and 256 columns in one item, 16384
// additions: 9e-4 off, more than three half steps of f16. 152 sequences of 32768 such positions take
// 712 us as one item each, 4096 additions, and 846 as four.)
inline int scored_max_tiles(const ScoredGeometry &g, int D, int p_terms, int rows, int out_dtype)
{
    const int T = scored_tile(D, p_terms);
    const int span = rows > 64 ? 128 : rows > 32 ? 64 : 32;
    const int reps = rows > 128 || g.rpad < span ? 1 : g.rpad / span;
    // additions of a unit to a lane (packed: a term has a lane of its own; or copies of its own, and
    // then half as many share the columns)
    const int per = T / 16 / reps * (g.kind == kScoredPacked ? 1 : p_terms);
    const int most = out_dtype == DA_F32 ? 48 : out_dtype == DA_F16 ? 1024 : 8192;
    const int units = most / (per > 1 ? per : 1);
    return rows > 128 || scored_accs(D) == 1 ? units : 2 * units;
}

struct ScoredParams {
    const void *q;
    void *out;               // written by the kernel itself if whole
    float2 *ml;              // workspace (m, l) per (slot, row)
    float *acc;              // workspace acc per (slot, row, D)
    int *status;
    const float *slopes;     // per query head, or NULL
    const int32_t *starts, *keep_lens;
    const int32_t *dev_lens;
    const int32_t *block_table, *shared_table;
    uint64_t timeout_ns;
    float scale, softcap;
    int32_t batch, rows, q_len, hq, hkv; // rows: q_len * hq
    int32_t group, per_seq;              // query heads of a KV head; rows of a sequence: times q_len
    uint32_t inv_group, inv_seq;         // scored_inverse of these
    int32_t q_f32, q_terms, out_dtype, whole, flags;
    int32_t window, keep;
    int32_t max_blocks, block_size, oob_block, box_rows;
    int32_t rpad, tile_rows, slots, q_bytes, join_bytes;
    int32_t kind;
    int32_t row_groups;      // of a sequence's rows of one KV head
    // items of the shared positions: (split, KV head, row tile), the row tile fastest
    int32_t shared_len, shared_tiles, shared_chunk, shared_splits, row_tiles, shared_items;
    // then those of the sequences: entry e is sequence seq[e], (split, KV head, row group)
    int32_t n_items;
    int32_t lead;            // items of CTAs without a shared one beside the last shared items
    int32_t lens[DA_MAX_BATCH];      // of sequence b
    int32_t chunk[DA_MAX_BATCH];     // tiles of a split of sequence b
    int32_t slot[DA_MAX_BATCH];      // sequence b's first partial: the shared splits', then its own
    int32_t base[DA_MAX_BATCH + 1];  // splits before entry e
    uint8_t seq[DA_MAX_BATCH];
};

// x / d for x < 2^15 and d up to 128 is the upper word of x times ceil(2^32 / d): too much by x / 2^32 at
// most, less than 1 / d. (d = 1: x itself)
inline uint32_t scored_inverse(int d) { return (uint32_t)(((1ull << 32) + d - 1) / (uint64_t)d); }

// Which CTA works on which item: rounds from the first CTA to the last and back. Where the shared items
// end inside a round, the CTAs without one work on `lead` items of sequences meanwhile.
struct ScoredOrder {
    int32_t grid, all, lead; // CTAs, shared items
    // CTA c's r-th item, if there are so many
    __host__ __device__ int64_t item(int c, int r) const
    {
        const int full = all / grid, rest = all - full * grid;
        if (r < full) return (int64_t)r * grid + (r & 1 ? grid - 1 - c : c);
        if (rest == 0) {
            const int64_t first = (int64_t)r * grid;
            return first + (r & 1 ? grid - 1 - c : c);
        }
        const int pos = full & 1 ? grid - 1 - c : c, free = grid - rest;
        int later = r - full - 1;
        if (pos < rest) {
            if (later < 0) return (int64_t)full * grid + pos;
        } else {
            const int e = r - full, j = pos - rest;
            if (e < lead) return (int64_t)all + (int64_t)e * free + (e & 1 ? free - 1 - j : j);
            later = e - lead;
        }
        const int64_t first = (int64_t)all + (int64_t)lead * free + (int64_t)later * grid;
        return first + ((full + 1 + later) & 1 ? grid - 1 - c : c);
    }
    // the CTA of item i
    __host__ __device__ int cta(int64_t i) const
    {
        const int full = all / grid, rest = all - full * grid, free = grid - rest;
        if (rest == 0 || i < all) {
            const int64_t r = i / grid;
            const int at = (int)(i - r * grid);
            return r & 1 ? grid - 1 - at : at;
        }
        int64_t e = i - all;
        if (e < (int64_t)lead * free) {
            const int64_t r = e / free;
            const int j = (int)(e - r * free), pos = rest + (r & 1 ? free - 1 - j : j);
            return full & 1 ? grid - 1 - pos : pos;
        }
        e -= (int64_t)lead * free;
        const int64_t r = e / grid;
        const int at = (int)(e - r * grid);
        return (full + 1 + r) & 1 ? grid - 1 - at : at;
    }
};

// by the cache's type and the output's (f32 outputs of bf16 caches take three terms)
#define SKV_SCORED_LAUNCH(name) \
    cudaError_t name(int grid, int smem, cudaStream_t st, const CUtensorMap &km, const CUtensorMap &vm, \
                     const ScoredParams &p)
SKV_SCORED_LAUNCH(launch_gqa_scored_f16_128);
SKV_SCORED_LAUNCH(launch_gqa_scored_f16_256);
SKV_SCORED_LAUNCH(launch_gqa_scored_bf16_128);
SKV_SCORED_LAUNCH(launch_gqa_scored_bf16_256);
SKV_SCORED_LAUNCH(launch_gqa_scored_bf16_f32_128);
SKV_SCORED_LAUNCH(launch_gqa_scored_bf16_f32_256);
// Planner (plan_scored.cpp, pure host code). Lengths in tiles.
struct ScoredWork {
    int batch, hkv, row_groups;
    const int32_t *tiles;   // of each sequence's visible span
    int shared_tiles, row_tiles;
    int units;              // row tiles of 128 rows in an item of the shared positions
    int shared_rows;        // its rows
    int own_rows;
    int tile, q_terms, p_terms, head_dim;
    int shared_max, own_max; // tiles of an item at most
    int slots;              // CTAs
    int force_splits;
};
struct ScoredSplit {
    int32_t chunk[DA_MAX_BATCH], n_splits[DA_MAX_BATCH]; // of the sequences' own tiles
    int32_t shared_chunk, shared_splits;
    int64_t items, cost;
};
// Returns 0 on success, 1 if no split has an acceptable number of items.
int plan_scored(const ScoredWork &w, ScoredSplit *out);
// Items of sequences that a CTA without one of the last, partial round of shared items works on
// meanwhile: by their costs, `own` items of sequences beside shared ones of `shared` tiles
int scored_lead(const ScoredWork &w, int shared, int64_t own);
// the sequences by their items' tiles, the longest first
void scored_order(const int32_t *tiles, const int32_t *chunk, int batch, uint8_t *order);

} // namespace skv
