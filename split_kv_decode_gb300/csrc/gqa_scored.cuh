// Scored attention on tcgen05 tensor cores, sm_103a: split-KV decode attention whose scores
// are capped, biased by the distance and masked, over 16-bit caches, and over positions that
// all sequences share.
//
//     y = c tanh(x / c), x = scale q.k  (or x without a cap)
//     y -= slope_h |position of the token - j|
//     out = sum_j 2^(y_j log2 e - m) v_j / sum_j 2^(y_j log2 e - m)   over the visible j
//
// An item is a slice of positions for up to 128 query rows of one KV head (256 where two row
// tiles share the slice's tiles): the (token, head) rows of one sequence, or, for shared
// positions, those of the whole batch, so that shared keys and values are read and multiplied
// once. Per tile of T positions
//     S = Q K^T       M = 128 rows, N = T, K = D          Q and K from shared memory
//     O += P V        M = 128 rows, N = D, K = T          P from TMEM, V from shared memory
// Row r is TMEM lane r of both, so its thread has its scores, its running maximum, its sum
// and its rescaling to itself; no score crosses a lane.
//
// Operands are 16-bit, sums f32. K and V are used as they stand. A weight is the sum of two 16-bit
// terms (three for f32 outputs of bf16 caches), so are the elements of an f32 q; the terms are
// MMAs into one accumulator. P takes the place of its scores in TMEM: 16 scores (16 columns) become
// two terms of 8 columns.
//
// Few rows leave most of the 128 lanes free. Up to 64 rows have copies at lanes 32 or 64 apart (Q
// rows stored several times), whose warps each take a share of a tile's columns; their other weights
// are zero. Half of the copies take the second term of the weights, so that O += P V is one set of
// MMAs. Without shared positions up to 16 rows (8 with three terms) are packed instead: the terms of q and of the
// weights lie in different lanes of a warp, a score is the sum over those lanes, and four threads
// share a row. The epilogue adds the copies' results, of up to 16 rows as fragments of 16 rows, two
// columns of every eight a thread.
//
// 256 columns, two terms: one term of Q lies in TMEM (128 columns), beside O (256) and two S slots of 64: the
// MMAs of S then read half as much shared memory, and the ring has room for four tiles or more.
//
// What bounds it: memory, where the rows are one sequence's. A tile of K and V (64 KB) takes 1.43 us
// at an SM's share of the rate; its MMAs take 0.6 to 1.1 and the softmax of a warpgroup 1.0 to 1.7,
// with two warpgroups taking tiles (or, for 256 rows, row tiles) in turn. 151552 positions of 16/4 heads
// of 256, capped, f32 q and output: 107 us, 5.8 TB/s. 32 sequences with a window of 4096, 32/8 heads
// of 128: 101 us, 5.4 TB/s (256 equal items on 152 SMs). Four tokens under a bias, 24/4 heads of 256: 152
// us, 6.0 TB/s. Many rows on shared positions are bound by the way of a unit of 128 rows through
// softmax (1.7 us for 128 positions of 128 columns, 2.3 for 64 capped ones of 256) and MMAs (0.9 and
// 1.2), of which two units overlap; the softmax warps issue an instruction every five cycles, waiting
// for instructions and for their last results (two warps a scheduler). Measured and not kept, in the
// figures of the time: the next columns on their way from TMEM meanwhile (70 -> 80 us for one
// document), 64 columns in registers between the two passes (224 -> 286 for drafts), halves of 16
// columns in a loop (241), caps between the passes (209 -> 214), one kernel for packed and other items
// (71 -> 76), a launch of its own for the shared positions (71 -> 82), tiles of 64 with four slots of
// scores and a warp for each product (70 -> 71: the softmax of half a tile takes more than half as
// long), and one warpgroup at 256 columns (252 -> 262).
//
// Roles: two softmax warpgroups, a warp for the copies of K, one for those of V, a warp of which one
// elected lane issues the MMAs. The K warp also works the items out and passes them on through a queue.
// Unit u of an item is tile u, or tile u / 2 and row tile u % 2; it has S slot and warpgroup u % 2. At
// 128 columns a warpgroup has an accumulator of its own, and a row as many states, which the
// epilogue joins. At 256 there is one: a row's reference is handed from unit to unit through
// shared memory, so that a unit waits for the last one's maximum but not for its weights, and
// whichever warpgroup raises a reference rescales O. The MMA order S0 S1 O0 S2 O1 S3 ... lets each
// unit's softmax run beside the other's MMAs, and makes P of unit u - 2 read before S of unit u takes
// its place. Every wait is bounded: one that runs out sets the status word, and all roles leave.
#pragma once
#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "merge.cuh"
#include "ptx.cuh"
#include "scored.h"

namespace skv {
namespace {

enum : int { kNone = 0, kCap = 1, kBias = 2, kAny = 3 };

template <typename DT_, int D_, int TP_, int XF_, int KIND_> struct Cfg {
    using DT = DT_;
    static constexpr int D = D_, TP = TP_;
    // scores are transformed before the maximum is taken: capped, biased, or as the call says (also:
    // scale <= 0)
    static constexpr bool XF = XF_ != kNone, CAP = XF_ == kCap, BIAS = XF_ == kBias, ANY = XF_ == kAny;
    static constexpr bool PK = KIND_ == kScoredPacked;
    static constexpr bool SH = KIND_ == kScoredShared;
    // lanes of a row's terms in a warp: 2 for up to 16 rows of two terms, 4 for up to 8 of three
    static constexpr int PARTS = !PK ? 1 : TP == 2 ? 2 : 4;
    static constexpr bool BF = std::is_same<DT, __nv_bfloat16>::value;
    static constexpr int T = scored_tile(D, TP);
    static constexpr int NWG = 2;           // softmax warpgroups
    static constexpr int NACC = scored_accs(D);
    static constexpr int NCH = D / 64;      // 64-column chunks of a row
    static constexpr int CHUNK = T * 128;   // bytes of a chunk of a tile
    static constexpr int SLOT = NCH * CHUNK;
    // softmax warps, then those of the K copies, the V copies and the MMAs, and one without work
    static constexpr int WARPS = NWG * 4, K_WARP = WARPS, V_WARP = WARPS + 1, MMA_WARP = WARPS + 2;
    static constexpr int THREADS = (WARPS + 4) * 32;
    // registers (168 a thread at launch, of which the last four warps leave some to the others:
    // 8 * 184 + 4 * 136 = 12 * 168)
    static constexpr int SOFTMAX_REGS = 184, OTHER_REGS = 136;
    // TMEM columns: accumulator w at D w, S slot s at S_COL + S_SLOT s, a term of Q at Q_COL
    static constexpr bool QTM = scored_q_in_tmem(D, TP);
    static constexpr int S_COL = 256, S_SLOT = QTM ? 64 : 128, Q_COL = 384;
    // A row's reference moves when a weight passes 2^LIM, and then to 2^-OFF of the largest: an f16
    // term keeps weights down to 2^-(24 + OFF) of it, bf16 has the exponents of f32.
    static constexpr float LIM = BF ? 8.f : 15.f, OFF = BF ? 0.f : 7.f;
};

// barriers
constexpr int SB_FULL = 0, SB_EMPTY = kScoredMaxSlots, SB_SFULL = 2 * kScoredMaxSlots,
              SB_PFULL = SB_SFULL + 2, SB_PVDONE = SB_PFULL + 2, SB_OREADY = SB_PVDONE + 2,
              SB_OFREE = SB_OREADY + 1, SB_QFULL = SB_OFREE + 1, SB_QFREE = SB_QFULL + 1,
              SB_XCH = SB_QFREE + 1, SB_GROUP = SB_XCH + 1, SB_DRAIN = SB_GROUP + 2,
              SB_ITEM = SB_DRAIN + 1, SB_TAKEN = SB_ITEM + 2, SB_REF = SB_TAKEN + 2,
              SB_N = SB_REF + 2;

struct Item {
    int tiles;              // of the visible span; < 0: no more items
    int b;                  // sequence, or -1: shared positions
    int kvh, split;
    int row0, rows;         // of the (sequence's or batch's) rows of the KV head
    int v0;                 // first tile of the span
    int n1, a0, w0;         // its tile v: at a0 + v T below n1, else at w0 + (v - n1) T
    int end;                // positions from here on are not there
    int start, keep1;       // visible to every row: [start, keep1)
    int S;                  // the sequence's length
    int last;               // of its CTA
    int back;               // tiles from the last to the first
    __device__ __forceinline__ int row_tiles() const { return rows > 128 ? 2 : 1; }
};
static_assert(sizeof(Item) == 64, "item");

// the part of shared memory behind the ring
template <int NACC> struct Sums;
template <> struct Sums<2> {
    float2 state[2][128];     // (m, l) of a warpgroup's lanes
    float row_scale[2][128];  // of an f32 q beside an f16 cache (at most 128 rows), every other item
};
template <> struct Sums<1> {
    float ref[128];           // m of a lane, passed from unit to unit
    float sum[2][128];        // l of a warpgroup's lanes
};
template <int NACC> struct alignas(16) Misc {
    Item item[2];             // the queue
    uint64_t bar[SB_N];
    uint32_t tmem;
    int abort;
    int started[2];           // an accumulator holds something before its first MMA
    uint32_t bad[2][4];       // rows of a unit's V tile that hold no numbers, by its S slot
    Sums<NACC> of;
};
static_assert(sizeof(Misc<1>) <= scored_misc(256) && sizeof(Misc<2>) <= scored_misc(128), "misc");
// in the epilogue, of rows that several lanes share: what their sum is multiplied by, and the row that
// it goes to
struct JoinRows {
    float factor[64];
    uint32_t to[64];
};
static_assert(sizeof(JoinRows) == kScoredRowBytes, "rows");

// rows by their group of heads, or by their sequence (see scored_inverse)
__device__ __forceinline__ int over_group(const ScoredParams &p, int row)
{
    return p.group == 1 ? row : (int)__umulhi((uint32_t)row, p.inv_group);
}
__device__ __forceinline__ int over_seq(const ScoredParams &p, int row)
{
    return p.per_seq == 1 ? row : (int)__umulhi((uint32_t)row, p.inv_seq);
}

__device__ __forceinline__ int length_of(const ScoredParams &p, int b)
{
    const int L = p.lens[b];
    return p.dev_lens ? max(0, min(__ldg(p.dev_lens + b), L)) : L;
}

// Lanes from one copy of a row tile to the next, and copies.
__device__ __forceinline__ int span_of(int rows)
{
    return rows > 64 ? 128 : rows > 32 ? 64 : 32;
}
__device__ __forceinline__ int reps_of(const ScoredParams &p, int rows)
{
    return rows > 128 ? 1 : max(1, p.rpad / span_of(rows));
}
// Copies of a row by the weights' terms: with two terms, half of the copies take the second.
template <typename C> __device__ __forceinline__ int shares_of_terms(int reps)
{
    return C::TP == 2 && !C::PK && reps > 1 ? 2 : 1;
}
// An item of the shared positions (known at compile time where there are none).
template <typename C> __device__ __forceinline__ bool of_all(const Item &it)
{
    return C::SH && it.b < 0;
}

// Sequence, head and (own) position of a row of an item.
template <typename C>
__device__ __forceinline__ void row_of(const ScoredParams &p, const Item &it, int row, int &b, int &h,
                                       int &own)
{
    const int Gh = p.group, per_seq = p.per_seq;
    int rr = it.row0 + row, S = it.S;
    b = it.b;
    if (of_all<C>(it)) {
        b = over_seq(p, rr);
        rr -= b * per_seq;
        S = length_of(p, b);
    }
    const int tk = over_group(p, rr);
    h = it.kvh * Gh + rr - tk * Gh;
    own = S - p.q_len + tk;
}

// What a softmax thread holds of an item: a row of it, and a share of its columns.
template <typename C> struct Lane {
    int nrt, span, reps, copies, shares;
    int rep, share, part;   // copy of the row tile, share of the columns, term of the weights
    int local;              // row of the item
    bool in_use, owner, busy; // (of its warp: in_use, busy)
    bool one_p;             // a lane holds one term of the weights
    int b, tk, h, own, S;   // sequence, token, head, the token's position, the sequence's length
    int out_row;
    __device__ __forceinline__ Lane(const ScoredParams &p, const Item &it, int w, int warp4, int lane)
    {
        nrt = it.row_tiles();
        constexpr int parts = C::PARTS;
        span = span_of(it.rows);
        reps = reps_of(p, it.rows);
        copies = reps * parts;
        const int terms = shares_of_terms<C>(reps);
        shares = reps / terms;
        one_p = parts * terms > 1;
        rep = warp4 * 32 / span;
        in_use = rep < reps;
        share = in_use ? rep % shares : 0;
        part = parts > 1 ? lane / (32 / parts) : in_use ? rep / shares : 0;
        local = nrt == 2     ? w * 128 + warp4 * 32 + lane
                : parts == 1 ? warp4 * 32 + lane - rep * span
                             : lane & (32 / parts - 1);
        owner = in_use && local < it.rows;
        busy = in_use && (local & ~31) < it.rows;
        const int Gh = p.group, per_seq = p.per_seq;
        int row = it.row0 + (owner ? local : 0);
        b = it.b;
        S = it.S;
        if (of_all<C>(it)) {
            b = over_seq(p, row);
            row -= b * per_seq;
            S = length_of(p, b);
        }
        tk = over_group(p, row);
        h = it.kvh * Gh + row - tk * Gh;
        own = S - p.q_len + tk;
        out_row = tk * p.hq + h;
    }
};

// The idx-th item.
template <typename C>
__device__ __forceinline__ void get_item(const ScoredParams &p, int idx, Item &it)
{
    constexpr int T = C::T;
    const int per_seq = p.per_seq;
    it.last = 0;
    // (a bias by distance favours the last positions: the references are set at once)
    it.back = p.slopes != nullptr;
    if (C::SH && idx < p.shared_items) {
        it.b = -1;
        const int u = idx / p.row_tiles;
        it.row0 = (idx - u * p.row_tiles) * p.tile_rows;
        it.split = u / p.hkv;
        it.kvh = u - it.split * p.hkv;
        it.rows = min(p.batch * per_seq - it.row0, p.tile_rows);
        it.v0 = it.split * p.shared_chunk;
        it.tiles = min(p.shared_tiles - it.v0, p.shared_chunk);
        it.n1 = it.a0 = it.w0 = 0;
        it.end = p.shared_len;
        it.start = it.keep1 = it.S = 0;
        return;
    }
    int t = C::SH ? idx - p.shared_items : idx;
    int u = t / p.row_groups;
    it.row0 = (t - u * p.row_groups) * p.tile_rows;
    it.rows = min(per_seq - it.row0, p.tile_rows);
    t = u / p.hkv;
    it.kvh = u - t * p.hkv;
    int lo = 0, hi = p.batch - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.base[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    const int b = p.seq[lo];
    it.b = b;
    it.split = t - p.base[lo];
    const int S = length_of(p, b);
    it.S = it.end = S;
    if (C::SH) { // (neither windows nor starts nor a kept prefix)
        it.start = it.keep1 = it.n1 = it.a0 = it.w0 = 0;
        it.v0 = it.split * p.chunk[b];
        it.tiles = max(0, min((S + T - 1) / T - it.v0, p.chunk[b]));
        return;
    }
    it.start = p.starts ? max(0, __ldg(p.starts + b)) : 0;
    int keep = p.keep;
    if (p.keep_lens) keep = max(0, min(__ldg(p.keep_lens + b), keep));
    it.keep1 = min(keep, S);
    // the visible span: what is kept, and from the first token's window on
    int from = it.start;
    if (p.window) from = max(from, max(S - p.q_len, 0) - p.window + 1);
    it.n1 = 0;
    it.a0 = 0;
    it.w0 = from / T * T;
    if (it.keep1 > it.start) {
        it.a0 = it.start / T * T;
        const int end1 = (it.keep1 + T - 1) / T * T;
        if (it.w0 > end1) it.n1 = (end1 - it.a0) / T;
        else it.w0 = it.a0;
    }
    const int n2 = S > from ? (S - it.w0 + T - 1) / T : 0;
    it.v0 = it.split * p.chunk[b];
    it.tiles = max(0, min(it.n1 + n2 - it.v0, p.chunk[b]));
}

template <int T> __device__ __forceinline__ int tile_at(const Item &it, int i)
{
    const int v = it.v0 + (it.back ? it.tiles - 1 - i : i);
    return v < it.n1 ? it.a0 + v * T : it.w0 + (v - it.n1) * T;
}

// byte offset of (row, byte) in a chunk: 128-byte rows, 128-byte swizzle
__device__ __forceinline__ uint32_t swz(uint32_t row, uint32_t byte)
{
    return (row >> 3) * 1024 + (row & 7) * 128 + ((((byte >> 4) ^ row) & 7) << 4) + (byte & 15);
}

// Waits for a phase as mbar_wait_bounded does, but looks at the clock and the flag now and then
// only (the loop is in many places, and has to be short).
__device__ __forceinline__ bool wait_phase(uint64_t *bar, uint32_t parity, uint64_t limit_ns,
                                           volatile int *abort)
{
    uint64_t t0 = 0;
#pragma unroll 1
    for (uint32_t n = 1; !mbar_try_wait(bar, parity); ++n) {
        if (n & 31u) continue;
        const uint64_t t = global_ns();
        if (t0 == 0) t0 = t;
        if (*abort || t - t0 > limit_ns) return false;
    }
    return true;
}

// The same for a whole warp. Its branches depend on votes only: lanes that left such a loop at different
// times would run what follows apart from each other, joining at every exchange (measured on the
// warps of the copies: five times slower until their next wait).
__device__ __forceinline__ bool wait_phase_warp(uint64_t *bar, uint32_t parity, uint64_t limit_ns,
                                                volatile int *abort)
{
    uint64_t t0 = 0;
#pragma unroll 1
    for (uint32_t n = 1; !__all_sync(0xffffffffu, mbar_try_wait(bar, parity)); ++n) {
        if (n & 31u) continue;
        const uint64_t t = global_ns();
        if (t0 == 0) t0 = t;
        if (__any_sync(0xffffffffu, *abort || t - t0 > limit_ns)) return false;
    }
    return true;
}

template <typename DT> struct Pair;
template <> struct Pair<__half> {
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t w)
    {
        return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    }
};
template <> struct Pair<__nv_bfloat16> {
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t w)
    {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
};

__device__ __forceinline__ uint4 lds_v4(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}

// A from TMEM (16-bit, two columns of A a word), B from shared memory
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                          uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
                 "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
                 : "memory");
}

__device__ __forceinline__ void tmem_st16w(uint32_t taddr, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,"
                 "%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
                 "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
                 "r"(r[14]), "r"(r[15])
                 : "memory");
}

__device__ __forceinline__ void tmem_st8w(uint32_t taddr, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
                 "r"(r[7])
                 : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float *v)
{
    uint32_t r[32];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// The scores of few rows, spread over a warp: lanes 0 - 15 (or 16 - 31, of taddr) of 8 N columns.
// Thread t gets row t / 4 (r[4 g], r[4 g + 1]) and row t / 4 + 8 (r[4 g + 2], r[4 g + 3]) of columns
// 8 g + 2 (t % 4) and the one behind it.
template <int N> __device__ __forceinline__ void tmem_ld_rows(uint32_t taddr, float *v)
{
    static_assert(N == 2 || N == 4, "groups of 8 columns");
    uint32_t r[4 * N];
    if constexpr (N == 2) {
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                     "=r"(r[6]), "=r"(r[7])
                     : "r"(taddr));
    } else {
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,"
                     "%11,%12,%13,%14,%15}, [%16];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                     "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
                     "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                     : "r"(taddr));
    }
#pragma unroll
    for (int i = 0; i < 4 * N; ++i) v[i] = __uint_as_float(r[i]);
}
template <int N> __device__ __forceinline__ void tmem_st_rows(uint32_t taddr, const float *v)
{
    static_assert(N == 2 || N == 4, "groups of 8 columns");
    uint32_t r[4 * N];
#pragma unroll
    for (int i = 0; i < 4 * N; ++i) r[i] = __float_as_uint(v[i]);
    if constexpr (N == 2) {
        asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,"
                     "%8};" ::"r"(taddr),
                     "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
                     "r"(r[7])
                     : "memory");
    } else {
        asm volatile("tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,"
                     "%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
                     "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
                     "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
                     "r"(r[13]), "r"(r[14]), "r"(r[15])
                     : "memory");
    }
}
// 16-bit pairs of the same rows and positions: 4 N columns, thread t's word of group g is column
// 4 g + t % 4 of row t / 4 (r[2 g]) and of row t / 4 + 8 (r[2 g + 1]).
template <int N> __device__ __forceinline__ void tmem_st_pairs(uint32_t taddr, const uint32_t *r)
{
    static_assert(N == 2 || N == 4 || N == 8 || N == 16, "groups of 4 columns");
    if constexpr (N == 2) {
        asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr),
                     "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
                     : "memory");
    } else if constexpr (N == 4) {
        asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,"
                     "%8};" ::"r"(taddr),
                     "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
                     "r"(r[7])
                     : "memory");
    } else if constexpr (N == 8) {
        asm volatile("tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,"
                     "%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
                     "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
                     "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
                     "r"(r[13]), "r"(r[14]), "r"(r[15])
                     : "memory");
    } else {
        asm volatile("tcgen05.st.sync.aligned.16x128b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,"
                     "%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,"
                     "%28,%29,%30,%31,%32};" ::"r"(taddr),
                     "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
                     "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
                     "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
                     "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
                     "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]),
                     "r"(r[31])
                     : "memory");
    }
}

// one lane of a whole warp
__device__ __forceinline__ bool elect_one()
{
    uint32_t on;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(on));
    return on != 0;
}

template <int N> __device__ __forceinline__ void setmaxnreg_inc()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void setmaxnreg_dec()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// (volatile, in program order with the other TMEM accesses)
__device__ __forceinline__ float tmem_ld1(uint32_t taddr)
{
    uint32_t r;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
    tmem_wait_ld();
    return __uint_as_float(r);
}

__device__ __forceinline__ uint64_t l2_normal_policy()
{
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}

// What turns a row's raw score into y log2 e. (Kernels for a cap, for a bias, and for both: the softmax
// warps are as fast as their instructions come. With one for all three: drafts behind 61440 shared
// positions, capped, 226 us, without the bias 209; bias by distance 153 and 149.)
struct Scorer {
    float mult;      // scale log2 e of the row
    float cap;       // softcap log2 e; 0: none
    float turn;      // scale / softcap of the row
    float slope;     // slope log2 e
};

__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// c tanh z. For |z| < 0.75, where (e^2z - 1) / (e^2z + 1) is far off relative to tanh z, Lambert's
// continued fraction to its fifth term, z (945 + 105 z^2 + z^4) / (945 + 420 z^2 + 15 z^4), off by less
// than 2^-26 there; both are one quotient. (Comparisons that keep a NaN.)
__device__ __forceinline__ float capped(float z, float c)
{
    z = z > 10.f ? 10.f : z;
    z = z < -10.f ? -10.f : z;
    const float t = ex2(z * (2.f * kLog2e)), zz = z * z;
    const bool near = fabsf(z) < 0.75f;
    const float num = near ? z * fmaf(zz, zz + 105.f, 945.f) : t - 1.f;
    const float den = near ? fmaf(zz, fmaf(zz, 15.f, 420.f), 945.f) : t + 1.f;
    return c * num * rcp(den);
}

// c tanh z of two scores with |z| < 1 / 4, where a cap is far above the scores, from the series
// z - z^3 / 3 + 2 z^5 / 15 - 17 z^7 / 315 + 62 z^9 / 2835: off by less than 2^-26 of it, and without
// the special function unit's two steps a score, which take four times as long.
constexpr float kNearCap = 0.25f;
__device__ __forceinline__ float2 capped_near(float2 z, float c)
{
    const float2 zz = __fmul2_rn(z, z);
    float2 s = __ffma2_rn(zz, make_float2(62.f / 2835.f, 62.f / 2835.f),
                          make_float2(-17.f / 315.f, -17.f / 315.f));
    s = __ffma2_rn(zz, s, make_float2(2.f / 15.f, 2.f / 15.f));
    s = __ffma2_rn(zz, s, make_float2(-1.f / 3.f, -1.f / 3.f));
    s = __fmul2_rn(zz, s);
    z = __fmul2_rn(z, make_float2(c, c));
    return __ffma2_rn(z, s, z);
}

// bits i of 0 .. 31 with lo <= i < hi
__device__ __forceinline__ uint32_t range32(int lo, int hi)
{
    lo = max(lo, 0);
    hi = min(hi, 32);
    return hi > lo ? (0xffffffffu >> (32 - hi)) & (0xffffffffu << lo) : 0u;
}

// the power of two at or below a, from its exponent's bits (subnormals, infinities: 1)
__device__ __forceinline__ float pow2_of(float a)
{
    const uint32_t e = __float_as_uint(a) >> 23;
    return e < 1 || e > 253 ? 1.f : __uint_as_float(e << 23);
}

// largest |q| of the f32 row at `at`
template <int D> __device__ __forceinline__ float row_max(const void *q, int64_t at)
{
    const float4 *src = reinterpret_cast<const float4 *>(static_cast<const float *>(q) + at);
    float a = 0.f;
#pragma unroll 32
    for (int i = 0; i < D / 4; ++i) {
        const float4 y = __ldg(src + i);
        a = fmaxf(a, fmaxf(fmaxf(fabsf(y.x), fabsf(y.y)), fmaxf(fabsf(y.z), fabsf(y.w))));
    }
    return a;
}

template <typename C>
__global__ void __launch_bounds__(C::THREADS, 1)
    gqa_scored_kernel(const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap,
                      const __grid_constant__ ScoredParams p)
{
    using DT = typename C::DT;
    constexpr int D = C::D, T = C::T, NCH = C::NCH, NACC = C::NACC, TP = C::TP, CHUNK = C::CHUNK;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(sm);
    const int nst = p.slots;
    auto *ms = reinterpret_cast<Misc<NACC> *>(sm + p.q_bytes + nst * C::SLOT + p.join_bytes);
    uint64_t *bar = ms->bar;
    volatile int *abort_flag = &ms->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int Gh = p.group;
    const int qch = p.rpad * 128; // bytes of a Q chunk
    volatile int never = 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < nst; ++s) {
            mbar_init(bar + SB_FULL + s, 1);
            mbar_init(bar + SB_EMPTY + s, 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar + SB_SFULL + s, 1);
            mbar_init(bar + SB_PFULL + s, 4);
            mbar_init(bar + SB_PVDONE + s, 1);
            mbar_init(bar + SB_GROUP + s, 4);
            mbar_init(bar + SB_REF + s, 4);
        }
        mbar_init(bar + SB_OREADY, 1);
        mbar_init(bar + SB_OFREE, C::WARPS);
        mbar_init(bar + SB_QFULL, C::WARPS);
        mbar_init(bar + SB_QFREE, 1);
        mbar_init(bar + SB_XCH, C::WARPS);
        mbar_init(bar + SB_DRAIN, 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar + SB_ITEM + s, 1);
            mbar_init(bar + SB_TAKEN + s, C::WARPS + 2); // softmax warps, V copies, MMAs
        }
        ms->abort = 0;
        if (blockIdx.x == 0) *p.status = 0;
        fence_mbar_init();
    }
    if (warp == C::MMA_WARP) tmem_alloc(&ms->tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ms->tmem;
    auto timed_out = [&]() {
        *abort_flag = 1;
        atomicCAS(p.status, 0, kStatusTimeoutScored);
    };

    // slots 0 .. nk - 1 of the ring are for K tiles, the others for V tiles (which are held longer)
    const int nk = nst / 2;
    // a walk through slots first .. last - 1 and the phases of their barriers
    struct Ring {
        int first, last, slot;
        uint32_t phase;
        __device__ __forceinline__ void advance()
        {
            if (++slot == last) {
                slot = first;
                phase ^= 1u;
            }
        }
    };
    int taken = 0; // items from the queue

    if (warp == C::K_WARP || warp == C::V_WARP) {
        // ============================ copies of K, or of V ============================
        setmaxnreg_dec<C::OTHER_REGS>();
        const bool is_v = warp == C::V_WARP;
        if (lane == 0) tma_prefetch_map(is_v ? &vmap : &kmap);
        const uint64_t once = l2_evict_first_policy(), normal = l2_normal_policy();
        const bool paged = p.block_table != nullptr;
        Ring ring = {is_v ? nk : 0, is_v ? nst : nk, is_v ? nk : 0, 0u};
        bool ok = true;
        auto wait = [&](int b, uint32_t parity) {
            ok = ok && wait_phase_warp(bar + b, parity, p.timeout_ns, abort_flag);
            return ok;
        };
        // lanes hold the 64 table entries from `base` on, the second half ahead of its use
        const int32_t *tab = nullptr;
        int width = 0, base = -1;
        int32_t near = 0, next = 0;
        auto entry = [&](int i) { return i >= 0 && i < width ? __ldg(tab + i) : p.oob_block; };
        struct At { // of this lane's box of a tile: block (or sequence) and position in it
            int blk, pos;
        };
        const int h = paged ? p.box_rows : T, nbox = T / h;
        auto locate = [&](const Item &it, int tile) {
            const int t0 = tile_at<T>(it, tile);
            if (!paged) return At{it.b, t0};
            // box j: h rows of one block, h a divisor of the tile and of the block
            const int bs = p.block_size, pos = t0 + min(lane, nbox - 1) * h, e = pos / bs;
            const int lo = __shfl_sync(0xffffffffu, e, 0);
            if (base < 0 || lo < base || lo >= base + 64) {
                base = lo;
                near = entry(base + lane);
                next = entry(base + 32 + lane);
            } else if (lo >= base + 32) {
                base += 32;
                near = next;
                next = entry(base + 32 + lane);
            }
            // (a tile lies in at most 9 blocks)
            const int i = e - base;
            const int x = __shfl_sync(0xffffffffu, near, i & 31);
            const int y = __shfl_sync(0xffffffffu, next, i & 31);
            int blk = i < 32 ? x : y;
            if (pos >= it.end || blk < 0) blk = p.oob_block; // reads as zeros
            return At{blk, pos - e * bs};
        };
        auto copies = [&](const Item &it, const CUtensorMap *map) {
            if (it.tiles == 0) return;
            if (paged) {
                tab = of_all<C>(it) ? p.shared_table : p.block_table + (size_t)it.b * p.max_blocks;
                width = of_all<C>(it) ? p.shared_len / p.block_size : p.max_blocks;
                base = -1;
            }
            // shared tiles are read by every row tile's items
            const uint64_t pol = C::SH && p.row_tiles > 1 && it.b < 0 ? normal : once;
            At at = locate(it, 0);
#pragma unroll 1
            for (int i = 0; i < it.tiles; ++i) {
                if (!wait(SB_EMPTY + ring.slot, ring.phase ^ 1u)) return;
                if (!(p.flags & DA_FLAG_TEST_NO_TMA)) {
                    uint8_t *dst = sm + p.q_bytes + ring.slot * C::SLOT;
                    uint64_t *full = bar + SB_FULL + ring.slot;
                    if (elect_one()) mbar_arrive_expect_tx(full, C::SLOT);
#pragma unroll 1
                    for (int j = 0; j < nbox; ++j, dst += h * 128) {
                        const int blk = __shfl_sync(0xffffffffu, at.blk, j);
                        const int pos = __shfl_sync(0xffffffffu, at.pos, j);
                        if (elect_one()) {
#pragma unroll
                            for (int c = 0; c < NCH; ++c)
                                tma_load_4d(dst + c * CHUNK, map, full, c * 64, it.kvh, pos, blk, pol);
                        }
                    }
                    __syncwarp();
                }
                ring.advance();
                if (i + 1 < it.tiles) at = locate(it, i + 1);
            }
        };
        if (!is_v) {
            // this warp works the items out
            int passed = 0; // items put in the queue
            auto pass_on = [&](const Item &it) {
                const int s = passed & 1;
                if (!wait(SB_TAKEN + s, ((uint32_t)(passed >> 1) & 1u) ^ 1u)) return false;
                if (lane == 0) {
                    ms->item[s] = it;
                    mbar_arrive(bar + SB_ITEM + s);
                }
                ++passed;
                return true;
            };
            const int g = gridDim.x;
            const ScoredOrder order = {g, C::SH ? p.shared_items : 0, p.lead};
            auto nth = [&](int r) { // this CTA's items
                const int64_t idx = order.item(blockIdx.x, r);
                return idx < p.n_items ? (int)idx : -1;
            };
            Item it;
            // (behind the first that is not there there are none)
#pragma unroll 1
            for (int r = 0, idx = nth(0); ok && idx >= 0; ++r) {
                const int then = nth(r + 1);
                get_item<C>(p, idx, it);
                it.last = then < 0;
                if (pass_on(it)) copies(it, &kmap);
                idx = then;
            }
            it.tiles = -1;
            if (ok) (void)pass_on(it);
        } else {
#pragma unroll 1
            for (;; ++taken) {
                const int q = taken & 1;
                if (!wait(SB_ITEM + q, (uint32_t)(taken >> 1) & 1u)) break;
                const Item it = ms->item[q];
                __syncwarp();
                if (lane == 0) mbar_arrive(bar + SB_TAKEN + q);
                if (it.tiles < 0) break;
                copies(it, &vmap);
                if (!ok) break;
            }
        }
        if (lane == 0) {
            if (!ok) timed_out();
            // Nothing may be in flight when the CTA ends: the last copy into every slot, those of
            // the current round up to this slot and the round's before behind it.
            if (!(p.flags & DA_FLAG_TEST_NO_TMA))
                for (int s = ring.first; s < ring.last; ++s) {
                    const uint32_t ph = s < ring.slot ? ring.phase : ring.phase ^ 1u;
                    // (a slot that has not been used is in its first phase: the one before it
                    // counts as complete)
                    (void)wait_phase(bar + SB_FULL + s, ph, p.timeout_ns, &never);
                }
        }
        __syncwarp();
    } else if (warp == C::MMA_WARP) {
        // ============================ MMA issue (one thread) ============================
        setmaxnreg_dec<C::OTHER_REGS>();
        if (elect_one()) {
            constexpr uint32_t idesc_qk = idesc_f16kind(128, T, 0, 0, C::BF);
            constexpr uint32_t idesc_pv = idesc_f16kind(128, D, 0, 1, C::BF);
            uint32_t pph = 0;      // phases of PFULL, by slot
            bool ok = true;
            auto wait = [&](int b, uint32_t parity) {
                ok = ok && wait_phase(bar + b, parity, p.timeout_ns, abort_flag);
                return ok;
            };
            Ring kr = {0, nk, 0, 0u}, vr = {nk, nst, nk, 0u};
            auto take = [&](Ring &x, int &slot) { // waits for the next tile
                slot = x.slot;
                if (!wait(SB_FULL + x.slot, x.phase)) return false;
                x.advance();
                return true;
            };
            const uint32_t ring = sb + p.q_bytes;
            auto item = [&](int tiles, int rows, uint32_t nth) {
                const int sh = rows > 128 ? 1 : 0, nu = tiles << sh;
                const bool one_p = C::PK || shares_of_terms<C>(reps_of(p, rows)) > 1;
                const int q_terms = C::PK ? 1 : p.q_terms;
                int ks = 0, vs = 0;
                if (!wait(SB_QFULL, nth & 1u)) return false;
                for (int v = 0; v < nu + 2; ++v) {
                    if (v >= 2) { // O += P V of unit v - 2
                        const int u = v - 2, s = u & 1, w = NACC == 2 ? s : 0;
                        if (u == 0 && !wait(SB_OFREE, nth & 1u)) return false;
                        if (!wait(SB_PFULL + s, (pph >> s) & 1u)) return false;
                        pph ^= 1u << s;
                        if ((sh == 0 || !(u & 1)) && !take(vr, vs)) return false;
                        tc_fence_after();
                        const uint64_t vd = smem_desc_sw128(ring + vs * C::SLOT, CHUNK, 1024);
                        const uint32_t a = tmem + C::S_COL + s * C::S_SLOT;
                        const bool more = u >= NACC ||
                                          *static_cast<volatile int *>(ms->started + w);
                        if (one_p) {
#pragma unroll 4
                            for (int k = 0; k < T / 16; ++k)
                                tc_mma_ts(tmem + w * D, a + 8 * k, vd + (uint64_t)((k * 2048) >> 4),
                                          idesc_pv, k || more ? 1u : 0u);
                        } else {
#pragma unroll 1
                            for (int x = 0; x < TP; ++x)
#pragma unroll 4
                                for (int k = 0; k < T / 16; ++k)
                                    tc_mma_ts(tmem + w * D,
                                              x < 2 ? a + 16 * k + 8 * x : a + T + 8 * k,
                                              vd + (uint64_t)((k * 2048) >> 4), idesc_pv,
                                              x || k || more ? 1u : 0u);
                        }
                        if (sh == 0 || (u & 1)) tc_commit(bar + SB_EMPTY + vs);
                        tc_commit(bar + SB_PVDONE + w);
                    }
                    if (v < nu) { // S of unit v
                        const int s = v & 1;
                        if ((sh == 0 || !(v & 1)) && !take(kr, ks)) return false;
                        tc_fence_after();
                        const uint32_t sd = tmem + C::S_COL + s * C::S_SLOT;
                        const uint64_t qd = smem_desc_sw128(
                            sb + (sh ? (v & 1) * p.q_terms * NCH * qch : 0), 16, 1024);
                        const uint64_t kd = smem_desc_sw128(ring + ks * C::SLOT, 16, 1024);
                        // the small terms first: an MMA's sums are cut off at their 24th bit, so
                        // that each addition to a large sum costs about 2^-24 of it
                        constexpr int tm = C::QTM ? 1 : 0; // terms in TMEM
#pragma unroll 1
                        for (int x = q_terms - 1; x >= tm; --x)
#pragma unroll 1
                            for (int c = 0; c < NCH; ++c)
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    tc_mma_bf16(
                                        sd, qd + (uint64_t)((((x - tm) * NCH + c) * qch + k * 32) >> 4),
                                        kd + (uint64_t)((c * CHUNK + k * 32) >> 4), idesc_qk,
                                        x != q_terms - 1 || (c | k) != 0 ? 1u : 0u);
                        if (C::QTM) {
#pragma unroll 1
                            for (int c = 0; c < NCH; ++c)
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    tc_mma_ts(sd, tmem + C::Q_COL + (c * 4 + k) * 8,
                                              kd + (uint64_t)((c * CHUNK + k * 32) >> 4), idesc_qk,
                                              q_terms > 1 || (c | k) != 0 ? 1u : 0u);
                        }
                        tc_commit(bar + SB_SFULL + s);
                        if (sh == 0 || (v & 1)) tc_commit(bar + SB_EMPTY + ks);
                        if (v == nu - 1) tc_commit(bar + SB_QFREE);
                    }
                }
                tc_commit(bar + SB_OREADY);
                return true;
            };
            uint32_t live = 0;     // items with tiles so far
            for (int i = 0; ok; ++i) {
                const int q = i & 1;
                if (!wait(SB_ITEM + q, (uint32_t)(i >> 1) & 1u)) break;
                const int tiles = ms->item[q].tiles, rows = ms->item[q].rows;
                mbar_arrive(bar + SB_TAKEN + q);
                if (tiles < 0) break;
                if (tiles > 0) (void)item(tiles, rows, live++);
            }
            if (!ok) timed_out();
            // no MMA may be in flight when TMEM is freed
            tc_commit(bar + SB_DRAIN);
            (void)wait_phase(bar + SB_DRAIN, 0, p.timeout_ns, &never);
        }
        __syncwarp();
    } else if (warp < C::WARPS) {
        // ========================= softmax and epilogue =========================
        setmaxnreg_inc<C::SOFTMAX_REGS>();
        const int w = warp >> 2;              // warpgroup
        const int r = threadIdx.x & 127;      // row of the row tile, TMEM lane
        const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t to = tl + (NACC == 2 ? w : 0) * D; // its accumulator
        int n = 0, items = 0;                 // V tiles and items with tiles before this item
        uint32_t sph = 0;                     // phases of SFULL, by slot
        int done = 0;                         // units of its accumulator so far
        int handed = 0;                       // units of the other warpgroup before this item
        uint32_t groups = 0, joints = 0;      // uses of SB_GROUP and SB_XCH
        bool ok = true;
        auto wait = [&](int b, uint32_t parity) {
            ok = wait_phase_warp(bar + b, parity, p.timeout_ns, abort_flag);
            return ok;
        };
        auto arrive = [&](int b) {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar + b);
        };
        // all warps of the warpgroup, or of both, have come here
        auto group_sync = [&]() {
            arrive(SB_GROUP + w);
            return wait(SB_GROUP + w, groups++ & 1u);
        };
        auto all_sync = [&]() {
            arrive(SB_XCH);
            return wait(SB_XCH, joints++ & 1u);
        };
        arrive(SB_OFREE);

        // Q of an item with tiles, once the last one's scores are done with it; returns false after a
        // timeout. scale: of this lane's row (256 columns, an f32 q beside an f16 cache)
        auto load_q = [&](const Item &it, int nth, float &row_scale) {
            const Lane<C> me(p, it, w, warp & 3, lane);
            constexpr int parts = C::PARTS;
            const int part = me.part, reps = me.reps, span = me.span;
            const bool busy = me.busy;
            const int per_seq = p.per_seq;
            if (nth > 0 && !wait(SB_QFREE, (uint32_t)(nth - 1) & 1u)) return false;
            tc_fence_after();
            const int64_t q_at = (((int64_t)me.b * p.q_len + me.tk) * p.hq + me.h) * D;
            row_scale = 1.f;
            if (C::QTM) {
                // each lane half of its own row: one term into TMEM, the second of an f32 q that is
                // not packed into shared memory
                if (busy && !p.q_f32) {
                    const uint4 *src = reinterpret_cast<const uint4 *>(
                        static_cast<const uint16_t *>(p.q) + q_at + w * (D / 2));
                    uint4 y[D / 16];
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) y[i] = __ldg(src + i);
#pragma unroll
                    for (int i = 0; i < D / 16; i += 4) {
                        const uint32_t v[16] = {
                            y[i].x,     y[i].y,     y[i].z,     y[i].w,     y[i + 1].x, y[i + 1].y,
                            y[i + 1].z, y[i + 1].w, y[i + 2].x, y[i + 2].y, y[i + 2].z, y[i + 2].w,
                            y[i + 3].x, y[i + 3].y, y[i + 3].z, y[i + 3].w};
                        tmem_st16w(tl + C::Q_COL + w * (D / 4) + i * 4, v);
                    }
                    tmem_wait_st();
                } else if (busy) {
                    if (!C::BF) row_scale = pow2_of(row_max<D>(p.q, q_at));
                    const float down = 1.f / row_scale;
                    const float4 *src = reinterpret_cast<const float4 *>(
                        static_cast<const float *>(p.q) + q_at);
                    {
                        const int c = w * (D / 2);
                        float4 y[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) y[i] = __ldg(src + c / 4 + i);
#pragma unroll
                        for (int i = 0; i < 32; i += 8) {
                            uint32_t v[16], second[16];
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const float f[4] = {y[i + k].x * down, y[i + k].y * down,
                                                    y[i + k].z * down, y[i + k].w * down};
#pragma unroll
                                for (int e = 0; e < 4; e += 2) {
                                    const uint32_t a = Pair<DT>::pack(f[e], f[e + 1]);
                                    const float2 z = Pair<DT>::unpack(a);
                                    const uint32_t a2 = Pair<DT>::pack(f[e] - z.x, f[e + 1] - z.y);
                                    v[2 * k + e / 2] = parts > 1 && part == 1 ? a2 : a;
                                    second[2 * k + e / 2] = a2;
                                }
                            }
                            tmem_st16w(tl + C::Q_COL + c / 2 + i * 2, v);
                            if (parts == 1) {
                                const int col = c + 4 * i; // of the row, 32 of them
                                const uint32_t at = sb + (col >> 6) * qch;
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    sts_v4(at + swz(r, (col & 63) * 2 + 16 * k), second[4 * k],
                                           second[4 * k + 1], second[4 * k + 2], second[4 * k + 3]);
                            }
                        }
                    }
                    tmem_wait_st();
                    if (parts == 1) fence_proxy_async_smem();
                }
                tc_fence_before();
            }
            if (!C::QTM) { // all terms in shared memory
                // 8-column units, a half-warp's or a warp's to a row; four of a thread in flight
                // (rows past the last eight give scores that nobody reads)
                constexpr int U8 = D / 8, STEP = C::WARPS * 32;
                const int units = (it.rows + 7) / 8 * 8 * U8;
                const int j = threadIdx.x % U8; // (the step is a multiple of a row)
                auto source = [&](int rr) { // element of q, or -1
                    if (rr >= it.rows) return (int64_t)-1;
                    int qrow = it.row0 + rr, qb = it.b;
                    if (of_all<C>(it)) {
                        qb = over_seq(p, qrow);
                        qrow -= qb * per_seq;
                    }
                    const int qt = over_group(p, qrow), qh = it.kvh * Gh + qrow - qt * Gh;
                    return (((int64_t)qb * p.q_len + qt) * p.hq + qh) * D + j * 8;
                };
                // unit j of row rr: term x, at all copies of the row
                auto put = [&](int rr, int x, const uint32_t *v) {
                    const uint32_t dst = sb + (rr >> 7) * p.q_terms * NCH * qch + (j >> 3) * qch +
                                         (parts == 1 ? x * NCH * qch : 0);
                    const int first = (rr & 127) + (parts == 1 ? 0 : x * (32 / parts));
#pragma unroll 1
                    for (int k = 0; k < reps; ++k)
                        sts_v4(dst + swz(first + k * span, (j & 7) * 16), v[0], v[1], v[2], v[3]);
                };
                if (!p.q_f32) {
#pragma unroll 1
                    for (int u0 = threadIdx.x; u0 < units; u0 += 4 * STEP) {
                        uint4 x[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int u = u0 + i * STEP;
                            const int64_t at = u < units ? source(u / U8) : -1;
                            x[i] = make_uint4(0, 0, 0, 0);
                            if (at >= 0) x[i] = __ldg(reinterpret_cast<const uint4 *>(
                                             static_cast<const uint16_t *>(p.q) + at));
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int u = u0 + i * STEP;
                            if (u >= units) break;
                            const uint32_t v[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                            for (int k = 0; k < parts; ++k) put(u / U8, k, v); // (every lane's score)
                        }
                    }
                } else {
#pragma unroll 1
                    for (int u0 = threadIdx.x; u0 < units; u0 += 4 * STEP) {
                        float4 xa[4], xb[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int u = u0 + i * STEP;
                            const int64_t at = u < units ? source(u / U8) : -1;
                            xa[i] = xb[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (at >= 0) {
                                const float4 *src = reinterpret_cast<const float4 *>(
                                    static_cast<const float *>(p.q) + at);
                                xa[i] = __ldg(src);
                                xb[i] = __ldg(src + 1);
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int u = u0 + i * STEP;
                            if (u >= units) break; // (whole warps: units is a multiple of 128)
                            float f[8] = {xa[i].x, xa[i].y, xa[i].z, xa[i].w,
                                          xb[i].x, xb[i].y, xb[i].z, xb[i].w};
                            if (!C::BF) {
                                // f16: the row scaled to a largest element in [1, 2), so that two
                                // terms keep 22 bits of it
                                float a = 0.f;
#pragma unroll
                                for (int e = 0; e < 8; ++e) a = fmaxf(a, fabsf(f[e]));
#pragma unroll
                                for (int o = U8 / 2; o > 0; o >>= 1)
                                    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
                                const float up = pow2_of(a);
                                if constexpr (NACC == 2) {
                                    if (j == 0) ms->of.row_scale[nth & 1][u / U8] = up;
                                }
                                const float down = 1.f / up;
#pragma unroll
                                for (int k = 0; k < 8; ++k) f[k] *= down;
                            }
#pragma unroll 1
                            for (int x = 0; x < (parts > 1 ? parts : p.q_terms); ++x) {
                                uint32_t v[4];
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    v[k] = Pair<DT>::pack(f[2 * k], f[2 * k + 1]);
                                    const float2 y = Pair<DT>::unpack(v[k]);
                                    f[2 * k] -= y.x;
                                    f[2 * k + 1] -= y.y;
                                    if (x >= p.q_terms) v[k] = 0u; // (four lanes, three terms)
                                }
                                put(u / U8, x, v);
                            }
                        }
                    }
                }
                fence_proxy_async_smem();
            }
            arrive(SB_QFULL);
            return true;
        };
        // An item without positions to see: neutral partials.
        auto neutral = [&](const Item &it) {
            const Lane<C> me(p, it, w, warp & 3, lane);
            if (!me.owner || me.rep || me.part || (me.nrt == 1 && w)) return;
            const size_t slot = (size_t)p.slot[me.b] + it.split + (of_all<C>(it) ? 0 : p.shared_splits);
            const size_t row = p.whole ? (size_t)me.b * p.rows + me.out_row : slot * p.rows + me.out_row;
            if (!p.whole) {
                p.ml[row] = make_float2(kNeutralM, 0.f);
                return;
            }
            const int bytes = D * (p.out_dtype == DA_F32 ? 4 : 2);
            uint4 *out = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.out) + row * bytes);
#pragma unroll 1
            for (int i = 0; i < bytes / 16; ++i) out[i] = make_uint4(0, 0, 0, 0);
        };
        // The units and the epilogue of an item (of one without tiles: neither). before_join is called
        // between them, once this warp's scores of the item are done with.
        auto work = [&](const Item &it, float row_scale, auto &&before_join) {
            const Lane<C> me(p, it, w, warp & 3, lane);
            const int nrt = me.nrt, part = me.part, span = me.span, reps = me.reps;
            const int copies = me.copies, shares = me.shares, rep = me.rep, share = me.share;
            const int local = me.local, b = me.b, h = me.h, own = me.own;
            const bool owner = me.owner, busy = me.busy, one_p = me.one_p;
            const int cols = T / shares, cb = share * cols;
            const int q0 = it.S - p.q_len;         // of a sequence's own item: its first token
            const bool dead = !owner || own < 0;   // no such token: it sees nothing
            const size_t slot = (size_t)p.slot[b] + it.split + (of_all<C>(it) ? 0 : p.shared_splits);
            // its row of the output, or of the partials
            const size_t dst_row =
                p.whole ? (size_t)b * p.rows + me.out_row : slot * p.rows + me.out_row;
            auto write4 = [&](size_t row_at, int c, const float4 &f) {
                if (!p.whole) {
                    store4(p.acc + row_at * D + c, f);
                    return;
                }
                const size_t at = row_at * D + c;
                if (p.out_dtype == DA_F32) store4(static_cast<float *>(p.out) + at, f);
                else if (p.out_dtype == DA_F16) store4(static_cast<__half *>(p.out) + at, f);
                else store4(static_cast<__nv_bfloat16 *>(p.out) + at, f);
            };

            if (TP == 3 && !one_p && reps > 1 && busy) {
                // the third terms have columns of their own: zero but for this warp's share
                const uint32_t z[16] = {};
                for (int c = 0; c < T / 2; c += 16)
                    tmem_st16w(tl + C::S_COL + w * C::S_SLOT + T + c, z);
                tmem_wait_st();
            }

            const int window = C::SH ? 0 : p.window, start = C::SH ? 0 : it.start;
            const int keep1 = C::SH ? 0 : it.keep1;

            // ---- what rows see and how they score: of unpacked items this lane's row (the first of
            // two), of packed ones rows lane / 4 and lane / 4 + 8, four lanes to a row
            constexpr bool packed = C::PK;
            constexpr int PR = C::PK && TP == 2 ? 2 : 1; // rows of a thread in packed items
            struct Row {
                bool real;
                int pos, x_lo, x_hi;
                Scorer sc;
                float m, l;
            } rows[PR];
#pragma unroll
            for (int k = 0; k < PR; ++k) {
                Row &y = rows[k];
                int rr = local, rb = b, rh = h, at = own;
                y.real = owner;
                if (packed) {
                    rr = (lane >> 2) + 8 * k;
                    y.real = me.in_use && rr < it.rows;
                    row_of<C>(p, it, y.real ? rr : 0, rb, rh, at);
                }
                y.pos = at + (of_all<C>(it) ? p.shared_len : 0); // in this item's positions
                y.x_lo = window ? max(start, at - window + 1) : start;
                y.x_hi = !y.real || at < 0 ? 0 : at + 1;
                y.sc.slope = C::XF && p.slopes && y.real ? __ldg(p.slopes + rh) * kLog2e : 0.f;
                y.sc.cap = p.softcap * kLog2e;
                y.sc.mult = y.sc.turn = 0.f;
                y.m = -INFINITY;
                y.l = 0.f;
            }
            // a value of a packed item's row, for the lanes that hold a term of it
            auto of_lane = [&](float first, float second) {
                const int src = (local & 7) * 4;
                const float x = __shfl_sync(0xffffffffu, first, src);
                const float y = __shfl_sync(0xffffffffu, second, src);
                return local >= 8 ? y : x;
            };

            // where a lane's state is exchanged (packed: that of a row, by its warp)
            auto state_at = [&](int k) {
                return packed ? (warp & 3) * 32 + (lane >> 2) + 8 * k : r;
            };
            // the references as unit u left them, one of the other warpgroup (if there is one)
            auto take = [&](int u) {
                if constexpr (NACC == 1) {
                    if (u < 0) return true;
                    if (!wait(SB_REF + 1 - w, (uint32_t)(handed + (u >> 1)) & 1u)) return false;
#pragma unroll
                    for (int k = 0; k < PR; ++k) {
                        const float m = ms->of.ref[state_at(k)];
                        if (rows[k].l != 0.f && m != rows[k].m) rows[k].l *= ex2(rows[k].m - m);
                        rows[k].m = m;
                    }
                }
                return true;
            };

            // ---- units
            const int nu = it.tiles * nrt;
            int mine = 0; // units of this item so far
#pragma unroll 1
            for (int u = w; u < nu; u += 2) {
                const int tile = nrt == 2 ? u >> 1 : u, s = w;
                const int t0 = tile_at<T>(it, tile);
                const uint32_t ts = tl + C::S_COL + s * C::S_SLOT;
                if (!wait(SB_SFULL + s, (sph >> s) & 1u)) return false;
                sph ^= 1u << s;
                tc_fence_after();
                const bool begun = NACC == 2 ? mine > 0 : u > 0; // there is an O
                if (mine == 0) { // (an f32 q's row scale is there once all of Q is)
                    // (before this warp's arrival, or a group_sync)
                    if (r == 0 && !begun) ms->started[NACC == 2 ? w : 0] = 0;
#pragma unroll
                    for (int k = 0; k < PR; ++k) {
                        Row &y = rows[k];
                        const int rr = packed ? (lane >> 2) + 8 * k : local;
                        float scale = row_scale;
                        if (packed) scale = __shfl_sync(0xffffffffu, row_scale, rr);
                        if constexpr (NACC == 2 && !C::BF) {
                            if (p.q_f32) scale = ms->of.row_scale[items & 1][y.real ? rr : 0];
                        }
                        scale *= p.scale;
                        y.sc.mult = scale * kLog2e;
                        y.sc.turn = p.softcap == 0.f ? 0.f : scale / p.softcap;
                    }
                }

                // does every row see all columns?
                bool full = t0 + T <= it.end;
                if (!of_all<C>(it)) {
                    const int o0 = max(q0, 0), o1 = it.S - 1;
                    full = full && t0 >= start &&
                           (t0 + T <= keep1 ||
                            (t0 + T - 1 <= o0 && (!window || t0 > o1 - window)));
                }
                // otherwise a row sees columns [k0, k1) and [x0, x1)
                const int k0 = max(start - t0, 0), k1 = min(keep1 - t0, T);
                auto x0_of = [&](const Row &y) { return of_all<C>(it) ? 0 : max(y.x_lo - t0, 0); };
                auto x1_of = [&](const Row &y) {
                    return min((of_all<C>(it) ? it.end : y.x_hi) - t0, T);
                };
                auto k1_of = [&](const Row &y) { return y.x_hi > 0 && !of_all<C>(it) ? k1 : 0; };
                // y of N scores of a row (c: their first columns less each one's own)
                auto transform = [&](const Row &y, float *x, auto count, auto &&col) {
                    constexpr int N = decltype(count)::value;
                    if (!C::CAP && (!C::ANY || p.softcap == 0.f)) {
                        const float2 k = make_float2(y.sc.mult, y.sc.mult);
#pragma unroll
                        for (int i = 0; i < N; i += 2) {
                            const float2 z = __fmul2_rn(make_float2(x[i], x[i + 1]), k);
                            x[i] = z.x;
                            x[i + 1] = z.y;
                        }
                    } else {
                        const float2 turn = make_float2(y.sc.turn, y.sc.turn);
                        float most = 0.f;
#pragma unroll
                        for (int i = 0; i < N; i += 2) {
                            const float2 z = __fmul2_rn(make_float2(x[i], x[i + 1]), turn);
                            x[i] = z.x;
                            x[i + 1] = z.y;
                            most = fmaxf(most, fmaxf(fabsf(z.x), fabsf(z.y)));
                        }
                        if (__all_sync(0xffffffffu, most < kNearCap || !y.real)) { // (NaN: stays NaN)
#pragma unroll
                            for (int i = 0; i < N; i += 2) {
                                const float2 z = capped_near(make_float2(x[i], x[i + 1]), y.sc.cap);
                                x[i] = z.x;
                                x[i + 1] = z.y;
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < N; ++i) x[i] = capped(x[i], y.sc.cap);
                        }
                    }
                    if (C::BIAS || (C::ANY && p.slopes)) {
                        const float d = (float)(y.pos - t0 - col(0));
#pragma unroll
                        for (int i = 0; i < N; ++i)
                            x[i] = fmaf(-y.sc.slope, fabsf(d - (float)(col(i) - col(0))), x[i]);
                    }
                };
                const float2 minus = make_float2(-1.f, -1.f);
                bool moves = false;
                float alpha = 1.f; // of this lane's row
                // where a row's reference goes when its largest score of the tile is tm: it moves
                // when a weight would pass 2^LIM
                auto refer = [&](Row &y, float tm) {
                    const bool on = y.real && tm > y.m + C::LIM;
                    moves = moves || on;
                    const float to_m = on ? tm - C::OFF : y.m;
                    const float f = on && y.m != -INFINITY ? ex2(y.m - to_m) : 1.f;
                    y.l *= f;
                    y.m = to_m;
                    return f;
                };
                // one accumulator: a lane's reference is its last unit's, of the other warpgroup
                auto take_refs = [&]() { return take(u - 1); };
                auto pass_refs = [&]() {
                    if constexpr (NACC == 1) {
#pragma unroll
                        for (int k = 0; k < PR; ++k)
                            if (!packed || (lane & 3) == 0) ms->of.ref[state_at(k)] = rows[k].m;
                        arrive(SB_REF + w);
                    }
                };
                const bool adds = packed && p.q_f32; // a score is the sum of its terms'
                const bool modified = adds || C::XF || !full, one = shares == 4;
                const bool back = modified && (!one || !full);
                // packed: G columns of a warp at a time, 2 of every 8 a thread
                constexpr int NG = T / 32, G = 8 * NG;
                constexpr bool ROWS = T == 64; // weights of whole rows at once (registers)
                float pk[PR][2 * NG];
                auto load_packed = [&](int c, bool sums) {
                    float v[4 * NG], v2[4 * NG];
                    tmem_ld_rows<NG>(ts + c, v);
                    if (sums) tmem_ld_rows<NG>(ts + (16u << 16) + c, v2);
                    tmem_wait_ld();
#pragma unroll
                    for (int g = 0; g < NG; ++g)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float y = v[4 * g + e];
                            if (sums) y += v2[4 * g + e] + (TP == 3 ? v[4 * g + 2 + e] : 0.f);
                            pk[0][2 * g + e] = y;
                            if (PR == 2)
                                pk[PR - 1][2 * g + e] =
                                    v[4 * g + 2 + e] + (sums ? v2[4 * g + 2 + e] : 0.f);
                        }
                };
                // unpacked: 32 columns of this lane's row, or 16
                const bool wide = T == 128 || cols > 16; // 32 at a time
                float x[32];
                auto load = [&](int c) {
                    if (wide) tmem_ld32(ts + c, x);
                    else tmem_ld16(ts + c, x);
                    tmem_wait_ld();
                };
                // f(16 of x, their first column, which half)
                auto halves = [&](int c, auto &&f) {
                    f(x, c, std::integral_constant<int, 0>());
                    if (wide) f(x + 16, c + 16, std::integral_constant<int, 1>());
                };
                if (packed && busy) {
                    float tm[PR];
#pragma unroll
                    for (int k = 0; k < PR; ++k) tm[k] = -INFINITY;
#pragma unroll 1
                    for (int c = cb; c < cb + cols; c += G) {
                        load_packed(c, adds);
                        const int c2 = c + 2 * (lane & 3);
#pragma unroll
                        for (int k = 0; k < PR; ++k) {
                            if (k == 1 && it.rows <= 8) continue;
                            if (C::XF || !full) {
                                transform(rows[k], pk[k], std::integral_constant<int, 2 * NG>(),
                                          [&](int i) { return c2 + 8 * (i >> 1) + (i & 1); });
                                if (__builtin_expect(!full, 0)) {
                                    const uint32_t see =
                                        range32(x0_of(rows[k]) - c, x1_of(rows[k]) - c) |
                                        range32(k0 - c, k1_of(rows[k]) - c);
#pragma unroll
                                    for (int i = 0; i < 2 * NG; ++i)
                                        if (!((see >> (c2 - c + 8 * (i >> 1) + (i & 1))) & 1u))
                                            pk[k][i] = -INFINITY;
                                }
                            }
#pragma unroll
                            for (int i = 0; i < 2 * NG; ++i) tm[k] = fmaxf(tm[k], pk[k][i]);
                        }
                        if (back) {
                            float v[4 * NG];
#pragma unroll
                            for (int i = 0; i < 4 * NG; ++i)
                                v[i] = pk[PR == 2 && (i & 2) ? 1 : 0][(i >> 2) * 2 + (i & 1)];
                            tmem_st_rows<NG>(ts + c, v);
                        }
                    }
                    if (back) tmem_wait_st();
                    if (!take_refs()) return false;
                    float f[PR];
#pragma unroll
                    for (int k = 0; k < PR; ++k) {
                        float y = tm[k];
                        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 1));
                        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 2));
                        if (!C::XF && full) y *= rows[k].sc.mult;
                        f[k] = refer(rows[k], y);
                    }
                    pass_refs();
                    if (__any_sync(0xffffffffu, moves)) {
                        moves = true;
                        alpha = of_lane(f[0], f[PR - 1]);
                    }
                } else if (busy) {
                    const bool back32 = modified && (cols > 32 || !full);
                    float tm = -INFINITY;
#pragma unroll 1
                    for (int c = cb; c < cb + cols; c += 32) {
                        load(c);
                        if (C::XF || !full) {
                            // y, -infinity where the row sees nothing
                            const uint32_t see =
                                full ? 0u
                                     : range32(x0_of(rows[0]) - c, x1_of(rows[0]) - c) |
                                           range32(k0 - c, k1_of(rows[0]) - c);
                            halves(c, [&](float *y, int e, auto) {
                                transform(rows[0], y, std::integral_constant<int, 16>(),
                                          [&](int i) { return e + i; });
                                if (__builtin_expect(!full, 0)) {
#pragma unroll
                                    for (int i = 0; i < 16; ++i)
                                        if (!((see >> (e - c + i)) & 1u)) y[i] = -INFINITY;
                                }
                            });
                        }
                        if (back32)
                            halves(c, [&](float *y, int e, auto) { tmem_st16(ts + e, y); });
                        halves(c, [&](float *y, int, auto) {
                            float a = y[0], b2 = y[1];
#pragma unroll
                            for (int i = 2; i < 16; i += 2) {
                                a = fmaxf(a, y[i]);
                                b2 = fmaxf(b2, y[i + 1]);
                            }
                            tm = fmaxf(tm, fmaxf(a, b2));
                        });
                    }
                    if (back32) tmem_wait_st();
                    if (!C::XF && full) tm *= rows[0].sc.mult;
                    if (!take_refs()) return false;
                    alpha = refer(rows[0], tm);
                    pass_refs();
                    moves = __any_sync(0xffffffffu, moves);
                } else {
                    // (a warp without rows passes nothing on, but in turn)
                    if (!take_refs()) return false;
                    pass_refs();
                }
                const int before = NACC == 2 ? done : done + u; // units of the accumulator
                auto last_done = [&]() { // O holds all of them
                    if (!wait(SB_PVDONE + (NACC == 2 ? w : 0), (uint32_t)(before - 1) & 1u))
                        return false;
                    tc_fence_after();
                    return true;
                };
                if (__builtin_expect(moves, 0) && begun) { // (before, there is no O)
                    if (!last_done()) return false;
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        float o[32];
                        tmem_ld32(to + c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] *= alpha;
                        tmem_st16(to + c, o);
                        tmem_st16(to + c + 16, o + 16);
                    }
                    tmem_wait_st();
                }
                auto ref_of = [&](const Row &y) { return y.m == -INFINITY ? 0.f : y.m; };

                // A tile that not all rows see in full: V rows that no row sees may hold anything (0 * NaN
                // is NaN), and so may rows that some see, which are looked for where there are
                // several tokens; then this comes before the weights take the scores' place.
                auto clean_v = [&]() {
                    const int f = n + tile, nv = nst - nk, st = nk + f % nv;
                    if (!wait(SB_FULL + st, (uint32_t)(f / nv) & 1u)) return false;
                    const uint32_t vt = sb + p.q_bytes + st * C::SLOT;
                    const int o0 = max(q0, 0), o1 = it.S - 1;
                    const int ka = max(start - t0, 0), kb = min(keep1 - t0, T);
                    const int lo_any = max(window ? max(start, o0 - window + 1) : start, 0) - t0;
                    const int lo_all = max(window ? max(start, o1 - window + 1) : start, 0) - t0;
                    const int hi_any = it.S - t0, hi_all = o0 + 1 - t0;
                    // (boxes of a paged cache past the end read as zeros)
                    const int top = p.block_table
                                        ? min(T, (max(hi_any, 0) + p.box_rows - 1) / p.box_rows * p.box_rows)
                                        : T;
                    const int low = min(max(lo_all, 0), T), high = max(min(hi_all, hi_any), low);
                    auto kept = [&](int c) { return c >= ka && c < kb; };
                    auto any = [&](int c) { return kept(c) || (c >= lo_any && c < hi_any); };
                    auto all = [&](int c) { return kept(c) || (c >= lo_all && c < hi_all); };
                    const bool partial = p.q_len > 1;
                    uint32_t *bad = ms->bad[u & 1]; // (one warpgroup: its next unit's is another)
                    if (partial) {
                        if (r < 4) bad[r] = 0u;
                        if (!group_sync()) return false;
                    }
                    // rows 0 .. low - 1 and high .. top - 1, D / 8 units each
#pragma unroll 1
                    for (int i = r; i < (low + max(top - high, 0)) * (D / 8); i += 128) {
                        const int nth = i / (D / 8), j = i - nth * (D / 8);
                        const int c = nth < low ? nth : nth - low + high;
                        const uint32_t at = vt + (j >> 3) * CHUNK + swz(c, (j & 7) * 16);
                        if (!any(c)) {
                            sts_v4(at, 0u, 0u, 0u, 0u);
                        } else if (partial && !all(c)) {
                            const uint4 y = lds_v4(at);
                            const uint32_t e = C::BF ? 0x7f80u : 0x7c00u; // exponent of infinities, NaN
                            bool odd = false;
                            for (uint32_t z : {y.x, y.y, y.z, y.w})
                                odd = odd || (z & e) == e || ((z >> 16) & e) == e;
                            if (odd) atomicOr(bad + (c >> 5), 1u << (c & 31));
                        }
                    }
                    if (partial) {
                        if (!group_sync()) return false;
                        uint32_t word[4];
                        for (int i = 0; i < 4; ++i)
                            word[i] = *reinterpret_cast<volatile uint32_t *>(bad + i);
                        if (word[0] | word[1] | word[2] | word[3]) {
                            // (rare) such rows are added here, to the rows that see them, and
                            // leave the tile
                            if (begun) {
                                if (!last_done()) return false;
                            } else { // the accumulator starts here
                                // (the other warpgroup may still read the last item's from it)
                                if (!wait(SB_OFREE, (uint32_t)items & 1u)) return false;
                                tc_fence_after();
                                const float z[16] = {};
#pragma unroll 1
                                for (int c = 0; c < D; c += 16) tmem_st16(to + c, z);
                                tmem_wait_st();
                                ms->started[NACC == 2 ? w : 0] = 1;
                            }
                            const float ref = packed ? of_lane(ref_of(rows[0]), ref_of(rows[PR - 1]))
                                                     : ref_of(rows[0]);
                            const int k1r = dead ? 0 : k1, x1r = dead ? 0 : min(own + 1 - t0, T);
                            const int x0r =
                                max((window ? max(start, own - window + 1) : start) - t0, 0);
#pragma unroll 1
                            for (int c = 0; c < T; ++c) {
                                if (!((word[c >> 5] >> (c & 31)) & 1u)) continue;
                                const float y = tmem_ld1(ts + c);
                                const bool sees = !dead && part == 0 && c >= cb && c < cb + cols &&
                                                  ((c >= x0r && c < x1r) || (c >= k0 && c < k1r));
                                const float pr = ex2(y - ref);
#pragma unroll 1
                                for (int j = 0; j < D / 16; ++j) {
                                    float o[16];
                                    tmem_ld16(to + 16 * j, o);
                                    tmem_wait_ld();
                                    const uint32_t at = vt + (j >> 2) * CHUNK;
                                    const uint4 a = lds_v4(at + swz(c, (j & 3) * 32));
                                    const uint4 e = lds_v4(at + swz(c, (j & 3) * 32 + 16));
                                    const uint32_t v[8] = {a.x, a.y, a.z, a.w, e.x, e.y, e.z, e.w};
#pragma unroll
                                    for (int i = 0; i < 8; ++i) {
                                        const float2 z = Pair<DT>::unpack(v[i]);
                                        if (sees) {
                                            o[2 * i] = fmaf(pr, z.x, o[2 * i]);
                                            o[2 * i + 1] = fmaf(pr, z.y, o[2 * i + 1]);
                                        }
                                    }
                                    tmem_st16(to + 16 * j, o);
                                    tmem_wait_st();
                                }
                            }
                            if (!group_sync()) return false;
#pragma unroll 1
                            for (int i = r; i < T * (D / 8); i += 128) {
                                const int c = i / (D / 8), j = i - c * (D / 8);
                                if ((word[c >> 5] >> (c & 31)) & 1u)
                                    sts_v4(vt + (j >> 3) * CHUNK + swz(c, (j & 7) * 16), 0u, 0u, 0u, 0u);
                            }
                        }
                    }
                    fence_proxy_async_smem();
                    return true;
                };
                const bool edge = __builtin_expect(!full, 0) && !of_all<C>(it);
                if (edge && p.q_len > 1 && !clean_v()) return false;

                // ---- P: the weights, in terms, in the place of their scores. One term of 16
                // positions takes 8 columns: those of a lane's one term lie side by side, of several
                // 16 apart (16 k: the first term, 16 k + 8: the second, T + 8 k: the third)
                if (packed && busy) {
#pragma unroll 1
                    for (int c = cb; c < cb + cols; c += G) {
                        if (!one) load_packed(c, !modified && adds);
                        // pairs of G positions: first, second and third terms
                        uint32_t v[3][PR][NG];
#pragma unroll
                        for (int k = 0; k < PR; ++k) {
                            const float mult = C::XF || !full ? 1.f : rows[k].sc.mult;
                            const float2 mult2 = make_float2(mult, mult);
                            const float2 ref2 = make_float2(-ref_of(rows[k]), -ref_of(rows[k]));
#pragma unroll
                            for (int g = 0; g < NG; ++g) {
                                v[0][k][g] = v[1][k][g] = v[2][k][g] = 0u;
                                if (k == 1 && it.rows <= 8) continue;
                                const float2 e2 = __ffma2_rn(
                                    make_float2(pk[k][2 * g], pk[k][2 * g + 1]), mult2, ref2);
                                const float2 a = make_float2(ex2(e2.x), ex2(e2.y));
                                rows[k].l += a.x + a.y;
                                v[0][k][g] = Pair<DT>::pack(a.x, a.y);
                                const float2 z = __ffma2_rn(Pair<DT>::unpack(v[0][k][g]), minus, a);
                                v[1][k][g] = Pair<DT>::pack(z.x, z.y);
                                if (TP == 3) {
                                    const float2 y =
                                        __ffma2_rn(Pair<DT>::unpack(v[1][k][g]), minus, z);
                                    v[2][k][g] = Pair<DT>::pack(y.x, y.y);
                                }
                            }
                        }
                        // lanes 0 - 15 and 16 - 31: two terms of 16 rows, or three of 8 and none
                        if (ROWS && one) {
                            // whole rows: this share's weights, zeros for the others'
                            uint32_t lo[4 * T / 16], hi[4 * T / 16];
#pragma unroll
                            for (int q = 0; q < T / 8; ++q) {
                                const bool on = q / NG == share;
                                lo[2 * q] = on ? v[0][0][q % NG] : 0u;
                                lo[2 * q + 1] =
                                    on ? (TP == 2 ? v[0][PR - 1][q % NG] : v[1][0][q % NG]) : 0u;
                                hi[2 * q] = on ? (TP == 2 ? v[1][0][q % NG] : v[2][0][q % NG]) : 0u;
                                hi[2 * q + 1] = on && TP == 2 ? v[1][PR - 1][q % NG] : 0u;
                            }
                            tmem_st_pairs<T / 8>(ts, lo);
                            tmem_st_pairs<T / 8>(ts + (16u << 16), hi);
                        } else {
                            uint32_t lo[2 * NG], hi[2 * NG];
#pragma unroll
                            for (int g = 0; g < NG; ++g) {
                                lo[2 * g] = v[0][0][g];
                                lo[2 * g + 1] = TP == 2 ? v[0][PR - 1][g] : v[1][0][g];
                                hi[2 * g] = TP == 2 ? v[1][0][g] : v[2][0][g];
                                hi[2 * g + 1] = TP == 2 ? v[1][PR - 1][g] : 0u;
                            }
                            tmem_st_pairs<NG>(ts + c / 2, lo);
                            tmem_st_pairs<NG>(ts + (16u << 16) + c / 2, hi);
                        }
                    }
                } else if (busy) {
                    const float mult = C::XF || !full ? 1.f : rows[0].sc.mult, ref = ref_of(rows[0]);
                    float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    const float2 mult2 = make_float2(mult, mult), ref2 = make_float2(-ref, -ref);
#pragma unroll 1
                    for (int c = cb; c < cb + cols; c += 32) {
                        if (cols > 32) load(c);
                        uint32_t words[16];
                        halves(c, [&](float *y, int e, auto half) {
                            uint32_t v[16]; // first terms, second terms
#pragma unroll
                            for (int i = 0; i < 16; i += 2) {
                                const float2 e2 = __ffma2_rn(make_float2(y[i], y[i + 1]), mult2, ref2);
                                const float2 a = make_float2(ex2(e2.x), ex2(e2.y));
                                l2[i / 2 & 1] = __fadd2_rn(l2[i / 2 & 1], a);
                                v[i / 2] = Pair<DT>::pack(a.x, a.y);
                                const float2 z = __ffma2_rn(Pair<DT>::unpack(v[i / 2]), minus, a);
                                y[i] = z.x;
                                y[i + 1] = z.y;
                                v[8 + i / 2] = Pair<DT>::pack(z.x, z.y);
                            }
                            if (TP == 3) {
                                uint32_t third[8];
#pragma unroll
                                for (int i = 0; i < 16; i += 2) {
                                    const float2 z = Pair<DT>::unpack(v[8 + i / 2]);
                                    third[i / 2] = Pair<DT>::pack(y[i] - z.x, y[i + 1] - z.y);
                                }
                                tmem_st8w(ts + T + e / 2, third);
                            }
                            if (TP == 2 && one_p) {
                                uint32_t *to_w = words + 8 * half.value;
#pragma unroll
                                for (int i = 0; i < 8; ++i) to_w[i] = part == 1 ? v[8 + i] : v[i];
                            } else {
                                tmem_st16w(ts + e, v);
                            }
                        });
                        if (TP == 2 && one_p) {
                            if (wide) {
                                tmem_st16w(ts + c / 2, words);
                            } else {
                                tmem_st8w(ts + c / 2, words);
                            }
                        }
                    }
                    rows[0].l += (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y);
                }
                if (busy) {
                    if (shares > 1 && !(ROWS && packed && one)) { // zeros for the other shares' positions
                        const uint32_t z[16] = {};
                        const int half = one_p ? 2 : 1; // columns of TMEM to 16 positions: 8 or 16
#pragma unroll 1
                        for (int c = 0; c < T / half; c += 16) {
                            // (shares are 16 positions and more: 8 columns, or 16)
                            const bool lo = c * half < cb || c * half >= cb + cols;
                            const bool hi = (c + 8) * half < cb || (c + 8) * half >= cb + cols;
                            if (lo && hi) {
                                tmem_st16w(ts + c, z);
                            } else {
                                if (lo) tmem_st8w(ts + c, z);
                                if (hi) tmem_st8w(ts + c + 8, z);
                            }
                        }
                    }
                    tmem_wait_st();
                }
                if (edge && p.q_len == 1 && !clean_v()) return false;
                tc_fence_before();
                arrive(SB_PFULL + s);
                if (NACC == 2) ++done;
                ++mine;
            }

            if (!before_join()) return false;
            if (it.tiles == 0) return true;
            if constexpr (NACC == 1) {
                if (((nu - 1) & 1) != w && !take(nu - 1)) return false;
                done += nu;
                handed += w == 0 ? nu / 2 : (nu + 1) / 2;
            }
            if (packed) {
#pragma unroll
                for (int k = 0; k < PR; ++k) {
                    rows[k].l += __shfl_xor_sync(0xffffffffu, rows[k].l, 1);
                    rows[k].l += __shfl_xor_sync(0xffffffffu, rows[k].l, 2);
                }
            }

            // ---- epilogue: a row's states, of the warpgroups that took tiles in turn and of the
            // copies of its lane, are joined; each warpgroup writes half of the columns
            if (!wait(SB_OREADY, (uint32_t)items & 1u)) return false;
            tc_fence_after();
            const bool joint = nrt == 1;
            const int c0 = joint ? w * (D / 2) : 0, nc = joint ? D / 2 : D; // this thread's columns
            const bool few = copies > 1 && it.rows <= 16; // rows lane / 4 and lane / 4 + 8 here too
            float m = rows[0].m, l = rows[0].l;
            float f_acc[NACC][2]; // what the accumulators of this copy of the rows are multiplied by
#pragma unroll
            for (int x = 0; x < NACC; ++x) f_acc[x][0] = f_acc[x][1] = x == 0 || joint ? 1.f : 0.f;
            auto state = [&](int x, int at) { // of a warpgroup
                if constexpr (NACC == 2) return ms->of.state[x][at];
                else return make_float2(ms->of.ref[at], ms->of.sum[x][at]);
            };
            // (a sum that is no number takes part: only an empty state does not)
            auto join_states = [&](int first, int here, int k, float &mm, float &ll) {
                float2 y[8];
                mm = -INFINITY;
                ll = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    y[i] = make_float2(-INFINITY, 0.f);
                    if (i < shares * 2) y[i] = state(i & 1, first + (i >> 1) * span);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (y[i].y != 0.f) mm = fmaxf(mm, y[i].x);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (y[i].y != 0.f) ll += y[i].y * ex2(y[i].x - mm);
                const float2 s0 = state(0, here), s1 = state(1, here);
                if constexpr (NACC == 2) {
                    f_acc[0][k] = s0.y == 0.f ? 0.f : ex2(s0.x - mm);
                    f_acc[1][k] = s1.y == 0.f ? 0.f : ex2(s1.x - mm);
                } else {
                    f_acc[0][k] = s0.y == 0.f && s1.y == 0.f ? 0.f : ex2(s0.x - mm);
                }
            };
            if (joint) {
#pragma unroll
                for (int k = 0; k < PR; ++k) {
                    if (packed && (lane & 3)) continue;
                    if constexpr (NACC == 2)
                        ms->of.state[w][state_at(k)] = make_float2(rows[k].m, rows[k].l);
                    else
                        ms->of.sum[w][state_at(k)] = rows[k].l;
                }
                if (!all_sync()) return false;
                if (packed || few) {
                    float mm[2], ll[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int rr = (lane >> 2) + 8 * k;
                        const bool on = rr < it.rows;
                        join_states(on ? rr : 0, on ? (warp & 3) * 32 + rr : 0, k, mm[k], ll[k]);
                    }
                    m = of_lane(mm[0], mm[1]);
                    l = of_lane(ll[0], ll[1]);
                } else {
                    join_states(owner ? local : 0, r, 0, m, l);
                }
            }
            if (dead) l = 0.f;
            const bool odd = !(l - l == 0.f); // no number, or infinite
            const float factor = l == 0.f ? 0.f : odd ? NAN : p.whole ? 1.f / l : 1.f;
            const bool writes = owner && rep == 0 && part == 0;
            if (writes && !p.whole && (!joint || w == 0))
                p.ml[dst_row] = odd ? make_float2(-kNeutralM, 1.f) // outweighs every other partial
                                : l == 0.f ? make_float2(kNeutralM, 0.f) : make_float2(m * kLn2, l);
            // (an accumulator that no unit went to holds anything)
            auto times = [](float f, float x) { return f != 0.f ? f * x : 0.f; };
            // 16 columns of the lane, of all accumulators
            auto lane16 = [&](int c, float *o) {
                if (NACC == 2 && joint) {
                    float o2[16];
                    tmem_ld16(tl + c, o);
                    tmem_ld16(tl + D + c, o2);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        o[i] = times(f_acc[0][0], o[i]) + times(f_acc[NACC - 1][0], o2[i]);
                } else {
                    tmem_ld16(to + c, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] = times(f_acc[0][0], o[i]);
                }
            };
            if (copies == 1) {
#pragma unroll 1
                for (int c = c0; c < c0 + nc; c += 16) {
                    float o[16];
                    lane16(c, o);
                    if (writes && (p.whole || l != 0.f)) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = factor == 0.f ? 0.f : o[i] * factor;
#pragma unroll
                        for (int i = 0; i < 16; i += 4)
                            write4(dst_row, c + i, make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]));
                    }
                }
            } else {
                // the copies' sums meet in shared memory: [warpgroup][copy][row][W columns], as many
                // columns at once as there is room for
                const int rows4 = (it.rows + 3) / 4 * 4;
                int W = nc;
                // (a CTA's last item finds the ring empty)
                const int room = it.last ? nst * C::SLOT : p.join_bytes - kScoredRowBytes;
                const int lanes = few ? reps : copies; // (those of a row's terms are added here)
                while (2 * lanes * rows4 * W * 4 > room) W >>= 1;
                const int w4 = W / 4, lw = 31 - __clz(w4);
                uint8_t *place = sm + p.q_bytes + nst * C::SLOT;
                auto *jr = reinterpret_cast<JoinRows *>(place);
                if (writes && w == 0) {
                    jr->factor[local] = factor;
                    jr->to[local] = (uint32_t)dst_row;
                }
                float *xs = reinterpret_cast<float *>(it.last ? sm + p.q_bytes : place + kScoredRowBytes) +
                            w * lanes * rows4 * W;
                // units of 8 columns (few rows), of 4 otherwise, swizzled so that lanes hit other banks
                const int mask8 = W / 8 - 1;
#pragma unroll 1
                for (int at = 0; at < nc; at += W) {
                    if (few && busy) {
                        // rows lane / 4 and lane / 4 + 8, two of every 8 columns, 32 columns at a time
#pragma unroll 1
                        for (int c = 0; c < W; c += 32) {
                            float o[NACC][16], o2[NACC][16];
#pragma unroll
                            for (int x = 0; x < NACC; ++x) {
                                tmem_ld_rows<4>(tl + x * D + c0 + at + c, o[x]);
                                if (packed) tmem_ld_rows<4>(tl + (16u << 16) + x * D + c0 + at + c, o2[x]);
                            }
                            tmem_wait_ld();
#pragma unroll
                            for (int k = 0; k < (packed ? PR : 2); ++k) {
                                const int rr = (lane >> 2) + 8 * k;
                                if (rr >= it.rows) continue;
                                float *to_row = xs + (rep * rows4 + rr) * W;
#pragma unroll
                                for (int g = 0; g < 4; ++g) {
                                    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                                    for (int x = 0; x < NACC; ++x) {
                                        const int i = 4 * g + 2 * k;
                                        float a = o[x][i], b2 = o[x][i + 1];
                                        if (packed) {
                                            a += o2[x][i];
                                            b2 += o2[x][i + 1];
                                        }
                                        if (packed && TP == 3) {
                                            a += o[x][4 * g + 2];
                                            b2 += o[x][4 * g + 3];
                                        }
                                        sum.x += times(f_acc[x][k], a);
                                        sum.y += times(f_acc[x][k], b2);
                                    }
                                    const int u8 = (c / 8 + g) ^ (rr & mask8);
                                    *reinterpret_cast<float2 *>(to_row + u8 * 8 + 2 * (lane & 3)) = sum;
                                }
                            }
                        }
                    } else if (busy) {
                        float4 *to_row = reinterpret_cast<float4 *>(xs) + (rep * rows4 + local) * w4;
#pragma unroll 1
                        for (int c = 0; c < W; c += 16) {
                            float o[16];
                            lane16(c0 + at + c, o);
                            if (owner) {
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    to_row[(c / 4 + i) ^ (local & 3)] = make_float4(
                                        o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                            }
                        }
                    }
                    if (!(at == 0 ? all_sync() : group_sync())) return false;
                    // w4 threads to a row
                    const int c = r & (w4 - 1);
#pragma unroll 1
                    for (int rr = r >> lw; rr < it.rows; rr += 128 >> lw) {
                        const float fac = jr->factor[rr];
                        if (fac == 0.f && !p.whole) continue;
                        const int at4 = few ? c ^ ((rr & mask8) << 1) : c ^ (rr & 3);
                        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                        for (int k = 0; k < lanes; ++k) {
                            const float4 y = reinterpret_cast<const float4 *>(xs)[(k * rows4 + rr) * w4 + at4];
                            sum.x += y.x;
                            sum.y += y.y;
                            sum.z += y.z;
                            sum.w += y.w;
                        }
                        sum = fac == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                                         : make_float4(sum.x * fac, sum.y * fac, sum.z * fac, sum.w * fac);
                        write4((size_t)jr->to[rr], c0 + at + 4 * c, sum);
                    }
                    if (at + W < nc && !group_sync()) return false;
                }
                // (the place, and the states, are written again behind the next item's exchange)
            }
            // (one accumulator: the next item's first unit passes references on)
            if (NACC == 1 && copies == 1 && !all_sync()) return false;
            tc_fence_before();
            arrive(SB_OFREE);
            n += it.tiles;
            ++items;
            return true;
        };
        // The next item with tiles (or the end), its Q on the way; those without are dealt with.
        auto next_item = [&](Item &it, int nth, float &row_scale) {
            for (;;) {
                const int q = taken & 1;
                if (!wait(SB_ITEM + q, (uint32_t)(taken >> 1) & 1u)) return false;
                it = ms->item[q];
                arrive(SB_TAKEN + q);
                ++taken;
                if (it.tiles < 0) return true;
                if (it.tiles > 0) return load_q(it, nth, row_scale);
                neutral(it);
            }
        };
        Item it = {};   // (before the first: an item without tiles, of one row)
        it.rows = 1;
        float row_scale = 1.f;
#pragma unroll 1
        while (it.tiles >= 0) {
            // the next item's Q goes out before this one's epilogue, so that its first scores are
            // there when the epilogue is done
            Item then;
            float then_scale = 1.f;
            if (!work(it, row_scale, [&]() {
                    return next_item(then, items + (it.tiles > 0 ? 1 : 0), then_scale);
                }))
                break;
            it = then;
            row_scale = then_scale;
        }
        if (!ok && lane == 0) timed_out();
    } else {
        setmaxnreg_dec<C::OTHER_REGS>();
    }

    // ---------------------------------- teardown ----------------------------------
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == C::MMA_WARP) tmem_dealloc(tmem, 512);
}

template <typename C>
cudaError_t launch(int grid, int smem, cudaStream_t st, const CUtensorMap &km, const CUtensorMap &vm,
                   const ScoredParams &p)
{
    auto *fn = gqa_scored_kernel<C>;
    // (the same limit in every call, whatever this one needs: another host thread's call that sets a
    // lower one in between would have the launch refused)
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kScoredSmemMax);
    if (e != cudaSuccess) return e;
    fn<<<grid, C::THREADS, smem, st>>>(km, vm, p);
    return cudaGetLastError();
}

template <typename DT, int D, int TP, int KIND>
cudaError_t launch_x(int grid, int smem, cudaStream_t st, const CUtensorMap &km, const CUtensorMap &vm,
                     const ScoredParams &p)
{
    const bool cap = p.softcap != 0.f;
    if (!(p.scale > 0.f) || (cap && p.slopes))
        return launch<Cfg<DT, D, TP, kAny, KIND>>(grid, smem, st, km, vm, p);
    return cap        ? launch<Cfg<DT, D, TP, kCap, KIND>>(grid, smem, st, km, vm, p)
           : p.slopes ? launch<Cfg<DT, D, TP, kBias, KIND>>(grid, smem, st, km, vm, p)
                      : launch<Cfg<DT, D, TP, kNone, KIND>>(grid, smem, st, km, vm, p);
}

} // namespace

template <typename DT, int D, int TP>
static cudaError_t launch_kind(int grid, int smem, cudaStream_t st, const CUtensorMap &km,
                               const CUtensorMap &vm, const ScoredParams &p)
{
    return p.kind == kScoredPacked ? launch_x<DT, D, TP, kScoredPacked>(grid, smem, st, km, vm, p)
           : p.kind == kScoredOwn  ? launch_x<DT, D, TP, kScoredOwn>(grid, smem, st, km, vm, p)
                                   : launch_x<DT, D, TP, kScoredShared>(grid, smem, st, km, vm, p);
}

} // namespace skv
