// GQA / MQA split kernel over an 8-bit paged cache, tcgen05 tensor cores, sm_103a.
//
// A page (block i of block_size positions) holds e4m3 or e5m2 codes Kc, Vc that
// stand for code * scale[i][head]. With page scales ks, vs (lv = log2 vs) and
// scores in log2 units,
//     s[r][pos]  = ks[page] * sum_d q[r][d] Kc[pos][d]        (q times scale * log2 e)
//     x[r][pos]  = 2^(s - m[r]) * vs[page] / V,  m[r] about the largest s + lv - log2 V
//     acc[r][d]  = sum_pos x[r][pos] Vc[pos][d],   l[r] = sum_pos 2^(s - m[r])
// so the value scales fold into the weights and the codes go to the tensor cores
// as they stand: TMA brings 128-position tiles of K and of V into shared memory
// in the 128-byte swizzle the MMA reads, and nothing converts or re-reads them.
//     S[pos][(j, r)]  = sum_d Kc[pos][d] q_j[r][d]      (M = 128 positions, K = D)
//     O^T[d][(j, r)] += sum_pos Vc[pos][d] x_j[r][pos]  (M = 128 value columns, K = 128)
// V is about the largest value scale of the item so far, a power of two: with it l stays
// near 1 whatever the scales are (pages of zeros have 2^-100, others up to 2^120), and
// neither l nor x leaves the range of an f32. References and V are even powers of two, so
// that moving them multiplies by an exact power, in two halves where one would underflow.
//
// The other operand of an 8-bit MMA is 8-bit too. q and x are split into e4m3 terms,
// y = y_0 + 2^-5 y_1 + 2^-10 y_2 + ...: a term rounds what the ones before it left, and
// each takes 5 bits off (4 significant bits and the sign of the rest). f32 outputs take
// five terms of both, 25 bits: four of both left an error of 0.4 to 1.4e-6 there, as much as
// or more than f32 arithmetic does. 16-bit outputs take four of both, 20 bits.
// y is at most 256, and e4m3's least step, 2^-9, is 2^-24 or 2^-29 in the last term: half of
// that is what a term of any size may be off by. Of q that is 2^-32 of the row's largest.
// Weights differ by far more, and a small one can be one of many whose values are all there
// is to sum (one position that holds the probability, with values near zero). So m follows
// the largest weight of the tile both ways: it is 2^2 to 2^4 when it sets m, and when a
// row's is above 2^8 or below 2^-10 (five terms: 2^-8) in a whole tile, m moves and l and
// O^T are rescaled. What is off by half a step is then at most 2^-15 (2^-22) of the largest
// weight of its tile. A fixed m lost 3.6% of 65536 equal positions beside one of 99.7% with
// values of zero, and with three terms (x of wide items) all of 16384.
// The terms are columns of the MMA (N = terms x rows, rounded to 16), whose time for N <= 64
// is that of reading the tile (46 to 48 cycles per 32-byte step); they are added in f32 when S
// or O^T leave TMEM. The products are exact and the sums f32 (measured: relative error 1e-7
// on full-range codes).
//
// An item is (sequence, KV head, split, row group), rows (query token, head). Roles, one
// CTA per SM:
//   softmax warpgroups (1 to 4, up to 8 rows each; for 5 to 16 rows of 128 two sets of them
//              take tiles in turn): a thread owns one position of the tile (TMEM lane); the
//              references stay for most tiles, which take one vote. In the epilogue a thread
//              owns a value column.
//   two warps  TMA producers, K and V tiles through one ring of slots, paged boxes as in the
//              16-bit tensor-core kernel.
//   two warps  MMA issue, one thread each for the scores and for the values.
//   one warp   the page scales of four tiles at a time (beside three or four softmax
//              warpgroups the K producer does it, looking them up two batches ahead).
// Where every sequence has one split there is nothing to merge: the epilogue divides by l
// and writes the output itself, and no combine follows (256 sequences of 40 positions, 32/8
// heads of 128: 41 us instead of 60; 128 of 100, 32 heads of 256 over one: 14 instead of 34).
// Every wait is bounded; a wait that runs out sets the status word and the CTA drains
// and returns.
#include <climits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "gqa_split.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace skv {
namespace {

constexpr int T = kQ8Tile;
constexpr float kTermStep = 1.f / 32.f;
// m is this much, or up to 2 more, below the maximum that set it: higher maxima then seldom
// move it again (24 rows of 256, batch of 4: 85.5 us; 4: 89; ragged 32: 661 and 665)
constexpr float kHead = 2.f;
constexpr float kTau = 8.f;  // and moves when a score is this much above it,
                             // or a tile's largest kLow below it
constexpr float kDeep = 64.f; // but not further below its highest than this: l and O^T keep
                              // the weights of before, times 2^64 at most
constexpr float kWide = 16.f; // log2 V moves when a page's is this much above it
constexpr float kLeast = -32.f; // and pages further below it count as this far in a reference:
                                // 2^(s - m) stays below 2^(8 + 32)
constexpr int kMaxSlots = 12;
constexpr float kMinScale = 7.8886090522101181e-31f; // 2^-100

// barriers
constexpr int B_FULL = 0, B_EMPTY = kMaxSlots, B_SFULL = 2 * kMaxSlots, B_SFREE = B_SFULL + 2,
              B_PFULL = B_SFREE + 2, B_PFREE = B_PFULL + 2, B_PVDONE = B_PFREE + 2,
              B_OREADY = B_PVDONE + 2, B_OFREE = B_OREADY + 1, B_MFULL = B_OFREE + 1,
              B_QFULL = B_MFULL + 1, B_QFREE = B_QFULL + 1, B_SCFULL = B_QFREE + 1,
              B_SCFREE = B_SCFULL + 2, B_QKDRAIN = B_SCFREE + 2, B_PVDRAIN = B_QKDRAIN + 1,
              B_N = B_PVDRAIN + 1;

// Shape and shared memory of <D, RP, QT, PT>: RP rows an item at most, QT terms of q, PT of x. A
// softmax warpgroup takes RPW rows of every tile, 8, or 4 where that is enough: a
// thread's share of a tile must not outlast the tile's time on the memory side, and 32
// rows in one thread took 5200 cycles against 2800. Smaller shares repeat more of a tile's
// fixed part: 8 rows of 128 as 2 x 4 in one set take 60.1 us instead of 56.9 (1.2M positions,
// bf16), 16 as 4 x 4 69.4 instead of 68.4 as 2 x 8; 8 rows of 256, whose tiles take twice the
// time, 54.3 as 2 x 4 and 58.3 as one 8.
template <int D, int RP, int QT, int PT> struct Layout {
    static constexpr int N = (QT * RP + 15) / 16 * 16;  // columns of S
    static constexpr int NP = (PT * RP + 15) / 16 * 16; // columns of O^T
    static constexpr int W = RP > 8 ? RP / 8 : RP == 8 && D == 256 ? 2 : 1; // per tile
    static constexpr int RPW = RP / W;
    // 5 to 16 rows of 128 columns: two sets of warpgroups take turns, each with its own
    // references and its own O^T, joined at the item's end. There a tile's waits, vote, terms
    // and fences add up to 1800 cycles and more, the memory side's share to 1400 (1.2M
    // positions, bf16: 8 rows 59.9 us with one set, 56.9 with two; 16 rows 68.4 and 66.6, with
    // f32 outputs 71.9 and 69.1; 4 rows 53.9 with either, but 256 sequences of 40 positions 41.0
    // and 44.4; 24 rows would be 28 warps; 256 columns have twice the time).
    static constexpr int X = D == 128 && (RP == 8 || RP == 16) ? 2 : 1;
    static constexpr int WT = W * X; // softmax warpgroups
    // Warps after the softmax warps. Beside three or four warpgroups the K producer fetches
    // the page scales too: a warp less, a thread has 128 registers and not 96, or 96 and not
    // 80, with which the tile loop spilled.
    static constexpr bool KSCALE = WT >= 3;
    static constexpr int KPROD = 4 * WT, VPROD = KPROD + 1, QK = KPROD + 2, PV = KPROD + 3,
                         SCALE = KSCALE ? -1 : KPROD + 4;
    static constexpr int THREADS = 32 * (KPROD + (KSCALE ? 4 : 5));
    // weights as [row term][position] (K-major), or for wide items [position][row term]
    // (MN-major, rows of 128 bytes): there a thread stores 8 bytes at a time
    static constexpr bool PMN = RP >= 16 || D == 128;
    static constexpr int NCH = D / 128;        // 128-column chunks of a row
    static constexpr int CHUNK = T * 128;      // bytes of a chunk of a tile
    static constexpr int SLOT = NCH * CHUNK;   // a K or V tile
    static constexpr int QCH = N * 128;        // a chunk of Q
    static constexpr int PSLOT = PMN ? T * 128 : NP * 128; // one P buffer
    static constexpr int Q_OFF = 0;
    static constexpr int P_OFF = Q_OFF + NCH * QCH;
    static constexpr int SLOT_OFF = (P_OFF + 2 * PSLOT + 1023) / 1024 * 1024;
    // after the slots: barriers, flags, page scales (2 batches of 4 tiles of 8 groups of
    // 16 positions), per-row tables (of two items), warp maxima, sums, references and log2 V
    // (of two items), flags, columns with a NaN (of two items)
    static constexpr int BAR = 0, MISC = BAR + B_N * 8, SC = (MISC + 16 + 15) / 16 * 16,
                         ROW = SC + 2 * 4 * 8 * 16,
                         RED = ROW + 2 * 3 * RP * 4, SUM = RED + 4 * RP * X * 4,
                         REF = SUM + 2 * 4 * RP * X * 4, LGV = REF + 2 * RP * X * 4,
                         BAD = LGV + 2 * X * 4,
                         NANC = BAD + 2 * WT * 4,
                         TAIL = NANC + 2 * D * 4;
    static constexpr int SLOTS_FIT = (232448 - 1024 - SLOT_OFF - TAIL) / SLOT;
    // even: K tiles then use the even slots and V tiles the odd ones, so the two producers
    // never wait for each other's slots (a barrier's parity tells one phase back, not two)
    static constexpr int NS = (SLOTS_FIT > kMaxSlots ? kMaxSlots : SLOTS_FIT) / 2 * 2;
    static constexpr int TAIL_OFF = SLOT_OFF + NS * SLOT;
    static constexpr int BYTES = TAIL_OFF + TAIL + 1024;
    static_assert(NS >= 4 && NS % 2 == 0, "K and V tiles of two steps in flight");
    static_assert(2 * N + X * NCH * NP <= 512, "TMEM columns: two S slots and O^T");
    static_assert(QCH % 1024 == 0 && BYTES <= 232448, "swizzle atoms, shared memory");
    static_assert(!PMN || NP <= 128, "a position's weights in one row of the swizzle");
};

// byte offset of (row, byte) in a region of 128-byte rows with the 128-byte swizzle
__device__ __forceinline__ uint32_t swz(uint32_t row, uint32_t byte)
{
    return (row >> 3) * 1024 + (row & 7) * 128 + ((((byte >> 4) ^ row) & 7) << 4) + (byte & 15);
}

__device__ __forceinline__ void sts_u8(uint32_t saddr, uint32_t v)
{
    asm volatile("st.shared.u8 [%0], %1;" ::"r"(saddr), "r"(v) : "memory");
}
__device__ __forceinline__ void sts_u32(uint32_t saddr, uint32_t v)
{
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(saddr), "r"(v) : "memory");
}

// D[128][N] (+)= A . B, 8-bit operands, K = 32
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
                 : "memory");
}

// f32 accumulation; A e4m3 or e5m2, B e4m3, each K-major or (a_mn, b_mn) MN-major
__device__ __forceinline__ uint32_t idesc_f8(int n, bool a_mn, bool b_mn, bool a_e5m2)
{
    return (1u << 4) | ((a_e5m2 ? 1u : 0u) << 7) | ((a_mn ? 1u : 0u) << 15) |
           ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

// C consecutive 32-bit TMEM columns of this warp's lane quarter
template <int C> __device__ __forceinline__ void tmem_ld(uint32_t taddr, float *v)
{
    static_assert(C == 4 || C == 8, "four or eight columns");
    uint32_t r[C];
    if constexpr (C == 4)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(taddr));
    else
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                       "=r"(r[6]), "=r"(r[7])
                     : "r"(taddr));
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_st4(uint32_t taddr, const float *v)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr),
                 "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])),
                 "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3]))
                 : "memory");
}

// two values of at most 256 to e4m3 (x in the low byte); *x, *y: what is left, times 32 (at
// most 256 again: a code is within 2^3 of a value below 2^8)
__device__ __forceinline__ uint32_t term2(float &x, float &y)
{
    const __nv_fp8x2_storage_t c =
        __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
    const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(c, __NV_E4M3)));
    x = (x - f.x) * 32.f;
    y = (y - f.y) * 32.f;
    return c;
}

// The PT terms of two values, x in the low byte of each. What is left after all but two
// fits an f16 (11 bits for 10), so the last two are taken two values at a time.
template <int PT> __device__ __forceinline__ void terms(float x, float y, uint32_t *c)
{
#pragma unroll
    for (int j = 0; j < PT - 2; ++j) c[j] = term2(x, y);
    const __half2 h = __floats2half2_rn(x, y);
    c[PT - 2] = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(h), __NV_SATFINITE, __NV_E4M3);
    const __half2 f(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)c[PT - 2], __NV_E4M3));
    const __half2 rest = __hmul2(__hsub2(h, f), __half2(__half(32.f), __half(32.f)));
    c[PT - 1] = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(rest), __NV_SATFINITE, __NV_E4M3);
}

// how many of a barrier's threads have pred
__device__ __forceinline__ int named_bar_count(int id, int threads, bool pred)
{
    int n;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %3, 0;\n\t"
                 "barrier.cta.red.popc.aligned.u32 %0, %1, %2, p;\n\t}"
                 : "=r"(n)
                 : "r"(id), "r"(threads), "r"((int)pred)
                 : "memory");
    return n;
}

// 2^k, k in [-126, 127]
__device__ __forceinline__ float pow2(int k) { return __int_as_float((k + 127) << 23); }

// the length the items of entry e, sequence b, attend over: the plan's, or the device's,
// kept within [0, the plan's]
__device__ __forceinline__ int len8(const SplitParams &p, int e, int b)
{
    const int L = p.items.seq_lens[e];
    return p.dev_lens ? max(0, min(p.dev_lens[b], L)) : L;
}

// one output element, in the output's type
__device__ __forceinline__ void put_out(const FusedOut &f, size_t i, float v)
{
    switch (f.out_dtype) {
    case DA_F32: static_cast<float *>(f.out)[i] = v; break;
    case DA_F16: static_cast<__half *>(f.out)[i] = __float2half_rn(v); break;
    default: static_cast<__nv_bfloat16 *>(f.out)[i] = __float2bfloat16_rn(v); break;
    }
}

// item k of this CTA
__device__ __forceinline__ int64_t item8(int k)
{
    return (int64_t)k * gridDim.x + ((k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

// The (item, tile) sequence of a CTA, the same for every role: its items in turn, each in
// tiles of T positions, the last one cut at the item's end; items without positions have
// no tiles and are skipped.
struct Walk8 {
    int k, b, kvh, s, rg, p0, p1, t0, t1, gt, L;
    bool done, first;
    __device__ __forceinline__ void load_item(const SplitParams &p, const Order8 &od)
    {
        for (;; ++k) {
            const int64_t item = item8(k);
            // in a round that is not full the CTAs at its end have none
            done = item >= p.items.n_items;
            if (done) return;
            int e;
            decode_item(p.items, (int)item, e, kvh, s, rg);
            b = od.seq[e];
            p0 = s * p.items.chunk[e];
            L = len8(p, e, b);
            p1 = min(L, p0 + p.items.chunk[e]);
            if (p1 > p0) break;
        }
        t0 = p0;
        t1 = tile_end<T>(t0, p1);
        first = true;
    }
    __device__ __forceinline__ void start(const SplitParams &p, const Order8 &od)
    {
        k = 0;
        gt = 0;
        load_item(p, od);
    }
    __device__ __forceinline__ bool last() const { return t1 >= p1; }
    __device__ __forceinline__ void next(const SplitParams &p, const Order8 &od)
    {
        ++gt;
        if (t1 >= p1) {
            ++k;
            load_item(p, od);
        } else {
            t0 = t1;
            t1 = tile_end<T>(t0, p1);
            first = false;
        }
    }
};

template <int D, int RP, int QT, int PT>
__global__ void __launch_bounds__((Layout<D, RP, QT, PT>::THREADS), 1)
    gqa_8bit_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                    const __grid_constant__ Scales8 sc, const __grid_constant__ Order8 od,
                    const __grid_constant__ SplitParams p,
                    const int e5m2)
{
    using L = Layout<D, RP, QT, PT>;
    constexpr int N = L::N, NP = L::NP, NCH = L::NCH, NS = L::NS, W = L::W, RPW = L::RPW,
                  X = L::X, WT = L::WT;
    // a tile's largest weight is 2^-kLow at least, half a step of the terms 2^-30 or 2^-25
    constexpr float kLow = PT == 5 ? 8.f : 10.f;
    constexpr int RC = 4; // rows taken from TMEM at a time
    // and of the scores: 8 at a time save a round trip where they fit the registers (16 rows of
    // 128, 1.2M positions, f32: 73.5 -> 71.9 us; 24 rows 83.4 -> 87.0, 32 bf16 93.6 -> 98.4)
    constexpr int SC = RP == 16 ? RPW : RC;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(sm);
    uint8_t *tail = sm + L::TAIL_OFF;
    uint64_t *bar = reinterpret_cast<uint64_t *>(tail + L::BAR);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(tail + L::MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tail + L::MISC + 4);
    // of 16 positions: (ks, log2 vs, vs, the largest log2 vs of the tile rounded down to even)
    float4 *sc_sm = reinterpret_cast<float4 *>(tail + L::SC);
    // per row, of items in turn: 1 / (q's scaling), positions seen (below lim), workspace row
    float *const qf2 = reinterpret_cast<float *>(tail + L::ROW);
    int *const lim2 = reinterpret_cast<int *>(qf2 + 2 * RP), *const wrow2 = lim2 + 2 * RP;
    float *red_sm = reinterpret_cast<float *>(tail + L::RED); // maxima, [4 WT warps][RPW]
    float *sum_sm = reinterpret_cast<float *>(tail + L::SUM); // l, [2 items][4 WT warps][RPW]
    float *ref_sm = reinterpret_cast<float *>(tail + L::REF); // m, [2 items][X][RP]
    float *lgv_sm = reinterpret_cast<float *>(tail + L::LGV); // log2 V, [2 items][X]
    volatile int *bad_sm = reinterpret_cast<volatile int *>(tail + L::BAD); // [WT][tile parity]
    int *const nan2 = reinterpret_cast<int *>(tail + L::NANC); // first token that sees a NaN
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const ItemTable &it = p.items;
    volatile int never = 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(bar + B_FULL + s, 1);
            mbar_init(bar + B_EMPTY + s, 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar + B_SFULL + s, 1);
            mbar_init(bar + B_SFREE + s, 4 * W);
            mbar_init(bar + B_PFULL + s, 4 * W);
            mbar_init(bar + B_PFREE + s, 1);
            mbar_init(bar + B_SCFULL + s, 1);
            mbar_init(bar + B_SCFREE + s, 4 * WT);
            mbar_init(bar + B_PVDONE + s, 1);
        }
        mbar_init(bar + B_MFULL, 4 * WT);
        mbar_init(bar + B_OREADY, 1);
        mbar_init(bar + B_OFREE, 4 * WT);
        mbar_init(bar + B_QFULL, 4 * WT);
        mbar_init(bar + B_QFREE, 1);
        mbar_init(bar + B_QKDRAIN, 1);
        mbar_init(bar + B_PVDRAIN, 1);
        *abort_flag = 0;
        for (int i = 0; i < 2 * WT; ++i) bad_sm[i] = 0;
        fence_mbar_init();
    }
    if (warp == L::QK) tmem_alloc(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // The set-up above overlaps the end of the stream's last kernel (a programmatic launch:
    // 0.25 us of 7 on short contexts); nothing of it is touched before here, and what that
    // kernel may have written (lengths, tables, scales, q) is read by ordinary loads, which
    // the wait orders.
    griddep_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;

    // A whole warp: the page scales of four tiles at a time (a batch), a lane a group of 16
    // positions. The K producer looks the blocks of a batch up a batch ahead of its scales, and
    // those a batch ahead of their use, so that it waits for neither. Batches take two buffers
    // in turn.
    struct Batch {
        int blk, kvh;  // of the next batch: this lane's block (-1: none)
        float ks, vs;  // of this batch
    };
    auto blocks = [&](Walk8 &w, Batch &x) {
        int b = -1, pos = 0;
        for (int i = 0; i < 4 && !w.done; ++i, w.next(p, od))
            if ((lane >> 3) == i && w.t0 + 16 * (lane & 7) < w.t1) {
                b = w.b;
                x.kvh = w.kvh;
                pos = w.t0 + 16 * (lane & 7);
            }
        x.blk = b < 0 ? -1 : p.block_table[(size_t)b * p.max_blocks + pos / p.block_size];
    };
    auto scales = [&](Batch &x) {
        x.ks = x.vs = 0.f;
        if (x.blk >= 0 && x.blk < sc.num_blocks) {
            x.ks = sc.k[x.blk * sc.k_block + x.kvh * sc.k_head];
            x.vs = sc.v[x.blk * sc.v_block + x.kvh * sc.v_head];
        }
    };
    // false when the wait for the buffer runs out
    auto put_scales = [&](const Batch &x, int batch) {
        const int half = batch & 1;
        const bool got = mbar_wait_bounded(bar + B_SCFREE + half, ((uint32_t)(batch >> 1) & 1u) ^ 1u,
                                           p.timeout_ns, abort_flag);
        if (__any_sync(0xffffffffu, !got)) return false;
        const float vs = fmaxf(x.vs, kMinScale), lv = __log2f(vs);
        float top = lv; // over the tile's 8 lanes
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        sc_sm[half * 32 + lane] = make_float4(x.ks, lv, vs, 2.f * floorf(0.5f * top));
        __syncwarp();
        if (lane == 0) mbar_arrive(bar + B_SCFULL + half);
        return true;
    };

    if (warp == L::KPROD || warp == L::VPROD) {
        // =================== TMA producers, one for K and one for V ===================
        // box j holds positions [t0 + j*h, t0 + (j+1)*h) of a 128-column chunk, h =
        // box_rows (16 to 128: a divisor of the tile and of block_size), so no box spans
        // two blocks and a tile spans blocks freely; h * 128 bytes is a multiple of the
        // swizzle atom, so the boxes land as one box of the tile would. A box costs its
        // warp about 75 cycles to issue, and pages of 16 positions make 8 of each 16 KB:
        // one warp for both tiles took 2100 cycles per 128 positions of 128 columns,
        // the memory 1400.
        const bool isv = warp == L::VPROD;
        const CUtensorMap *map = isv ? &vmap : &kmap;
        if (lane == 0) tma_prefetch_map(map);
        fence_proxy_async_global(); // the pages as the append wrote them, for the copies
        const uint64_t pol = l2_evict_first_policy();
        const int bs = p.block_size, h = p.box_rows, nbox = T / h;
        // this lane's box of tile w: its block as the table has it (not looked at until the tile
        // is issued, so that the load has a tile's time), the first slot in it
        auto look_up = [&](const Walk8 &w, int &slot0) {
            int blk = p.oob_block;
            if (!w.done && lane < nbox) {
                const int pos = w.t0 + lane * h, idx = pos / bs;
                slot0 = pos - idx * bs;
                if (pos < w.t1 && idx < p.max_blocks) // past the tile: zeros, nothing is read
                    blk = p.block_table[(size_t)w.b * p.max_blocks + idx];
            }
            return blk;
        };
        uint32_t ph = 0, issued = 0, last = 0; // slots with copies, their last phases
        int slot = isv ? 1 : 0;                // slots of tile t: K 2t, V 2t + 1 (mod NS)
        bool ok = true;
        Walk8 w;
        w.start(p, od);
        int slot0 = 0, blk = look_up(w, slot0);
        const bool with_scales = L::KSCALE && !isv;
        Walk8 ws = w;
        Batch sb = {};
        if (with_scales) {
            blocks(ws, sb);
            scales(sb);
            blocks(ws, sb);
        }
        while (!w.done) {
            Walk8 nx = w; // the next tile's blocks are looked up while this one is issued
            nx.next(p, od);
            int nslot0 = 0;
            const int nblk = look_up(nx, nslot0);
            // a slot's first use finds its barrier's previous phase complete
            bool got = true;
            if (lane == 0)
                got = mbar_wait_bounded(bar + B_EMPTY + slot, ph ^ 1u, p.timeout_ns, abort_flag);
            if (!__shfl_sync(0xffffffffu, got, 0)) {
                ok = false;
                break;
            }
            if (!(p.flags & DA_FLAG_TEST_NO_TMA)) {
                issued |= 1u << slot;
                last = (last & ~(1u << slot)) | (ph << slot);
                uint8_t *dst = sm + L::SLOT_OFF + slot * L::SLOT + lane * h * 128;
                if (lane == 0) mbar_arrive_expect_tx(bar + B_FULL + slot, L::SLOT);
                if (blk < 0 || blk > p.oob_block) blk = p.oob_block; // reads as zeros
                __syncwarp();
                if (lane < nbox) {
#pragma unroll
                    for (int c = 0; c < NCH; ++c)
                        tma_load_4d(dst + c * L::CHUNK, map, bar + B_FULL + slot, c * 128, w.kvh,
                                    slot0, blk, pol);
                }
            }
            if (with_scales && (w.gt & 3) == 0) { // four tiles' scales, behind the first of them
                if (!put_scales(sb, w.gt >> 2)) {
                    ok = false;
                    break;
                }
                scales(sb);
                blocks(ws, sb);
            }
            if ((slot += 2) >= NS) {
                slot -= NS;
                ph ^= 1u;
            }
            w = nx;
            blk = nblk;
            slot0 = nslot0;
        }
        if (!ok && lane == 0) {
            *abort_flag = 1;
            atomicCAS(p.status, 0, kStatusTimeoutQ8);
        }
        // nothing may be in flight when the CTA exits: wait (bounded) for the last copies
        if (lane == 0)
            for (int s = 0; s < NS; ++s)
                if ((issued >> s) & 1u)
                    (void)mbar_wait_bounded(bar + B_FULL + s, (last >> s) & 1u, p.timeout_ns,
                                            &never);
    } else if (warp == L::SCALE) {
        Walk8 w;
        w.start(p, od);
        Batch sb = {};
        for (int batch = 0; !w.done; ++batch) { // (this warp has the time to wait for the loads)
            blocks(w, sb);
            scales(sb);
            if (!put_scales(sb, batch)) {
                if (lane == 0) {
                    *abort_flag = 1;
                    atomicCAS(p.status, 0, kStatusTimeoutQ8);
                }
                break;
            }
        }
    } else if (warp == L::QK || warp == L::PV) {
        // ================ MMA issue: one thread for S, one for O^T ================
        // Two issuers, so that neither polls for the other's inputs.
        if (lane == 0) {
            const bool qk = warp == L::QK;
            const uint32_t idesc = idesc_f8(qk ? N : NP, !qk, !qk && L::PMN, e5m2);
            uint32_t ph = 0, iph = 0, sph = 0; // phases: tile slot, item, S or P buffer
            uint32_t begun = 0;                // O^T sets of this item that hold something
            int slot = qk ? 0 : 1, items = 0;  // slots of tile t: K 2t, V 2t + 1 (mod NS)
            bool ok = true;
            Walk8 w;
            for (w.start(p, od); ok && !w.done; w.next(p, od)) {
                const int ss = w.gt & 1;
                const uint64_t ad = smem_desc_sw128(sb + L::SLOT_OFF + slot * L::SLOT, 16, 1024);
                auto wait = [&](int which, uint32_t parity) {
                    ok = ok && mbar_wait_bounded(bar + which, parity, p.timeout_ns, abort_flag);
                };
                if (qk) {
                    // S = K . q^T once q of the item and the K tile are in and the softmax has
                    // released this S slot
                    if (w.first) {
                        wait(B_QFULL, iph);
                        iph ^= 1u;
                    }
                    wait(B_FULL + slot, ph);
                    wait(B_SFREE + ss, ((sph >> ss) & 1u) ^ 1u);
                    sph ^= 1u << ss;
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t qd = smem_desc_sw128(sb + L::Q_OFF, 16, 1024);
#pragma unroll
                    for (int c = 0; c < NCH; ++c)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_f8(tmem + ss * N, ad + (uint64_t)((c * L::CHUNK + k * 32) >> 4),
                                   qd + (uint64_t)((c * L::QCH + k * 32) >> 4), idesc,
                                   (c | k) != 0 ? 1u : 0u);
                    tc_commit(bar + B_SFULL + ss);
                    tc_commit(bar + B_EMPTY + slot);
                    if (w.last()) tc_commit(bar + B_QFREE);
                } else {
                    // O^T += V^T . x^T once the V tile is in, x(t) is written and, at an item's
                    // first tile, the previous item's epilogue has read O^T
                    wait(B_FULL + slot, ph);
                    if (w.first && items++ > 0) {
                        wait(B_OFREE, iph);
                        iph ^= 1u;
                    }
                    wait(B_PFULL + ss, (sph >> ss) & 1u);
                    sph ^= 1u << ss;
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t pd = smem_desc_sw128(sb + L::P_OFF + ss * L::PSLOT, 16, 1024);
                    const int x = X > 1 ? ss : 0; // the tile's O^T, and whether it has begun
                    if (w.first) begun = 0;
                    const uint32_t more = (begun >> x) & 1u;
                    begun |= 1u << x;
#pragma unroll
                    for (int j = 0; j < NCH; ++j)
#pragma unroll
                        for (int k = 0; k < T / 32; ++k)
                            mma_f8(tmem + 2 * N + (x * NCH + j) * NP,
                                   ad + (uint64_t)((j * L::CHUNK + k * 4096) >> 4),
                                   pd + (uint64_t)((k * (L::PMN ? 4096 : 32)) >> 4), idesc,
                                   k == 0 ? more : 1u);
                    tc_commit(bar + B_EMPTY + slot);
                    tc_commit(bar + B_PFREE + ss);
                    tc_commit(bar + B_PVDONE + x);
                    if (w.last()) tc_commit(bar + B_OREADY);
                }
                if ((slot += 2) >= NS) {
                    slot -= NS;
                    ph ^= 1u;
                }
            }
            if (!ok) {
                *abort_flag = 1;
                atomicCAS(p.status, 0, kStatusTimeoutQ8);
            }
            // no MMA may be in flight when TMEM is freed
            tc_commit(bar + (qk ? B_QKDRAIN : B_PVDRAIN));
            (void)mbar_wait_bounded(bar + (qk ? B_QKDRAIN : B_PVDRAIN), 0, p.timeout_ns, &never);
        }
        __syncwarp();
    } else {
        // ===================== softmax and epilogue (warpgroups 0..WT-1) =====================
        const int wg = WT > 1 ? warp >> 2 : 0;
        const int turn = X > 1 ? wg / W : 0;            // tiles of this parity (X = 2)
        const int r00 = (W > 1 ? wg % W : 0) * RPW;     // this warpgroup's first row
        const int tid = threadIdx.x & 127; // position of the tile (TMEM lane), value column
        float *red = red_sm + wg * 4 * RPW;
        auto bar_or = [&](bool pred) { return named_bar_or(1 + wg, 128, pred); };
        const int Gh = p.hq / it.n_kv_heads, rows = Gh * p.q_len;
        const int per = (rows + it.row_groups - 1) / it.row_groups;
        const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16) + r00;
        const bool causal = p.q_len > 1 && !(p.flags & DA_FLAG_NO_CAUSAL);
        const bool direct = p.fused.on; // writes the output itself
        uint32_t sph = 0, pfp = 0, iph = 0, scp = 0; // iph: item parity
        bool ab = false;
        int gt = 0;
        int vslot = 1;
        uint32_t vph = 0;
        // The CTA's items in turn; those without positions get neutral partials and are
        // skipped. Where registers allow, every warp works out 32 items at a time, one a lane
        // (the look-ups of one item take 1500 cycles, as long as a tile), and reads them by
        // shuffles.
        struct Item {
            int k, b, kvh, Lb, p0, p1, row0, R, slot; // k: number in the CTA, -1 past the last
        };
        auto look = [&](int k) { // item k by itself; k = -1 past the last
            Item x;
            const int64_t item = item8(k);
            x.k = item < it.n_items ? k : -1;
            x.b = x.kvh = x.Lb = x.p0 = x.p1 = x.row0 = x.slot = 0;
            if (x.k >= 0) {
                int e, s, rg;
                decode_item(it, (int)item, e, x.kvh, s, rg);
                x.b = od.seq[e];
                x.Lb = len8(p, e, x.b);
                x.p0 = s * it.chunk[e];
                x.p1 = max(x.p0, min(x.Lb, x.p0 + it.chunk[e]));
                x.row0 = rg * per;
                x.slot = od.slot[e] + s;
            }
            x.R = min(per, rows - x.row0);
            return x;
        };
        // workspace row of row r of an item (with one split a sequence: the output row)
        auto row_of = [&](const Item &x, int r) {
            const int jf = x.row0 + r;
            return (size_t)x.slot * p.n_heads + (size_t)x.kvh * Gh + jf / Gh * p.hq + jf % Gh;
        };
        // an item without positions, by thread i of n: neutral partials, or zeros in the output
        auto empty_item = [&](const Item &x, int i, int n) {
            if (direct) {
                for (int r = 0; r < x.R; ++r)
                    for (int d = i; d < D; d += n) put_out(p.fused, row_of(x, r) * D + d, 0.f);
            } else {
                for (int r = i; r < x.R; r += n) p.ml[row_of(x, r)] = make_float2(kNeutralM, 0.f);
            }
        };
        constexpr bool kLanes = RP <= 8;
        int k0 = -32;
        Item mine; // item k0 + lane
        auto seek = [&](int k) {
            Item x;
            if constexpr (kLanes) {
                for (;;) {
                    if (k >= k0 + 32) {
                        k0 += 32;
                        mine = look(k0 + lane);
                        unsigned none =
                            __ballot_sync(0xffffffffu, mine.k >= 0 && mine.p1 == mine.p0);
                        while (warp == 0 && none) {
                            const int i = __ffs(none) - 1;
                            none &= none - 1;
                            x.kvh = __shfl_sync(0xffffffffu, mine.kvh, i);
                            x.row0 = __shfl_sync(0xffffffffu, mine.row0, i);
                            x.slot = __shfl_sync(0xffffffffu, mine.slot, i);
                            x.R = min(per, rows - x.row0);
                            empty_item(x, lane, 32);
                        }
                    }
                    const unsigned live =
                        __ballot_sync(0xffffffffu, mine.p1 > mine.p0) >> (k - k0);
                    if (live || __any_sync(0xffffffffu, mine.k < 0)) {
                        const int i = live ? k - k0 + __ffs(live) - 1 : 0;
                        x.k = live ? k0 + i : -1;
                        x.b = __shfl_sync(0xffffffffu, mine.b, i);
                        x.kvh = __shfl_sync(0xffffffffu, mine.kvh, i);
                        x.Lb = __shfl_sync(0xffffffffu, mine.Lb, i);
                        x.p0 = __shfl_sync(0xffffffffu, mine.p0, i);
                        x.p1 = __shfl_sync(0xffffffffu, mine.p1, i);
                        x.row0 = __shfl_sync(0xffffffffu, mine.row0, i);
                        x.slot = __shfl_sync(0xffffffffu, mine.slot, i);
                        x.R = min(per, rows - x.row0);
                        return x;
                    }
                    k = k0 + 32;
                }
            } else {
                for (;; ++k) {
                    x = look(k);
                    if (x.k < 0 || x.p1 > x.p0) return x;
                    if (wg == 0) empty_item(x, tid, 128);
                }
            }
        };
        // q of an item: the warps take rows in turn (QR each), a lane has 4 columns of every
        // chunk. get_q loads it, put_q writes it to shared memory, scaled to [128, 256) and
        // cut into terms, and the row tables (buffer `buf`), then arrives on QFULL.
        constexpr int QR = (RP + 4 * WT - 1) / (4 * WT);
        float4 qv[QR][NCH];
        auto get_q = [&](const Item &x) {
#pragma unroll
            for (int i = 0; i < QR; ++i) {
                const int r = warp + 4 * WT * i;
                const int tok = (x.row0 + r) / Gh, g = x.row0 + r - tok * Gh;
                const float *qr = p.q +
                                  ((size_t)(x.b * p.q_len + tok) * p.hq + (size_t)x.kvh * Gh + g) * D +
                                  4 * lane;
#pragma unroll
                for (int c = 0; c < NCH; ++c) {
                    qv[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (r < x.R) qv[i][c] = *reinterpret_cast<const float4 *>(qr + 128 * c);
                }
            }
        };
        auto put_q = [&](const Item &x, int buf) {
#pragma unroll
            for (int i = 0; i < QR; ++i) {
                const int r = warp + 4 * WT * i;
                if (RP % (4 * WT) && r >= RP) break;
                float4 (&v)[NCH] = qv[i];
                float a = 0.f;
                const int tok = (x.row0 + r) / Gh, g = x.row0 + r - tok * Gh;
#pragma unroll
                for (int c = 0; c < NCH; ++c) {
                    v[c].x *= p.scale_log2;
                    v[c].y *= p.scale_log2;
                    v[c].z *= p.scale_log2;
                    v[c].w *= p.scale_log2;
                    a = fmaxf(a, fmaxf(fmaxf(fabsf(v[c].x), fabsf(v[c].y)),
                                       fmaxf(fabsf(v[c].z), fabsf(v[c].w))));
                }
                a = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(a)));
                // 2^k with a * 2^k in [128, 256); k within what 2^k and 2^-k can be
                int k = 134 - (int)(__float_as_uint(a) >> 23);
                k = a > 0.f ? max(-120, min(120, k)) : 0;
                const float f = __uint_as_float((uint32_t)(127 + k) << 23);
                if (lane == 0) {
                    qf2[buf * RP + r] = __uint_as_float((uint32_t)(127 - k) << 23);
                    lim2[buf * RP + r] =
                        r >= x.R ? 0 : causal ? x.Lb - p.q_len + 1 + tok : INT_MAX;
                    wrow2[buf * RP + r] = r < x.R ? tok * p.hq + g : 0;
                }
                // an infinite q makes NaN scores, as infinities weighted against each other do
                const bool nan = !(a <= 3.402823466e38f);
#pragma unroll
                for (int c = 0; c < NCH; ++c) {
                    float y0 = v[c].x * f, y1 = v[c].y * f, y2 = v[c].z * f, y3 = v[c].w * f;
                    if (nan) y0 = __int_as_float(0x7fffffff);
#pragma unroll
                    for (int j = 0; j < QT; ++j) {
                        const uint32_t lo = term2(y0, y1), hi = term2(y2, y3);
                        sts_u32(sb + L::Q_OFF + c * L::QCH + swz(j * RP + r, 4 * lane),
                                lo | (hi << 16));
                    }
                }
            }
            if (causal)
                for (int i = threadIdx.x; i < D; i += 128 * WT) nan2[buf * D + i] = INT_MAX;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar + B_QFULL);
        };
        // narrow items have the registers to load the next item's q a tile ahead
        constexpr bool kAhead = RP <= 8;
        Item cur = seek(0);
        if (cur.k >= 0) {
            get_q(cur);
            put_q(cur, 0);
        }
        for (int n = 0; !ab && cur.k >= 0; ++n) {
            const int Lb = cur.Lb, p0 = cur.p0, p1 = cur.p1, row0 = cur.row0, R = cur.R;
            const size_t wbase = (size_t)cur.slot * p.n_heads + (size_t)cur.kvh * Gh;
            const float *qf_sm = qf2 + iph * RP;
            const int *lim_sm = lim2 + iph * RP, *wrow_sm = wrow2 + iph * RP;
            int *nan_sm = nan2 + iph * D;
            { // the other warps' row tables
                const bool okw = mbar_wait_bounded(bar + B_QFULL, iph, p.timeout_ns, abort_flag);
                if (bar_or(!okw)) {
                    ab = true;
                    break;
                }
            }

            const Item nxt = seek(cur.k + 1);
            const bool more = nxt.k >= 0;
            // ---- tiles
            float m[RPW], l[RPW]; // reference (uniform over the threads), this thread's share of l
#pragma unroll
            for (int r = 0; r < RPW; ++r) {
                m[r] = kNeutralM; // none yet
                l[r] = 0.f;
            }
            float high = kNeutralM; // the highest reference moved to so far of row lane % RPW
            float lgv = 0.f, inv_v = 1.f; // log2 V, 1 / V (uniform over the warpgroup)
            const int lim0 = causal ? Lb - p.q_len + 1 : INT_MAX; // the first token's limit
            bool firsttile = true;
            for (int t0 = p0, t1; t0 < p1; t0 = t1, ++gt) {
                t1 = tile_end<T>(t0, p1);
                if (kAhead && more && t1 >= p1) get_q(nxt);
                const int ss = gt & 1, half = (gt >> 2) & 1;
                if (X > 1 && ss != turn) { // the other set's tile
                    if ((vslot += 2) >= NS) {
                        vslot -= NS;
                        vph ^= 1u;
                    }
                    continue;
                }
                const int own = X > 1 ? gt >> 1 : gt; // number of this set's tile
                // the three barriers are looked at together (a look takes 110 cycles) and waited
                // for where they are not through
                const uint32_t sc_par = (scp >> half) & 1u, s_par = (sph >> ss) & 1u,
                               pf_par = ((pfp >> ss) & 1u) ^ 1u;
                const bool sc_in = (gt & 3) != turn || mbar_test(bar + B_SCFULL + half, sc_par),
                           s_in = mbar_test(bar + B_SFULL + ss, s_par),
                           p_free = mbar_test(bar + B_PFREE + ss, pf_par);
                bool okw = sc_in || mbar_wait_bounded(bar + B_SCFULL + half, sc_par, p.timeout_ns,
                                                      abort_flag);
                okw = okw && (s_in || mbar_wait_bounded(bar + B_SFULL + ss, s_par, p.timeout_ns,
                                                        abort_flag));
                okw = okw && (p_free || mbar_wait_bounded(bar + B_PFREE + ss, pf_par, p.timeout_ns,
                                                          abort_flag));
                if ((gt & 3) == turn) scp ^= 1u << half;
                sph ^= 1u << ss;
                pfp ^= 1u << ss;
                const bool short_tile = t1 - t0 < T, new_tokens = t1 > lim0;
                const bool fix_v = r00 == 0 && (short_tile || new_tokens);
                if (fix_v)
                    okw = okw && mbar_wait_bounded(bar + B_FULL + vslot, vph, p.timeout_ns,
                                                   abort_flag);
                tc_fence_after();
                const float4 sv = sc_sm[half * 32 + (gt & 3) * 8 + (tid >> 4)];
                const int pos = t0 + tid;
                if (okw && fix_v) {
                    const uint32_t vt = sb + L::SLOT_OFF + vslot * L::SLOT + tid * 128;
                    if (pos >= t1) {
                        // V rows past the tile hold whatever the pool has there: 0 * NaN would
                        // reach O^T. (K rows past it only give scores that are masked.)
#pragma unroll
                        for (int i = 0; i < NCH * 8; ++i)
                            sts_v4(vt + (i >> 3) * L::CHUNK + (((i + tid) & 7) << 4), 0u, 0u, 0u, 0u);
                    } else if (pos >= lim0) {
                        // a row that not every token sees: a NaN in it must not reach the others,
                        // so it is taken out and the epilogue puts it where it belongs
                        uint8_t *row = sm + L::SLOT_OFF + vslot * L::SLOT;
                        const uint32_t least = e5m2 ? 0x7c7c7c7cu : 0x7f7f7f7fu;
                        for (int i = 0; i < D; i += 4) {
                            uint32_t *c = reinterpret_cast<uint32_t *>(
                                row + (i >> 7) * L::CHUNK + swz(tid, i & 127));
                            const uint32_t u = *c, bad = __vcmpgeu4(u & 0x7f7f7f7fu, least);
                            if (bad) {
                                *c = u & ~bad;
                                for (int e = 0; e < 4; ++e)
                                    if ((bad >> (8 * e)) & 1u)
                                        atomicMin(nan_sm + i + e, pos - (Lb - p.q_len));
                            }
                        }
                    }
                }
                // a[r]: this position's score in row r, less the row's reference (`less`), -inf
                // where it is masked
                float a[RPW];
                auto scores = [&](bool less) {
#pragma unroll
                    for (int r0 = 0; r0 < RPW; r0 += SC) {
                        float v[QT][SC];
#pragma unroll
                        for (int j = 0; j < QT; ++j)
                            tmem_ld<SC>(tl + ss * N + j * RP + r0, v[j]);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < SC; ++i) {
                            float y = v[QT - 1][i];
#pragma unroll
                            for (int j = QT - 2; j >= 0; --j) y = fmaf(y, kTermStep, v[j][i]);
                            a[r0 + i] = fmaf(y, qf_sm[r00 + r0 + i] * sv.x, less ? -m[r0 + i] : 0.f);
                        }
                    }
                    if (pos >= t1) {
#pragma unroll
                        for (int r = 0; r < RPW; ++r) a[r] = -INFINITY;
                    } else if (new_tokens) {
#pragma unroll
                        for (int r = 0; r < RPW; ++r)
                            if (pos >= lim_sm[r00 + r]) a[r] = -INFINITY;
                    }
                };
                // One vote a tile, whether a row outgrew its reference or left it; a wait that ran out
                // joins it through a flag of this tile's parity (written before the tile's first
                // barrier, read after it, so the warpgroup leaves together). An item's first tile
                // always sets references.
                if (!okw) bad_sm[2 * wg + (own & 1)] = 1;
                // V first: the same for the whole warpgroup
                const bool wider = firsttile || sv.w > lgv + kWide;
                float half_v = 1.f; // sqrt(old V / new V)
                if (wider) {
                    if (!firsttile) half_v = pow2(max(-126, (int)(0.5f * (lgv - sv.w))));
                    lgv = sv.w;
                    inv_v = pow2(-(int)lgv);
                }
                const float lv = fmaxf(sv.y - lgv, kLeast), vs = sv.z * inv_v;
                // the tile's largest weights, from a[] as scores(false) left it; false when a wait
                // of the warpgroup has run out
                auto largest = [&](float *tm) {
#pragma unroll
                    for (int r = 0; r < RPW; ++r) {
                        // as ordered integers; a NaN counts as -inf
                        const int u = __float_as_int(fmaxf(a[r] + lv, -INFINITY));
                        const int o = __reduce_max_sync(0xffffffffu, u ^ ((u >> 31) & 0x7fffffff));
                        if (lane == 0)
                            red[(warp & 3) * RPW + r] = __int_as_float(o ^ ((o >> 31) & 0x7fffffff));
                    }
                    named_bar_sync(1 + wg, 128);
#pragma unroll
                    for (int r = 0; r < RPW; ++r)
                        tm[r] = fmaxf(fmaxf(red[r], red[RPW + r]),
                                      fmaxf(red[2 * RPW + r], red[3 * RPW + r]));
                    return !bad_sm[2 * wg + (own & 1)];
                };
                // An item's first tile has a path of its own where items are narrow and often
                // short (256 sequences of 40 positions, 4 rows of 128: 45.3 -> 40.9 us; 76 of
                // 128, 8 rows: 19.8 -> 18.6; but 16 rows, 1.2M positions: 66 -> 69)
                constexpr bool kFirst = RP <= 8;
                bool ex = wider;
                if (kFirst && firsttile) {
                    float tm[RPW];
                    scores(false);
                    if (!largest(tm)) {
                        ab = true;
                        break;
                    }
#pragma unroll
                    for (int r = 0; r < RPW; ++r) {
                        if (tm[r] > -INFINITY) m[r] = 2.f * floorf(0.5f * (tm[r] - kHead));
                        a[r] -= m[r];
                    }
                    ex = false;
                } else if (!firsttile) {
                    scores(true);
                    const float most = kTau - lv, least = -kLow - lv;
                    float top = a[0];
                    unsigned low = 0; // rows of which this warp's positions all lie low
#pragma unroll
                    for (int r = RPW - 1; r >= 0; --r) {
                        top = fmaxf(top, a[r]);
                        low = __funnelshift_l(__float_as_uint(a[r] - least), low, 1); // its sign
                    }
                    ex |= top > most;
                    low = __reduce_and_sync(0xffffffffu, low);
                    if (t0 + 32 * (warp & 3) >= t1) low = 0; // it has none
                    // a row that lies low in the whole tile counts once for each warp that has
                    // positions, and a warp with any other cause 32 times
                    ex = __any_sync(0xffffffffu, ex || !okw);
                    ex = named_bar_count(1 + wg, 128, ex || ((low >> lane) & 1u)) >=
                         (t1 - t0 + 31) >> 5;
                }
                if (ex) {
                    // move the references that scores outgrew or left; rescale l and O^T
                    float al[RPW]; // the tile's largest, then square roots of the factors, exact
                    scores(false);
                    if (!largest(al)) {
                        ab = true;
                        break;
                    }
                    bool moved = wider;
#pragma unroll
                    for (int r = 0; r < RPW; ++r) {
                        const float tm = al[r];
                        float hi = __shfl_sync(0xffffffffu, high, r);
                        if (kFirst) hi = fmaxf(hi, m[r]); // (the first tile's)
                        float mn = m[r];
                        if (tm > mn + kTau || (tm < mn - kLow && tm > -INFINITY))
                            mn = fmaxf(2.f * floorf(0.5f * (tm - kHead)), hi - kDeep);
                        if (lane % RPW == r) high = fmaxf(hi, mn);
                        moved |= mn != m[r];
                        al[r] = m[r] - mn;
                        m[r] = mn;
                        a[r] -= mn;
                    }
                    // the set's last PV is done with O^T before it is rescaled
                    if (!firsttile && moved) {
#pragma unroll
                        for (int r = 0; r < RPW; ++r) {
                            al[r] = pow2(max(-126, (int)(0.5f * al[r])));
                            l[r] = l[r] * al[r] * al[r];
                            al[r] *= half_v;
                        }
                        okw = mbar_wait_bounded(bar + B_PVDONE + turn, (uint32_t)(own - 1) & 1u,
                                                p.timeout_ns, abort_flag);
                        if (bar_or(!okw)) {
                            ab = true;
                            break;
                        }
                        tc_fence_after();
                        // the columns of two terms at a time: one round trip for each
                        for (int j = 0; j < NCH; ++j)
#pragma unroll
                            for (int k = 0; k < PT; k += 2) {
                                float o[2][RPW];
                                const uint32_t at = tl + 2 * N + (turn * NCH + j) * NP + k * RP;
                                const int two = k + 1 < PT ? 2 : 1;
#pragma unroll
                                for (int e = 0; e < two; ++e)
#pragma unroll
                                    for (int r0 = 0; r0 < RPW; r0 += RC)
                                        tmem_ld<RC>(at + e * RP + r0, o[e] + r0);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < two; ++e) {
#pragma unroll
                                    for (int r = 0; r < RPW; ++r) o[e][r] = o[e][r] * al[r] * al[r];
#pragma unroll
                                    for (int r0 = 0; r0 < RPW; r0 += RC)
                                        tmem_st4(at + e * RP + r0, o[e] + r0);
                                }
                            }
                        tmem_wait_st();
                    }
                }
                // weights: l, and the terms of x into the P buffer
                const uint32_t pt = sb + L::P_OFF + ss * L::PSLOT;
#pragma unroll
                for (int r = 0; r < RPW; ++r) {
                    a[r] = ex2(a[r]);
                    l[r] += a[r];
                    a[r] *= vs;
                }
                uint32_t c[RPW / 2][PT]; // codes of two rows
#pragma unroll
                for (int r = 0; r < RPW; r += 2) terms<PT>(a[r], a[r + 1], c[r / 2]);
#pragma unroll
                for (int j = 0; j < PT; ++j) {
                    const uint32_t at = pt + swz(tid, j * RP + r00);
                    if constexpr (L::PMN && RPW == 4) {
                        sts_u32(at, c[0][j] | (c[1][j] << 16));
                    } else if constexpr (L::PMN) {
                        sts_v2(at, c[0][j] | (c[1][j] << 16), c[2][j] | (c[3][j] << 16));
                    } else {
#pragma unroll
                        for (int r = 0; r < RPW; r += 2) {
                            sts_u8(pt + swz(j * RP + r00 + r, tid), c[r / 2][j] & 0xff);
                            sts_u8(pt + swz(j * RP + r00 + r + 1, tid), c[r / 2][j] >> 8);
                        }
                    }
                }
                tc_fence_before();
                fence_proxy_async_smem();
                __syncwarp();
                firsttile = false;
                // lanes 0 to 2: S and (after four tiles) the scales are read, x is written
                if (lane < ((gt & 3) == (X > 1 ? 2 + turn : 3) ? 3 : 2))
                    mbar_arrive(bar + (lane == 0   ? B_SFREE + ss
                                       : lane == 1 ? B_PFULL + ss
                                                   : B_SCFREE + half));
                if ((vslot += 2) >= NS) {
                    vslot -= NS;
                    vph ^= 1u;
                }
            }
            if (ab) break;
            // l over the threads (lanes by a transposing reduce, the warps later), m and log2 V,
            // where the other set and the epilogue find them
            float *sum = sum_sm + iph * 4 * RP * X, *ref = ref_sm + iph * RP * X;
            tr_reduce<RPW, 16>(l, lane);
            if (tr_writer<RPW, 16>(lane)) {
#pragma unroll
                for (int i = 0; i < tr_out<RPW, 16>(); ++i)
                    sum[warp * RPW + tr_base<RPW, 16>(lane) + i] = l[i];
            }
            if (tid == 0) {
#pragma unroll
                for (int r = 0; r < RPW; ++r) ref[turn * RP + r00 + r] = m[r];
                if (X > 1) lgv_sm[iph * X + turn] = lgv;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar + B_MFULL);
            // ---- q of the next item, while the last value MMA runs: once the last QK is done
            // with Q, and every warp with the row tables of the item before this one
            if (more) {
                if (!kAhead) get_q(nxt);
                bool okw = mbar_wait_bounded(bar + B_QFREE, iph, p.timeout_ns, abort_flag);
                if (n > 0)
                    okw = okw &&
                          mbar_wait_bounded(bar + B_OFREE, iph ^ 1u, p.timeout_ns, abort_flag);
                if (bar_or(!okw)) {
                    ab = true;
                    break;
                }
                put_q(nxt, iph ^ 1);
            }
            // ------------------------------- epilogue -------------------------------
            bool okw = mbar_wait_bounded(bar + B_MFULL, iph, p.timeout_ns, abort_flag);
            // Lane r works out row r of this warpgroup (all lanes, RPW in turn), while the last
            // value MMA runs. A set's l is between 2^E and 2^(E + 1): the row's partial is
            // published under the larger m + E of the sets, so that l is in [1, 4), the sums of
            // values are about the size of a value, and merges meet the extremes of neither. A
            // set's O^T comes under that by f = 2^(m - the row's) and V (0: the set has nothing,
            // and its O^T may hold anything; a set whose only scores are NaN has no reference,
            // but a NaN in l).
            float fl[X], Ml = kNeutralM, ll = 0.f, inv = 1.f;
            const int lr = lane % RPW, wl = wrow_sm[r00 + lr];
            {
                float me[X], l2[X]; // m + E, and l / 2^E (or the 0 or NaN that l is)
#pragma unroll
                for (int x = 0; x < X; ++x) {
                    const float *s4 = sum + (x * W + r00 / RPW) * 4 * RPW + lr;
                    const float l1 = s4[0] + s4[RPW] + s4[2 * RPW] + s4[3 * RPW];
                    const int u = __float_as_int(l1);
                    const bool some = l1 > 0.f;
                    l2[x] = some ? __int_as_float((u & 0x7fffff) | 0x3f800000) : l1;
                    fl[x] = some ? __int_as_float((254 << 23) - (u & 0x7f800000)) : l1; // 2^-E
                    me[x] = some ? ref[x * RP + r00 + lr] + (float)((u >> 23) - 127) : kNeutralM;
                    Ml = fmaxf(Ml, me[x]);
                }
#pragma unroll
                for (int x = 0; x < X; ++x) {
                    if (X > 1 && l2[x] > 0.f) {
                        l2[x] *= pow2(max(-126, (int)(me[x] - Ml)));
                        fl[x] = pow2(max(-126, (int)(ref[x * RP + r00 + lr] - Ml)));
                    }
                    ll += l2[x];
                }
                if (direct) inv = ll == 0.f ? 0.f : 1.f / ll; // nothing seen: zero; NaN: NaN
            }
            float vx[X]; // V of the sets
#pragma unroll
            for (int x = 0; x < X; ++x) vx[x] = pow2((int)(X > 1 ? lgv_sm[iph * X + x] : lgv));
            okw = okw && mbar_wait_bounded(bar + B_OREADY, iph, p.timeout_ns, abort_flag);
            if (bar_or(!okw)) {
                ab = true;
                break;
            }
            tc_fence_after();
            // the sets of warpgroups take the row chunks in turn
#pragma unroll
            for (int r0 = 0; r0 < RPW; r0 += RC) {
                if (X > 1 && (r0 / RC) % X != turn) continue;
                float v[NCH][X][PT][RC];
#pragma unroll
                for (int j = 0; j < NCH; ++j)
#pragma unroll
                    for (int x = 0; x < X; ++x)
#pragma unroll
                        for (int k = 0; k < PT; ++k)
                            tmem_ld<RC>(tl + 2 * N + (x * NCH + j) * NP + k * RP + r0, v[j][x][k]);
                tmem_wait_ld();
                float y[NCH][RC];
                size_t at[RC];
#pragma unroll
                for (int i = 0; i < RC; ++i) {
                    at[i] = (wbase + __shfl_sync(0xffffffffu, wl, r0 + i)) * D + tid;
#pragma unroll
                    for (int j = 0; j < NCH; ++j) y[j][i] = 0.f;
#pragma unroll
                    for (int x = 0; x < X; ++x) {
                        const float f = __shfl_sync(0xffffffffu, fl[x], r0 + i);
#pragma unroll
                        for (int j = 0; j < NCH; ++j) {
                            float o = v[j][x][PT - 1][i];
#pragma unroll
                            for (int k = PT - 2; k >= 0; --k)
                                o = fmaf(o, kTermStep, v[j][x][k][i]);
                            if (f != 0.f) y[j][i] = fmaf(o * f, vx[x], y[j][i]);
                        }
                    }
                    if (direct) {
                        const float n1 = __shfl_sync(0xffffffffu, inv, r0 + i);
#pragma unroll
                        for (int j = 0; j < NCH; ++j) y[j][i] = n1 == 0.f ? 0.f : y[j][i] * n1;
                    }
                }
                if (causal)
#pragma unroll
                    for (int j = 0; j < NCH; ++j) {
                        const int from = nan_sm[128 * j + tid];
#pragma unroll
                        for (int i = 0; i < RC; ++i)
                            if (from != INT_MAX && (row0 + r00 + r0 + i) / Gh >= from)
                                y[j][i] = __int_as_float(0x7fffffff);
                    }
                if (QT == 5 || !direct) { // five terms: the output is f32 too
                    float *dst = direct ? static_cast<float *>(p.fused.out) : p.acc;
#pragma unroll
                    for (int i = 0; i < RC; ++i)
                        if (r00 + r0 + i < R)
#pragma unroll
                            for (int j = 0; j < NCH; ++j) dst[at[i] + 128 * j] = y[j][i];
                } else {
                    const bool half = p.fused.out_dtype == DA_F16;
#pragma unroll
                    for (int i = 0; i < RC; ++i)
                        if (r00 + r0 + i < R)
#pragma unroll
                            for (int j = 0; j < NCH; ++j)
                                static_cast<uint16_t *>(p.fused.out)[at[i] + 128 * j] =
                                    half ? __half_as_ushort(__float2half_rn(y[j][i]))
                                         : __bfloat16_as_ushort(__float2bfloat16_rn(y[j][i]));
                }
            }
            if (!direct && turn == 0 && (warp & 3) == 0 && lane < RPW && r00 + lane < R)
                // a NaN score makes the row NaN whatever the other splits hold
                p.ml[wbase + wl] = isnan(ll)
                                       ? make_float2(-kNeutralM, 1.f)
                                       : make_float2(ll > 0.f ? Ml * kLn2 : kNeutralM, ll);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar + B_OFREE);
            cur = nxt;
            iph ^= 1u;
        }
        if (ab && tid == 0 && !*abort_flag) {
            *abort_flag = 1;
            atomicCAS(p.status, 0, kStatusTimeoutQ8);
        }
    }

    // ---------------------------------- teardown ----------------------------------
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == L::QK) tmem_dealloc(tmem, 512);
    if (threadIdx.x == 0) griddep_launch_dependents();
}

template <int D, int RP, int QT, int PT>
cudaError_t launch_t(int grid, cudaStream_t st, const CUtensorMap &km, const CUtensorMap &vm,
                     const Scales8 &sc, const Order8 &od, const SplitParams &p, int e5m2)
{
    using L = Layout<D, RP, QT, PT>;
    auto *fn = gqa_8bit_kernel<D, RP, QT, PT>;
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(L::THREADS);
    cfg.dynamicSmemBytes = L::BYTES;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, fn, km, vm, sc, od, p, e5m2);
    const cudaError_t last = cudaGetLastError();
    return e != cudaSuccess ? e : last;
}

// The narrowest instantiation that holds the item's rows, with the terms of the output's type.
template <int D>
cudaError_t launch_d(int rows, bool out16, int grid, cudaStream_t st, const CUtensorMap &km,
                     const CUtensorMap &vm, const Scales8 &sc, const Order8 &od,
                     const SplitParams &p, int e5m2)
{
    if (out16) {
        if (rows <= 4) return launch_t<D, 4, 4, 4>(grid, st, km, vm, sc, od, p, e5m2);
        if (rows <= 8) return launch_t<D, 8, 4, 4>(grid, st, km, vm, sc, od, p, e5m2);
        if (rows <= 16) return launch_t<D, 16, 4, 4>(grid, st, km, vm, sc, od, p, e5m2);
        if (rows <= 24) return launch_t<D, 24, 4, 4>(grid, st, km, vm, sc, od, p, e5m2);
        return launch_t<D, 32, 4, 4>(grid, st, km, vm, sc, od, p, e5m2);
    }
    if (rows <= 4) return launch_t<D, 4, 5, 5>(grid, st, km, vm, sc, od, p, e5m2);
    if (rows <= 8) return launch_t<D, 8, 5, 5>(grid, st, km, vm, sc, od, p, e5m2);
    if (rows <= 16) return launch_t<D, 16, 5, 5>(grid, st, km, vm, sc, od, p, e5m2);
    return launch_t<D, 24, 5, 5>(grid, st, km, vm, sc, od, p, e5m2);
}

} // namespace

int q8_rows_per_item(int rows, int out_dtype)
{
    // five terms of 32 rows are more columns than TMEM and a row of weights hold
    const int most = out_dtype == DA_F32 ? 24 : 32, groups = (rows + most - 1) / most;
    return (rows + groups - 1) / groups;
}

cudaError_t launch_gqa_8bit(int code_dtype, int out_dtype, int head_dim, int grid, cudaStream_t st,
                            const CUtensorMap &km, const CUtensorMap &vm, const Scales8 &sc,
                            const Order8 &od, const SplitParams &p)
{
    const int rows = p.n_heads / p.items.n_kv_heads;
    const int per = (rows + p.items.row_groups - 1) / p.items.row_groups;
    const int e5m2 = code_dtype == DA_E5M2;
    const bool out16 = out_dtype != DA_F32;
    if (head_dim == 128) return launch_d<128>(per, out16, grid, st, km, vm, sc, od, p, e5m2);
    return launch_d<256>(per, out16, grid, st, km, vm, sc, od, p, e5m2);
}

} // namespace skv
