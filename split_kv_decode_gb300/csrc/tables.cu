// decode_attn_grow_tables: block tables and slot maps of a decode step, from the
// request lengths, on the device.
//
// With page size P, sequence b of length L that gets n tokens holds
// have = ceil(L / P) blocks and takes need = ceil((L + n) / P) - have more. The
// k-th block taken (over all sequences, in order) comes from the top of a
// stack on which the call's R released blocks were pushed last:
//     k < R:  released block R - 1 - k      (read from its sequence's table)
//     else:   free_list[F - 1 - (k - R)]    (F free blocks before the call)
// so every block taken, slot and table entry is a function of prefix sums over
// the batch (at most 256 sequences). Every CTA forms those sums for itself from
// the lengths, and no CTA waits for another: what is read (the free list below
// F, tables of released sequences, old table entries) is never written by the
// same call. The lengths and the state may be updated in place, so they are
// written by the last CTA to have read them (a ticket count).
#include <algorithm>
#include <cstdio>

#include "internal.h"
#include "ptx.cuh"

namespace skv {
int set_error(int code, const char *phase, const char *msg); // api.cpp
}

namespace {

constexpr int kThreads = 256;
static_assert(kThreads == DA_MAX_BATCH, "one sequence per thread in the prefix sums");

struct TablesParams {
    da_tables_t t;
    const int32_t *new_lens;
    int64_t *slot_map;
    int32_t *cu_new;
    int32_t slots; // entries of slot_map
    int32_t shift; // log2 of block_size, or -1
    int32_t wide;  // slot_map is 16-byte aligned
};

// the last i in [lo, hi] with base[i] <= x (base ascending, base[lo] <= x)
__device__ __forceinline__ int find(const int32_t *base, int lo, int hi, int x)
{
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (base[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Inclusive prefix sums of a and b over the warp's lanes.
__device__ __forceinline__ void warp_scan(int64_t &a, int64_t &b)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) {
            a += x;
            b += y;
        }
    }
}

// PER: consecutive slots a lane takes
template <int PER>
__global__ void __launch_bounds__(kThreads) grow_tables_kernel(const TablesParams p)
{
    // (no early launch of what follows: its waiting CTAs took 2.7 us of 8.9 for 2.1M slots)
    skv::griddep_wait();
    __shared__ int64_t sums[2][kThreads / 32];
    __shared__ int32_t len_s[kThreads], have_s[kThreads], add_base[kThreads],
        need_base[kThreads], given_base[kThreads];
    __shared__ int last_s;
    const da_tables_t &t = p.t;
    const int B = t.batch, P = t.block_size, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    const int32_t L = tid < B ? t.seq_lens[tid] : 0;
    const int32_t n = tid < B ? p.new_lens[tid] : 0;
    const int32_t F = t.state[0], old_status = t.state[1];
    const bool gone = n < 0;
    const int64_t end = (int64_t)L + (gone ? 0 : n);
    const bool fits = L >= 0 && end <= (int64_t)t.max_blocks_per_seq * P && end <= INT32_MAX;
    auto pages = [&](int x) { // ceil(x / P), x >= 0
        return p.shift >= 0 ? (int)(((uint32_t)x + (uint32_t)P - 1) >> p.shift)
                            : (int)(((uint32_t)x + (uint32_t)P - 1) / (uint32_t)P);
    };
    const int have = fits ? pages(L) : 0;
    const int need = fits && !gone ? pages((int)end) - have : 0;
    const int given = fits && gone ? have : 0;
    const int add = fits && !gone ? n : 0;

    // prefix sums of the blocks taken and given (each below 2^31: one word) and the rows
    int64_t blocks = ((int64_t)need << 32) | (int64_t)given, rows = add;
    const int64_t own_blocks = blocks, own_rows = rows;
    warp_scan(blocks, rows);
    if (lane == 31) {
        sums[0][warp] = blocks;
        sums[1][warp] = rows;
    }
    const bool all_fit = __syncthreads_and(fits);
    int64_t total_blocks = 0, total_rows = 0;
    blocks -= own_blocks;
    rows -= own_rows;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        blocks += w < warp ? sums[0][w] : 0;
        rows += w < warp ? sums[1][w] : 0;
        total_blocks += sums[0][w];
        total_rows += sums[1][w];
    }
    const int64_t total_need = total_blocks >> 32, total_given = total_blocks & 0x7fffffff;
    const bool sound =
        all_fit && F >= 0 && F + total_given <= t.num_blocks && total_rows <= p.slots;
    const bool ok = sound && total_need <= F + total_given;
    len_s[tid] = L;
    have_s[tid] = have;
    add_base[tid] = ok ? (int32_t)rows : 0;
    need_base[tid] = ok ? (int32_t)(blocks >> 32) : 0;
    given_base[tid] = ok ? (int32_t)(blocks & 0x7fffffff) : 0;
    const int adds = ok ? (int)total_rows : 0, takes = ok ? (int)total_need : 0,
              gives = ok ? (int)total_given : 0;
    // this CTA has read the lengths and the state: the last one to have writes them
    __threadfence();
    __syncthreads();
    if (tid == 0)
        last_s = gridDim.x == 1 || atomicAdd(t.state_out + 2, 1) == (int)gridDim.x - 1;

    // the k-th released block, and the k-th block taken
    auto released = [&](int k) {
        const int b = find(given_base, 0, B - 1, k);
        return t.block_table[(size_t)b * t.max_blocks_per_seq + k - given_base[b]];
    };
    auto taken = [&](int k) {
        return k < gives ? released(gives - 1 - k) : t.free_list[F - 1 - (k - gives)];
    };
    // the block of position i * P + off of sequence b; the caller of a block's first
    // position (a block taken begins with a new token) writes its table entry
    auto block_of = [&](int b, int i, int off) {
        int32_t *entry = t.block_table + (size_t)b * t.max_blocks_per_seq + i;
        if (i < have_s[b]) return *entry;
        const int blk = taken(need_base[b] + i - have_s[b]);
        if (off == 0) *entry = blk;
        return blk;
    };
    // Slots: a warp takes 32 * PER consecutive ones, a lane PER of them. One search finds
    // the sequences of the first and the last, and the lanes search between them only
    // where those differ.
    constexpr int SPAN = 32 * PER;
    const int gwarp = blockIdx.x * (kThreads / 32) + warp, warps = gridDim.x * (kThreads / 32);
    for (int64_t j0 = (int64_t)gwarp * SPAN; j0 < p.slots; j0 += (int64_t)warps * SPAN) {
        const int probe = min((int)(lane ? j0 + SPAN - 1 : j0), max(adds - 1, 0));
        const int at = find(add_base, 0, B - 1, probe);
        const int b0 = __shfl_sync(0xffffffffu, at, 0), b1 = __shfl_sync(0xffffffffu, at, 1);
        const int64_t j = j0 + PER * lane;
        int64_t slot[PER];
        int b = 0, i = 0, off = 0, blk = 0, left = 0; // left: rows of sequence b from here on
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const int je = (int)j + e;
            slot[e] = -1;
            if (je < adds) {
                if (left == 0) { // the first one, or the next sequence that has rows
                    b = b0 == b1 ? b0 : find(add_base, e ? b : b0, b1, je);
                    left = (b + 1 < B ? add_base[b + 1] : adds) - je;
                    const uint32_t pos = (uint32_t)(len_s[b] + (je - add_base[b]));
                    i = (int)(p.shift >= 0 ? pos >> p.shift : pos / (uint32_t)P);
                    off = (int)(pos - (uint32_t)i * (uint32_t)P);
                    blk = block_of(b, i, off);
                } else if (off == P) {
                    off = 0;
                    blk = block_of(b, ++i, 0);
                }
                slot[e] = (int64_t)blk * P + off;
                ++off;
                --left;
            }
        }
        if (PER > 1 && p.wide && j + PER <= p.slots) {
#pragma unroll
            for (int e = 0; e + 1 < PER; e += 2)
                *reinterpret_cast<longlong2 *>(p.slot_map + j + e) =
                    make_longlong2(slot[e], slot[e + 1]);
        } else {
#pragma unroll
            for (int e = 0; e < PER; ++e)
                if (j + e < p.slots) p.slot_map[j + e] = slot[e];
        }
    }
    // released blocks that nobody took
    const int stride = gridDim.x * kThreads, first = blockIdx.x * kThreads + tid;
#pragma unroll 4
    for (int k = first; k < gives - takes; k += stride) t.free_list[F + k] = released(k);

    __syncthreads(); // last_s
    if (last_s) {
        if (tid < B) {
            t.seq_lens_out[tid] = ok ? (gone ? 0 : (int32_t)end) : L;
            if (p.cu_new) p.cu_new[tid] = add_base[tid];
        }
        if (tid == 0) {
            if (p.cu_new) p.cu_new[B] = adds;
            t.state_out[0] = F + gives - takes;
            t.state_out[1] = old_status ? old_status : ok ? 0 : sound ? DA_ENOSPACE : DA_EINVAL;
            t.state_out[2] = 0;
        }
    }
}

int bad(const char *msg) { return skv::set_error(DA_EINVAL, "args", msg); }

} // namespace

extern "C" int decode_attn_grow_tables(const da_tables_t *t, const int32_t *new_lens,
                                       int64_t *slot_map, int64_t slot_capacity, int32_t *cu_new,
                                       da_stream_t stream)
{
    if (!t) return bad("tables is NULL");
    if (t->batch < 1 || t->batch > DA_MAX_BATCH) return bad("batch outside [1, 256]");
    if (t->block_size < 1 || t->max_blocks_per_seq < 1 || t->num_blocks < 1)
        return bad("block_size, max_blocks_per_seq and num_blocks must be >= 1");
    if ((int64_t)t->batch * t->max_blocks_per_seq > INT32_MAX)
        return bad("batch * max_blocks_per_seq must be below 2^31");
    if (!t->seq_lens || !t->seq_lens_out || !t->block_table || !t->free_list || !t->state ||
        !t->state_out || !new_lens)
        return bad("a table pointer is NULL");
    if (slot_capacity < 0 || slot_capacity > (INT32_MAX >> 1))
        return bad("slot_capacity outside [0, 2^30)");
    if (slot_capacity > 0 && !slot_map) return bad("slot_map is NULL");
    for (const void *x : {(const void *)t->seq_lens, (const void *)t->seq_lens_out,
                          (const void *)t->block_table, (const void *)t->free_list,
                          (const void *)t->state, (const void *)t->state_out,
                          (const void *)new_lens, (const void *)cu_new})
        if (reinterpret_cast<uintptr_t>(x) % 4) return bad("an int32 array is misaligned");
    if (reinterpret_cast<uintptr_t>(slot_map) % 8) return bad("slot_map is misaligned");
    const cudaError_t pre = cudaGetLastError();
    if (pre != cudaSuccess) return skv::set_error(DA_ECUDA, "before tables", cudaGetErrorString(pre));
    TablesParams p;
    p.t = *t;
    p.new_lens = new_lens;
    p.slot_map = slot_map;
    p.cu_new = cu_new;
    p.slots = (int32_t)slot_capacity;
    p.shift = -1;
    for (int s = 0; s < 31; ++s)
        if (t->block_size == 1 << s) p.shift = s;
    p.wide = reinterpret_cast<uintptr_t>(slot_map) % 16 == 0;
    // Few slots: one a lane, so that their look-ups go side by side (a decode step's are of
    // different sequences); many (over one a thread of the GPU): four, which share a look-up
    // where they lie in one block (2.1M slots of 256 prompts: 8.9 us; one a lane 2 more). CTAs
    // for the most that the call may have to write: the slots, or the free list's entries of
    // released blocks, 1024 a CTA; at most four an SM.
    const int per = slot_capacity > 152 * 4 * kThreads ? 4 : 1;
    const int64_t most = std::max(slot_capacity / (per * kThreads),
                                  (int64_t)t->batch * t->max_blocks_per_seq / 1024);
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(152 * 4, most));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = skv::launch_after(per == 4 ? grow_tables_kernel<4> : grow_tables_kernel<1>,
                                            grid, kThreads, st, p);
    if (e != cudaSuccess) return skv::set_error(DA_ELAUNCH, "tables", cudaGetErrorString(e));
    return DA_OK;
}

extern "C" int decode_attn_tables_status(int32_t *state, da_stream_t stream)
{
    if (!state) return bad("state is NULL");
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    int v = 0;
    cudaError_t e = cudaMemcpyAsync(&v, state + 1, sizeof v, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) return skv::set_error(DA_ECUDA, "sync", cudaGetErrorString(e));
    if (v == 0) return DA_OK;
    e = cudaMemsetAsync(state + 1, 0, sizeof v, st);
    if (e != cudaSuccess) return skv::set_error(DA_ECUDA, "status", cudaGetErrorString(e));
    if (v == DA_ENOSPACE)
        return skv::set_error(DA_ENOSPACE, "tables",
                              "the free list ran out of blocks; the call changed nothing");
    if (v == DA_EINVAL)
        return skv::set_error(DA_EINVAL, "tables",
                              "a length passed the table's width, the tokens did not fit the "
                              "slot map, or the state is inconsistent; the call changed nothing");
    return skv::set_error(DA_ECUDA, "status", "unexpected status word");
}
