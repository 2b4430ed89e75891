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
};

// exclusive prefix sum of v over the block's threads; *total: the sum
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *total, int64_t *warp_sums)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        before += w < warp ? warp_sums[w] : 0;
        all += warp_sums[w];
    }
    __syncthreads();
    *total = all;
    return before + x - v;
}

// the last i in [0, n) with base[i] <= x (base ascending, base[0] = 0)
__device__ __forceinline__ int find(const int32_t *base, int n, int x)
{
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (base[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kThreads) grow_tables_kernel(const TablesParams p)
{
    __shared__ int64_t warp_sums[kThreads / 32];
    __shared__ int32_t len_s[kThreads], have_s[kThreads], add_base[kThreads + 1],
        need_base[kThreads + 1], given_base[kThreads + 1];
    const da_tables_t &t = p.t;
    const int B = t.batch, P = t.block_size, tid = threadIdx.x;

    const int32_t L = tid < B ? t.seq_lens[tid] : 0;
    const int32_t n = tid < B ? p.new_lens[tid] : 0;
    const int32_t F = t.state[0], old_status = t.state[1];
    const bool gone = n < 0;
    const int64_t end = (int64_t)L + (gone ? 0 : n);
    bool fits = L >= 0 && end <= (int64_t)t.max_blocks_per_seq * P && end <= INT32_MAX;
    const int have = fits ? (int)(((int64_t)L + P - 1) / P) : 0;
    const int need = fits && !gone ? (int)((end + P - 1) / P) - have : 0;
    const int given = fits && gone ? have : 0;
    const int add = fits && !gone ? n : 0;

    int64_t total_need, total_given, total_add;
    const int64_t nb = block_scan(need, &total_need, warp_sums);
    const int64_t gb = block_scan(given, &total_given, warp_sums);
    const int64_t ab = block_scan(add, &total_add, warp_sums);
    fits = __syncthreads_and(fits) && F >= 0 && F + total_given <= t.num_blocks &&
           total_add <= p.slots;
    const bool enough = total_need <= F + total_given;
    const bool ok = fits && enough;
    len_s[tid] = L;
    have_s[tid] = have;
    add_base[tid] = ok ? (int32_t)ab : 0;
    need_base[tid] = ok ? (int32_t)nb : 0;
    given_base[tid] = ok ? (int32_t)gb : 0;
    const int adds = ok ? (int)total_add : 0, takes = ok ? (int)total_need : 0,
              gives = ok ? (int)total_given : 0;
    // this CTA has read the lengths and the state: the last one writes them
    __threadfence();
    __shared__ int last_s;
    __syncthreads();
    if (tid == 0) {
        last_s = 1;
        if (gridDim.x > 1) last_s = atomicAdd(t.state_out + 2, 1) == (int)gridDim.x - 1;
    }
    __syncthreads();
    if (last_s) {
        if (tid < B) {
            t.seq_lens_out[tid] = ok ? (gone ? 0 : (int32_t)end) : L;
            if (p.cu_new) p.cu_new[tid] = add_base[tid];
        }
        if (tid == 0) {
            if (p.cu_new) p.cu_new[B] = adds;
            t.state_out[0] = F + gives - takes;
            t.state_out[1] = old_status ? old_status
                             : ok       ? 0
                                        : (fits ? DA_ENOSPACE : DA_EINVAL);
            t.state_out[2] = 0;
        }
    }

    // the k-th released block, and the k-th block taken
    auto released = [&](int k) {
        const int b = find(given_base, B, k);
        return t.block_table[(size_t)b * t.max_blocks_per_seq + k - given_base[b]];
    };
    auto taken = [&](int k) {
        return k < gives ? released(gives - 1 - k) : t.free_list[F - 1 - (k - gives)];
    };
    const int stride = gridDim.x * kThreads, first = blockIdx.x * kThreads + tid;
    for (int j = first; j < p.slots; j += stride) {
        int64_t slot = -1;
        if (j < adds) {
            const int b = find(add_base, B, j);
            const int pos = len_s[b] + j - add_base[b], i = pos / P;
            const int blk = i < have_s[b]
                                ? t.block_table[(size_t)b * t.max_blocks_per_seq + i]
                                : taken(need_base[b] + i - have_s[b]);
            slot = (int64_t)blk * P + (pos - i * P);
        }
        p.slot_map[j] = slot;
    }
    for (int k = first; k < takes; k += stride) {
        const int b = find(need_base, B, k);
        t.block_table[(size_t)b * t.max_blocks_per_seq + have_s[b] + k - need_base[b]] = taken(k);
    }
    for (int k = first; k < gives - takes; k += stride) t.free_list[F + k] = released(k);
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
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(152 * 4, slot_capacity / kThreads));
    grow_tables_kernel<<<grid, kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
    const cudaError_t e = cudaGetLastError();
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
