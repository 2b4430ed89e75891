// GQA / MQA split kernel over an 8-bit paged cache, sm_103a.
//
// The codes of a page (block i of block_size positions) stand for code *
// scale[i][head], so with e4m3 or e5m2 codes Kc, Vc and page scales ks, vs
//     score[r][pos] = scale * ks[page(pos)] * sum_d q[r][d] Kc[pos][d]
//     out[r][d]     = sum_pos softmax(score)[r][pos] * vs[page(pos)] * Vc[pos][d].
// An item is (sequence, KV head, split, row group), as for the SIMT kernel. One
// warp takes one position at a time, its lanes the columns.
#include <climits>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "gqa_split.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace skv {
namespace {

constexpr int kWarps = 4;

template <__nv_fp8_interpretation_t F, int D>
__global__ void __launch_bounds__(kWarps * 32)
    gqa_8bit_kernel(const __grid_constant__ Q8Pools pools, const __grid_constant__ Scales8 sc,
                    const __grid_constant__ SplitParams p)
{
    constexpr int E = D / 32; // columns of a lane
    __shared__ float red[kWarps][kQ8Rows][D];
    __shared__ float2 red_ml[kWarps][kQ8Rows];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const ItemTable &it = p.items;
    const int Gh = p.hq / it.n_kv_heads, rows = Gh * p.q_len;
    const int per = (rows + it.row_groups - 1) / it.row_groups;
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
    for (int item = blockIdx.x; item < it.n_items; item += gridDim.x) {
        int b, kvh, s, rg;
        decode_item(it, item, b, kvh, s, rg);
        const int L = p.dev_lens ? max(0, min(__ldg(p.dev_lens + b), it.seq_lens[b]))
                                 : it.seq_lens[b];
        const int p0 = s * it.chunk[b], p1 = min(L, p0 + it.chunk[b]);
        const int row0 = rg * per, R = min(per, rows - row0);
        float q[kQ8Rows][E], acc[kQ8Rows][E], m[kQ8Rows], l[kQ8Rows];
        int lim[kQ8Rows]; // positions row r sees: below lim
        for (int r = 0; r < kQ8Rows; ++r) {
            m[r] = kNeutralM;
            l[r] = 0.f;
            lim[r] = 0;
            const int tok = (row0 + r) / Gh, g = (row0 + r) - tok * Gh;
            if (r < R)
                lim[r] = (p.flags & DA_FLAG_NO_CAUSAL) ? INT_MAX : L - p.q_len + 1 + tok;
            for (int e = 0; e < E; ++e) {
                acc[r][e] = 0.f;
                q[r][e] = r < R ? p.q[((size_t)(b * p.q_len + tok) * p.hq + kvh * Gh + g) * D +
                                      lane * E + e] * p.scale_log2
                                : 0.f;
            }
        }
        for (int pos = p0 + warp; pos < p1; pos += kWarps) {
            const int i = pos / p.block_size;
            const int blk = p.block_table[(size_t)b * p.max_blocks + i];
            float k[E], v[E], ks = 0.f, vs = 0.f;
            for (int e = 0; e < E; ++e) k[e] = v[e] = 0.f;
            if (blk >= 0 && blk < sc.num_blocks) {
                const int o = pos - i * p.block_size;
                const uint8_t *kr = pools.k + blk * pools.k_block + o * pools.k_pos + kvh * pools.k_head;
                const uint8_t *vr = pools.v + blk * pools.v_block + o * pools.v_pos + kvh * pools.v_head;
                ks = sc.k[blk * sc.k_block + kvh * sc.k_head];
                vs = sc.v[blk * sc.v_block + kvh * sc.v_head];
                for (int e = 0; e < E; ++e) {
                    k[e] = __half2float(__half(__nv_cvt_fp8_to_halfraw(kr[lane * E + e], F)));
                    v[e] = __half2float(__half(__nv_cvt_fp8_to_halfraw(vr[lane * E + e], F)));
                }
            }
            for (int r = 0; r < kQ8Rows; ++r) {
                float d = 0.f;
                for (int e = 0; e < E; ++e) d = fmaf(q[r][e], k[e], d);
                for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
                d *= ks;
                if (pos < lim[r]) {
                    const float mn = fmaxf(m[r], d), f = ex2(m[r] - mn), w = ex2(d - mn);
                    m[r] = mn;
                    l[r] = l[r] * f + w;
                    for (int e = 0; e < E; ++e) acc[r][e] = acc[r][e] * f + w * vs * v[e];
                }
            }
        }
        for (int r = 0; r < kQ8Rows; ++r) {
            for (int e = 0; e < E; ++e) red[warp][r][lane * E + e] = acc[r][e];
            if (lane == 0) red_ml[warp][r] = make_float2(m[r], l[r]);
        }
        __syncthreads();
        for (int i = threadIdx.x; i < R * D; i += kWarps * 32) {
            const int r = i / D, d = i - r * D;
            float M = kNeutralM, A = 0.f, S = 0.f;
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, red_ml[w][r].x);
            for (int w = 0; w < kWarps; ++w) {
                const float f = ex2(red_ml[w][r].x - M);
                S += red_ml[w][r].y * f;
                A += red[w][r][d] * f;
            }
            const int tok = (row0 + r) / Gh, g = (row0 + r) - tok * Gh;
            const size_t wr = ((size_t)it.split_base[b] + s) * p.n_heads + kvh * Gh + tok * p.hq + g;
            // a NaN score makes the row NaN whatever the other splits hold
            const bool nan = isnan(S);
            p.acc[wr * D + d] = nan ? S : A;
            if (d == 0)
                p.ml[wr] = nan ? make_float2(-kNeutralM, 1.f)
                               : make_float2(S > 0.f ? M * kLn2 : kNeutralM, S);
        }
        __syncthreads();
    }
}

template <__nv_fp8_interpretation_t F, int D>
cudaError_t launch_t(int grid, cudaStream_t st, const Q8Pools &pools, const Scales8 &sc,
                     const SplitParams &p)
{
    gqa_8bit_kernel<F, D><<<grid, kWarps * 32, 0, st>>>(pools, sc, p);
    return cudaGetLastError();
}

} // namespace

int q8_rows_per_item(int rows)
{
    const int groups = (rows + kQ8Rows - 1) / kQ8Rows;
    return (rows + groups - 1) / groups;
}

cudaError_t launch_gqa_8bit(int code_dtype, int head_dim, int grid, cudaStream_t st,
                            const Q8Pools &pools, const Scales8 &sc, const SplitParams &p)
{
    if (head_dim == 128)
        return code_dtype == DA_E4M3 ? launch_t<__NV_E4M3, 128>(grid, st, pools, sc, p)
                                     : launch_t<__NV_E5M2, 128>(grid, st, pools, sc, p);
    return code_dtype == DA_E4M3 ? launch_t<__NV_E4M3, 256>(grid, st, pools, sc, p)
                                 : launch_t<__NV_E5M2, 256>(grid, st, pools, sc, p);
}

} // namespace skv
