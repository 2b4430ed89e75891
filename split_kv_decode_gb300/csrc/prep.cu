// decode_attn_rope_append: what lies between a layer's projections and its attention. For
// every new token t and head h
//     y = x * (mean(x^2) + eps)^-1/2 * (offset + w)           (q and k; optional)
//     z_a = f (y_a cos A_i - y_b sin A_i), z_b = f (y_b cos A_i + y_a sin A_i)
// for the pairs (a, b) = (i, i + rot/2) or (2i, 2i + 1), A_i = position[axis_i] * inv_freq_i;
// columns past rot stay y. q goes to its own rows, k and v into the cache's slots, each
// rounded once.
//
// The angle is taken in whole turns: inv_freq_i / 2 pi as a fraction of 2^64 times the position,
// modulo 2^64, is exact but for the fraction's own rounding (2^-65 of a turn per position),
// so far positions lose nothing and a position costs one integer product. The top 32 bits
// give the octant and the argument of sinpi and cospi.
//
// Bound by memory: each row is read and written once. A row of a head is held by 2 to 32
// lanes, eight columns a lane (16 bytes of a 16-bit type); the sum of squares and the partner
// columns of halved pairs come by shuffles. A CTA forms the sines of its tokens once for all
// heads.
#include <algorithm>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "ptx.cuh"

namespace skv {
int set_error(int code, const char *phase, const char *msg); // api.cpp
}

using skv::griddep_launch_dependents;
using skv::griddep_wait;

namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = DA_MAX_ROT_PAIRS;
constexpr int kMaxTokens = 8; // tokens of a CTA

struct PrepParams {
    const void *q, *k, *v;
    void *q_out, *k_pool, *v_pool;
    const void *q_weight, *k_weight;
    const int64_t *positions, *slot_map;
    const uint64_t *turns;
    int64_t q_stride, q_head, k_stride, k_head, v_stride, v_head; // elements
    int64_t qo_stride, qo_head;
    int64_t kb, kp, kh, vb, vp, vh;
    int64_t qw_head, kw_head;
    int64_t slots; // of the pools
    int32_t tokens, hq, hkv, units_k, units_v; // 8-column units of a q/k and of a v row
    int32_t block_size, pairs, interleaved;
    int32_t q_dtype, cache_dtype, w_dtype;
    int32_t norm;
    int32_t lanes, per_cta, shares; // lanes of a row; tokens of a CTA; CTAs that share them
    float eps, offset, factor, inv_dim;
    uint8_t axis[kMaxPairs];
};

// eight consecutive elements, widened
__device__ __forceinline__ void load8(const float *p, float *f)
{
    const float4 a = *reinterpret_cast<const float4 *>(p);
    const float4 b = *reinterpret_cast<const float4 *>(p + 4);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ void load8(const __half *p, float *f)
{
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        f[2 * i] = x.x;
        f[2 * i + 1] = x.y;
    }
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float *f)
{
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void load8(const void *base, int dtype, int64_t at, float *f)
{
    if (dtype == DA_F32) load8(static_cast<const float *>(base) + at, f);
    else if (dtype == DA_F16) load8(static_cast<const __half *>(base) + at, f);
    else load8(static_cast<const __nv_bfloat16 *>(base) + at, f);
}

__device__ __forceinline__ void store8(void *base, int dtype, int64_t at, const float *f)
{
    if (dtype == DA_F32) {
        float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(base) + at);
        p[0] = make_float4(f[0], f[1], f[2], f[3]);
        p[1] = make_float4(f[4], f[5], f[6], f[7]);
        return;
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (dtype == DA_F16) {
            const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(base) + at) =
        make_uint4(w[0], w[1], w[2], w[3]);
}

// cosine and sine of `phase` * 2^-64 turns
__device__ __forceinline__ float2 unit(uint64_t phase)
{
    const uint32_t top = (uint32_t)(phase >> 32);
    const uint32_t quarter = (top + (1u << 29)) >> 30; // nearest quarter turn
    // the rest, within an eighth of a turn, in half turns
    const float x = (float)(int32_t)(top - (quarter << 30)) * 0x1p-31f;
    const float s = sinpif(x), c = cospif(x);
    switch (quarter & 3) {
    case 0: return make_float2(c, s);
    case 1: return make_float2(-s, c);
    case 2: return make_float2(-c, -s);
    default: return make_float2(s, -c);
    }
}

template <typename ST>
__global__ void __launch_bounds__(kThreads) prep_kernel(const __grid_constant__ PrepParams p)
{
    __shared__ float2 sm_unit[kMaxTokens][kMaxPairs];
    __shared__ int64_t sm_k[kMaxTokens], sm_v[kMaxTokens]; // offsets of the slots' rows, or -1

    // Nothing is touched before the stream's last kernel has ended; the next one may set
    // itself up from then on.
    griddep_wait();
    griddep_launch_dependents();

    const int group = blockIdx.x / p.shares, share = blockIdx.x - group * p.shares;
    const int t0 = group * p.per_cta;
    const int nt = min(p.per_cta, p.tokens - t0);
    for (int i = threadIdx.x; i < nt * p.pairs; i += kThreads) {
        const int t = i / p.pairs, j = i - t * p.pairs;
        const int64_t pos = p.positions[(int64_t)p.axis[j] * p.tokens + t0 + t];
        float2 u = unit((uint64_t)pos * p.turns[j]);
        u.x *= p.factor;
        u.y *= p.factor;
        sm_unit[t][j] = u;
    }
    if (threadIdx.x < nt) {
        const int t = t0 + threadIdx.x;
        const int64_t slot = p.slot_map ? p.slot_map[t] : t;
        int64_t k = -1, v = -1;
        if (slot >= 0 && slot < p.slots) {
            const int64_t blk = slot / p.block_size, at = slot - blk * p.block_size;
            k = blk * p.kb + at * p.kp;
            v = blk * p.vb + at * p.vp;
        }
        sm_k[threadIdx.x] = k;
        sm_v[threadIdx.x] = v;
    }
    __syncthreads();

    // rows (token, head): q heads, then k heads, then v heads
    const int heads = p.hq + 2 * p.hkv;
    const int sub = threadIdx.x & (p.lanes - 1), row0 = threadIdx.x / p.lanes;
    const int step = kThreads / p.lanes;
    const int half_units = p.pairs >> 3; // units of the first half of halved pairs
    const int rows = nt * heads;
    // every lane of a warp takes part in each round's shuffles
    for (int r0 = share * step; r0 < rows; r0 += p.shares * step) {
        const int r = r0 + row0;
        const bool live = r < rows;
        const int t = live ? r / heads : 0;
        const int h = live ? r - t * heads : 0;
        const bool is_v = h >= p.hq + p.hkv, is_k = h >= p.hq && !is_v;
        const bool mine = live && sub < (is_v ? p.units_v : p.units_k);
        const int hh = h - (is_v ? p.hq + p.hkv : is_k ? p.hq : 0);
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0.f;
        if (mine) {
            const int64_t tt = t0 + t;
            const ST *src = is_v   ? static_cast<const ST *>(p.v) + tt * p.v_stride + hh * p.v_head
                            : is_k ? static_cast<const ST *>(p.k) + tt * p.k_stride + hh * p.k_head
                                   : static_cast<const ST *>(p.q) + tt * p.q_stride + hh * p.q_head;
            load8(src + sub * 8, x);
        }
        if (p.norm) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
            for (int o = p.lanes >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (mine && !is_v) {
                const float inv = 1.f / sqrtf(fmaf(ss, p.inv_dim, p.eps));
                const void *w = is_k ? p.k_weight : p.q_weight;
                float g[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) g[i] = 1.f;
                if (w) {
                    load8(w, p.w_dtype, hh * (is_k ? p.kw_head : p.qw_head) + sub * 8, g);
#pragma unroll
                    for (int i = 0; i < 8; ++i) g[i] += p.offset;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * g[i];
            }
        }
        if (p.interleaved) {
            if (mine && !is_v && sub < 2 * half_units) {
                const float2 *u = sm_unit[t] + sub * 4;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float a = x[2 * i], b = x[2 * i + 1];
                    x[2 * i] = a * u[i].x - b * u[i].y;
                    x[2 * i + 1] = b * u[i].x + a * u[i].y;
                }
            }
        } else {
            const bool second = sub >= half_units;
            const bool turns = !is_v && sub < 2 * half_units;
            const int other = (threadIdx.x & 31) + (turns ? (second ? -half_units : half_units) : 0);
            const float2 *u = sm_unit[t] + (second ? sub - half_units : sub) * 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float y = __shfl_sync(0xffffffffu, x[i], other);
                if (turns) x[i] = x[i] * u[i].x + (second ? y * u[i].y : -y * u[i].y);
            }
        }
        if (!mine) continue;
        if (is_v) {
            if (sm_v[t] >= 0) store8(p.v_pool, p.cache_dtype, sm_v[t] + hh * p.vh + sub * 8, x);
        } else if (is_k) {
            if (sm_k[t] >= 0) store8(p.k_pool, p.cache_dtype, sm_k[t] + hh * p.kh + sub * 8, x);
        } else {
            store8(p.q_out, p.q_dtype, (int64_t)(t0 + t) * p.qo_stride + hh * p.qo_head + sub * 8, x);
        }
    }
}

int bad(const char *msg) { return skv::set_error(DA_EINVAL, "rope_append", msg); }

int size_of(int dt) { return dt == DA_F32 ? 4 : dt == DA_F16 || dt == DA_BF16 ? 2 : 0; }

bool off(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

} // namespace

extern "C" int decode_attn_rope_append(const da_prep_t *a, const da_rope_t *rope, const void *q,
                                       const void *k, const void *v, const int64_t *positions,
                                       const int64_t *slot_map, void *q_out, void *k_pool,
                                       void *v_pool, da_stream_t stream)
{
    if (!a || !rope) return bad("shapes or rope is NULL");
    if (a->n_tokens < 0 || a->n_tokens > 1 << 30) return bad("n_tokens must be in [0, 2^30]");
    if (a->n_heads < 1 || a->n_heads > 65535 || a->n_kv_heads < 1 || a->n_kv_heads > 65535)
        return bad("n_heads and n_kv_heads must be in [1, 65535]");
    for (int d : {a->head_dim, a->v_dim})
        if (d < 8 || d > 256 || d % 8)
            return bad("head_dim and v_dim must be multiples of 8 in [8, 256]");
    if (a->block_size < 1 || a->num_blocks < 1) return bad("block_size and num_blocks must be >= 1");
    for (int dt : {a->src_dtype, a->q_dtype, a->cache_dtype})
        if (!size_of(dt)) return bad("types must be DA_F32, DA_F16 or DA_BF16");
    if (rope->rot_dim < 0 || rope->rot_dim % 16 || rope->rot_dim > a->head_dim)
        return bad("rot_dim must be a multiple of 16, at most head_dim");
    if (rope->n_axes < 1 || rope->n_axes > DA_MAX_ROT_AXES) return bad("n_axes must be in [1, 8]");
    for (int i = 0; i < rope->rot_dim / 2; ++i)
        if (rope->axis[i] >= rope->n_axes) return bad("a frequency's axis must be below n_axes");
    if (!(rope->factor == rope->factor) || rope->factor - rope->factor != 0.f)
        return bad("factor must be finite");
    if (a->norm != 0 && a->norm != 1) return bad("norm must be 0 or 1");
    if (a->norm) {
        if (!(a->eps >= 0.f) || a->eps - a->eps != 0.f) return bad("eps must be finite and >= 0");
        if (a->weight_offset - a->weight_offset != 0.f) return bad("weight_offset must be finite");
        if (a->q_weight || a->k_weight) {
            const int ws = size_of(a->w_dtype);
            if (!ws) return bad("w_dtype must be DA_F32, DA_F16 or DA_BF16");
            if (off(a->q_weight, 16) || off(a->k_weight, 16))
                return bad("weights must be 16-byte aligned");
            for (int64_t s : {a->q_weight_head_stride, a->k_weight_head_stride})
                if (s < 0 || (s * ws) % 16)
                    return bad("weight strides must be multiples of 16 bytes, >= 0");
        }
    }
    const int ss = size_of(a->src_dtype), qs = size_of(a->q_dtype), cs = size_of(a->cache_dtype);
    for (int64_t s : {a->q_src_stride, a->q_src_head_stride, a->k_src_stride, a->k_src_head_stride,
                      a->v_src_stride, a->v_src_head_stride})
        if (s < 0 || (s * ss) % 16) return bad("source strides must be multiples of 16 bytes, >= 0");
    for (int64_t s : {a->q_out_stride, a->q_out_head_stride})
        if (s < 1 || (s * qs) % 16)
            return bad("strides of q_out must be positive multiples of 16 bytes");
    for (int64_t s : {a->k_block_stride, a->k_pos_stride, a->k_head_stride, a->v_block_stride,
                      a->v_pos_stride, a->v_head_stride})
        if (s < 1 || (s * cs) % 16) return bad("pool strides must be positive multiples of 16 bytes");
    if (a->n_tokens == 0) return DA_OK;
    if (!q || !k || !v || !q_out || !k_pool || !v_pool) return bad("a tensor pointer is NULL");
    if (rope->rot_dim && (!rope->turns || !positions)) return bad("turns or positions is NULL");
    if (off(q, 16) || off(k, 16) || off(v, 16) || off(q_out, 16) || off(k_pool, 16) ||
        off(v_pool, 16))
        return bad("rows and pools must be 16-byte aligned");
    if (off(positions, 8) || off(slot_map, 8) || off(rope->turns, 8))
        return bad("positions, slot_map and turns must be aligned to their elements");
    const cudaError_t pre = cudaGetLastError();
    if (pre != cudaSuccess)
        return skv::set_error(DA_ECUDA, "before rope_append", cudaGetErrorString(pre));

    PrepParams p;
    p.q = q; p.k = k; p.v = v;
    p.q_out = q_out; p.k_pool = k_pool; p.v_pool = v_pool;
    p.q_weight = a->q_weight; p.k_weight = a->k_weight;
    p.positions = positions; p.slot_map = slot_map; p.turns = rope->turns;
    p.q_stride = a->q_src_stride; p.q_head = a->q_src_head_stride;
    p.k_stride = a->k_src_stride; p.k_head = a->k_src_head_stride;
    p.v_stride = a->v_src_stride; p.v_head = a->v_src_head_stride;
    p.qo_stride = a->q_out_stride; p.qo_head = a->q_out_head_stride;
    p.kb = a->k_block_stride; p.kp = a->k_pos_stride; p.kh = a->k_head_stride;
    p.vb = a->v_block_stride; p.vp = a->v_pos_stride; p.vh = a->v_head_stride;
    p.qw_head = a->q_weight_head_stride; p.kw_head = a->k_weight_head_stride;
    p.slots = (int64_t)a->num_blocks * a->block_size;
    p.tokens = a->n_tokens; p.hq = a->n_heads; p.hkv = a->n_kv_heads;
    p.units_k = a->head_dim / 8; p.units_v = a->v_dim / 8;
    p.block_size = a->block_size;
    p.pairs = rope->rot_dim / 2;
    p.interleaved = rope->interleaved != 0;
    p.q_dtype = a->q_dtype; p.cache_dtype = a->cache_dtype; p.w_dtype = a->w_dtype;
    p.norm = a->norm;
    p.eps = a->eps; p.offset = a->weight_offset; p.factor = rope->factor;
    p.inv_dim = 1.f / (float)a->head_dim;
    for (int i = 0; i < kMaxPairs; ++i) p.axis[i] = i < p.pairs ? rope->axis[i] : 0;
    p.lanes = 1;
    while (p.lanes < std::max(p.units_k, p.units_v)) p.lanes *= 2;
    // Tokens of a CTA: as many as fill its threads once. Few tokens: several CTAs share
    // one token's heads, so that each thread has one row's unit to wait for.
    const int step = kThreads / p.lanes, heads = p.hq + 2 * p.hkv;
    p.per_cta = std::min(std::max(step / heads, 1), kMaxTokens);
    p.shares = 1;
    const int groups = (p.tokens + p.per_cta - 1) / p.per_cta;
    const int rounds = (p.per_cta * heads + step - 1) / step;
    while (p.shares * 2 <= rounds && (int64_t)groups * p.shares * 2 <= 1216) p.shares *= 2;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const unsigned grid = (unsigned)(groups * p.shares);
    const cudaError_t e =
        a->src_dtype == DA_F32   ? skv::launch_after(prep_kernel<float>, grid, kThreads, st, p)
        : a->src_dtype == DA_F16 ? skv::launch_after(prep_kernel<__half>, grid, kThreads, st, p)
                                 : skv::launch_after(prep_kernel<__nv_bfloat16>, grid, kThreads, st, p);
    if (e != cudaSuccess) return skv::set_error(DA_ELAUNCH, "rope_append", cudaGetErrorString(e));
    return DA_OK;
}
