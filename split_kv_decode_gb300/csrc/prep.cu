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
// Bound by memory: each row is read and written once. A warp holds one token (or 2 to 32 of
// narrow heads) and walks its heads, or a share of them; a lane holds both columns of four or eight
// pairs of every head, so that it needs four or eight angles a token, no exchange but the sum of
// squares, and q may be rotated in place. Two rows are worked on side by side while the next two are
// in flight: a row is a chain of a sum over the lanes, a root and two products, and its instructions
// bound it beside the memory. (32768 tokens of 16/4 heads of 256 columns, f16: 141 us, 5.7 TB/s; with 8
// columns a lane instead of 16 174, one row at a time 200; four rows in flight 146, fewer registers
// 212 and more. 9999 tokens of 8/2 heads of 128, f32: 26 us, 4.3 TB/s; with four rows in flight 30.)
#include <algorithm>
#include <cstring>
#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"

namespace skv {
int set_error(int code, const char *phase, const char *msg); // api.cpp
}

namespace {

constexpr int kThreads = 128;
constexpr int kAhead = 2; // rows of a warp in flight
constexpr int kFull = 1216; // warps: eight an SM
constexpr int kMaxPairs = DA_MAX_ROT_PAIRS;

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
    int32_t tokens, hq, hkv, units_k, units_v; // lanes of a q/k and of a v row
    int32_t block_size, pairs, interleaved;
    int32_t q_dtype, cache_dtype, w_dtype;
    int32_t q_size, cache_size; // bytes of an element
    int32_t lanes, shares; // lanes of a row; warps that share a token's heads
    float eps, offset, factor, inv_dim;
    uint8_t axis[kMaxPairs];
};

// twice H consecutive elements, as they are stored
template <typename ST, int H> struct Raw {
    static constexpr int WORDS = H * (int)sizeof(ST) / 4; // of a half: 2 or 4
    using V = typename std::conditional<WORDS == 2, uint2, uint4>::type;
    V a, b;
};
template <typename ST, int H>
__device__ __forceinline__ void load(Raw<ST, H> &r, const ST *first, int second)
{
    using V = typename Raw<ST, H>::V;
    r.a = *reinterpret_cast<const V *>(first);
    r.b = *reinterpret_cast<const V *>(first + second);
}
// a word's elements (two, or one f32)
template <typename ST> __device__ __forceinline__ float2 widen2(uint32_t w);
template <> __device__ __forceinline__ float2 widen2<__half>(uint32_t w)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
template <> __device__ __forceinline__ float2 widen2<__nv_bfloat16>(uint32_t w)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
// N elements from `at` on
template <typename ST, int N> __device__ __forceinline__ void widen(const uint32_t *w, float2 *f)
{
    if constexpr (sizeof(ST) == 4) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i)
            f[i] = make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    } else {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) f[i] = widen2<ST>(w[i]);
    }
}
template <typename ST, int H> __device__ __forceinline__ void widen(const Raw<ST, H> &r, float2 *f)
{
    uint32_t a[Raw<ST, H>::WORDS], b[Raw<ST, H>::WORDS];
    memcpy(a, &r.a, sizeof a);
    memcpy(b, &r.b, sizeof b);
    widen<ST, H>(a, f);
    widen<ST, H>(b, f + H / 2);
}
// four elements at a time
template <typename WT, int H>
__device__ __forceinline__ void load_as(const void *base, int64_t at, int second, float2 *f)
{
    const WT *w = static_cast<const WT *>(base) + at;
#pragma unroll
    for (int i = 0; i < H; i += 4)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint32_t x[sizeof(WT)];
            typename Raw<WT, 4>::V v =
                *reinterpret_cast<const typename Raw<WT, 4>::V *>(w + (k ? second : 0) + i);
            memcpy(x, &v, sizeof x);
            widen<WT, 4>(x, f + k * (H / 2) + i / 2);
        }
}

// twice H elements, rounded, to `first` and to `second` elements behind it
template <int H>
__device__ __forceinline__ void store(uint8_t *first, int dtype, int second, const float2 *f)
{
    if (dtype == DA_F32) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < H; i += 4) {
                const float2 x = f[k * (H / 2) + i / 2], y = f[k * (H / 2) + i / 2 + 1];
                *reinterpret_cast<float4 *>(first + ((k ? second : 0) + i) * 4) =
                    make_float4(x.x, x.y, y.x, y.y);
            }
        return;
    }
    uint32_t w[H];
    if (dtype == DA_F16) {
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const __half2 h = __floats2half2_rn(f[i].x, f[i].y);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    } else {
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[i].x, f[i].y);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    using V = typename std::conditional<H == 4, uint2, uint4>::type;
    V x, y;
    memcpy(&x, w, sizeof x);
    memcpy(&y, w + H / 2, sizeof y);
    *reinterpret_cast<V *>(first) = x;
    *reinterpret_cast<V *>(first + second * 2) = y;
}

// a^-1/2: the special function's, and one Newton step, which leaves the last rounding
__device__ __forceinline__ float inv_root(float a)
{
    const float y = rsqrtf(a);
    const float z = fmaf(0.5f * y, fmaf(-a * y, y, 1.f), y);
    return a > 0.f && a < INFINITY ? z : y;
}

// cosine and sine of `phase` * 2^-64 turns
__device__ __forceinline__ float2 unit(uint64_t phase)
{
    const uint32_t top = (uint32_t)(phase >> 32);
    const uint32_t quarter = (top + (1u << 29)) >> 30; // nearest quarter turn
    // the rest, within an eighth of a turn, in half turns
    const float x = (float)(int32_t)(top - (quarter << 30)) * 0x1p-31f;
    const float s = sinpif(x), c = cospif(x);
    const float a = quarter & 1 ? s : c, b = quarter & 1 ? c : s;
    return make_float2((quarter + 1) & 2 ? -a : a, quarter & 2 ? -b : b);
}

template <typename ST, bool NORM, int H>
__global__ void __launch_bounds__(kThreads, H == 4 ? 5 : 4) prep_kernel(const __grid_constant__ PrepParams p)
{
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t group = w / p.shares;
    const int share = (int)(w - group * p.shares);
    const int64_t t = group * (32 / p.lanes) + lane / p.lanes;
    const bool live = t < p.tokens;
    const int sub = lane & (p.lanes - 1);
    const int hk = p.hq, hv = p.hq + p.hkv, heads = hv + p.hkv; // the first k and v row
    const int h0 = (int)((int64_t)share * heads / p.shares);
    const int h1 = (int)((int64_t)(share + 1) * heads / p.shares);
    const int turning = p.pairs / H; // lanes that hold pairs
    const bool turns = sub < turning;
    // the lane's columns: both of H pairs, or 2 H in a row (those of a value row always)
    const bool halves = turns && !p.interleaved;
    const int ca = halves ? sub * H : sub * 2 * H, apart = halves ? p.pairs : H, va = sub * 2 * H;
    const bool has_k = live && sub < p.units_k, has_v = live && sub < p.units_v;

    // the next row to load: the lane's first columns, and where a row ends and another tensor starts
    const ST *src;
    int64_t step;
    int f = h0, second = apart;
    bool has = has_k;
    auto source = [&](int h) {
        if (h >= hv) {
            src = static_cast<const ST *>(p.v) + t * p.v_stride + (h - hv) * p.v_head + va;
            step = p.v_head;
            second = H;
            has = has_v;
        } else if (h >= hk) {
            src = static_cast<const ST *>(p.k) + t * p.k_stride + (h - hk) * p.k_head + ca;
            step = p.k_head;
        } else {
            src = static_cast<const ST *>(p.q) + t * p.q_stride + h * p.q_head + ca;
            step = p.q_head;
        }
    };
    source(h0);
    Raw<ST, H> raw[kAhead] = {};
    auto fetch = [&](Raw<ST, H> &r) {
        if (has) load(r, src, second);
        ++f;
        src += step;
        if (f == hk || f == hv) source(f);
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (h0 + i < h1) fetch(raw[i]);

    int64_t k_at = -1, v_at = -1; // the slot's rows
    float2 cs[H / 2], sn[H / 2];  // cosines and sines of two pairs each
#pragma unroll
    for (int i = 0; i < H / 2; ++i) {
        cs[i] = make_float2(1.f, 1.f);
        sn[i] = make_float2(0.f, 0.f);
    }
    if (live) {
        const int64_t slot = p.slot_map ? p.slot_map[t] : t;
        if (slot >= 0 && slot < p.slots) {
            const int64_t blk = p.slots <= UINT32_MAX ? (uint32_t)slot / (uint32_t)p.block_size
                                                      : slot / p.block_size;
            const int64_t at = slot - blk * p.block_size;
            k_at = blk * p.kb + at * p.kp;
            v_at = blk * p.vb + at * p.vp;
        }
        if (turns && h0 < hv) {
            auto turn_of = [&](int j) {
                const int64_t pos = p.positions[(int64_t)p.axis[j] * p.tokens + t];
                const float2 u = unit((uint64_t)pos * p.turns[j]);
                return make_float2(u.x * p.factor, u.y * p.factor);
            };
#pragma unroll
            for (int i = 0; i < H / 2; ++i) {
                const float2 x = turn_of(sub * H + 2 * i), y = turn_of(sub * H + 2 * i + 1);
                cs[i] = make_float2(x.x, y.x);
                sn[i] = make_float2(x.y, y.y);
            }
        }
    }
    // the row to write, in bytes
    uint8_t *dst;
    int64_t to_next;
    int dtype, apart_to;
    bool writes;
    auto target = [&](int h) {
        if (h < hk) {
            dst = static_cast<uint8_t *>(p.q_out) + (t * p.qo_stride + h * p.qo_head + ca) * p.q_size;
            to_next = p.qo_head * p.q_size;
            dtype = p.q_dtype;
            writes = has_k;
        } else if (h < hv) {
            dst = static_cast<uint8_t *>(p.k_pool) + (k_at + (h - hk) * p.kh + ca) * p.cache_size;
            to_next = p.kh * p.cache_size;
            dtype = p.cache_dtype;
            writes = has_k && k_at >= 0;
        } else {
            dst = static_cast<uint8_t *>(p.v_pool) + (v_at + (h - hv) * p.vh + va) * p.cache_size;
            to_next = p.vh * p.cache_size;
            dtype = p.cache_dtype;
            writes = has_v && v_at >= 0;
        }
        apart_to = h < hv ? apart : H;
    };
    // the norm's weights of a head
    float2 g[H];
    const void *weight = nullptr;
    int64_t weight_at = 0, weight_step = 0;
    auto weights = [&]() {
#pragma unroll
        for (int i = 0; i < H; ++i) g[i] = make_float2(1.f, 1.f);
        if (weight && has_k) {
            if (p.w_dtype == DA_F32) load_as<float, H>(weight, weight_at, apart, g);
            else if (p.w_dtype == DA_F16) load_as<__half, H>(weight, weight_at, apart, g);
            else load_as<__nv_bfloat16, H>(weight, weight_at, apart, g);
            const float2 offset = make_float2(p.offset, p.offset);
#pragma unroll
            for (int i = 0; i < H; ++i) g[i] = __fadd2_rn(g[i], offset);
        }
    };
    auto norm_of = [&](int h) { // from row h on
        const bool is_k = h >= hk;
        weight = is_k ? p.k_weight : p.q_weight;
        weight_step = is_k ? p.kw_head : p.qw_head;
        weight_at = (is_k ? h - hk : h) * weight_step + ca;
        weights();
    };

    // normalised and turned: N rows' columns (0 1), (2 3) .. of the lane's first H and its second H
    auto turn = [&](auto count, float2 (*x)[H]) {
        constexpr int N = decltype(count)::value;
        if (NORM) {
            float sum[N];
#pragma unroll
            for (int k = 0; k < N; ++k) {
                float2 ss = __fmul2_rn(x[k][0], x[k][0]);
#pragma unroll
                for (int i = 1; i < H; ++i) ss = __ffma2_rn(x[k][i], x[k][i], ss);
                sum[k] = ss.x + ss.y;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                if (o >= p.lanes) continue;
#pragma unroll
                for (int k = 0; k < N; ++k) sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], o);
            }
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const float inv = inv_root(fmaf(sum[k], p.inv_dim, p.eps));
                const float2 inv2 = make_float2(inv, inv);
#pragma unroll
                for (int i = 0; i < H; ++i) x[k][i] = __fmul2_rn(__fmul2_rn(x[k][i], inv2), g[i]);
            }
        }
        if (!turns) return;
        if (p.interleaved) {
#pragma unroll
            for (int k = 0; k < N; ++k)
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    const float2 z = x[k][i];
                    const float c = i & 1 ? cs[i / 2].y : cs[i / 2].x;
                    const float s = i & 1 ? sn[i / 2].y : sn[i / 2].x;
                    x[k][i] = make_float2(z.x * c - z.y * s, z.y * c + z.x * s);
                }
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k)
#pragma unroll
                for (int i = 0; i < H / 2; ++i) {
                    const float2 y = x[k][i], z = x[k][i + H / 2], minus = make_float2(-sn[i].x, -sn[i].y);
                    x[k][i] = __ffma2_rn(z, minus, __fmul2_rn(y, cs[i]));
                    x[k][i + H / 2] = __ffma2_rn(y, sn[i], __fmul2_rn(z, cs[i]));
                }
        }
    };
    // behind `row` and before the next one
    auto advance = [&](int row) {
        dst += to_next;
        const int next = row + 1;
        if (next == hk || next == hv) {
            target(next);
            if (NORM && next == hk && next < h1) norm_of(next);
        } else if (NORM && weight_step && next < hv) {
            weight_at += weight_step;
            weights();
        }
    };

    target(h0);
    if (NORM && h0 < hv) norm_of(h0);
    for (int h = h0; h < h1; h += kAhead) {
#pragma unroll
        for (int i = 0; i < kAhead; i += 2) {
            const int row = h + i;
            if (row >= h1) break;
            float2 y[2][H];
            widen<ST, H>(raw[i], y[0]);
            widen<ST, H>(raw[i + 1], y[1]);
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (f < h1) fetch(raw[i + k]);
            const bool pair = row + 1 < h1 && row + 1 != hk && row + 1 != hv && !(NORM && weight_step);
            if (pair) { // two rows of a tensor: their steps side by side
                if (row < hv) turn(std::integral_constant<int, 2>(), y);
                if (writes) {
                    store<H>(dst, dtype, apart_to, y[0]);
                    store<H>(dst + to_next, dtype, apart_to, y[1]);
                }
                dst += to_next;
                advance(row + 1);
                continue;
            }
#pragma unroll 1
            for (int k = row; k < min(row + 2, h1); ++k) {
                if (k < hv) turn(std::integral_constant<int, 1>(), y);
                if (writes) store<H>(dst, dtype, apart_to, y[0]);
                advance(k);
#pragma unroll
                for (int e = 0; e < H; ++e) y[0][e] = y[1][e];
            }
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
    // lanes of 8 columns, and their warps if each takes whole tokens
    const auto lanes_of = [&](int columns) {
        int n = 1;
        while (n < std::max(a->head_dim, a->v_dim) / columns) n *= 2;
        return n;
    };
    const auto warps_of = [&](int lanes) { return ((int64_t)a->n_tokens * lanes + 31) / 32; };
    // 16 columns a lane (16-byte accesses, and the steps of a row half as often) where rows have whole
    // ones, are of 16 bits and fill the SMs anyway: 32768 tokens of 256 columns take 141 instead of
    // 174 us, but 32 of 128 4.6 instead of 3.8, as a lane turns twice as many pairs
    const bool wide = a->src_dtype != DA_F32 && a->head_dim % 16 == 0 && a->v_dim % 16 == 0 &&
                      warps_of(lanes_of(8)) >= kFull;
    const int columns = wide ? 16 : 8;
    p.units_k = a->head_dim / columns; p.units_v = a->v_dim / columns;
    p.block_size = a->block_size;
    p.pairs = rope->rot_dim / 2;
    p.interleaved = rope->interleaved != 0;
    p.q_dtype = a->q_dtype; p.cache_dtype = a->cache_dtype; p.w_dtype = a->w_dtype;
    p.q_size = qs; p.cache_size = cs;
    p.eps = a->eps; p.offset = a->weight_offset; p.factor = rope->factor;
    p.inv_dim = 1.f / (float)a->head_dim;
    for (int i = 0; i < kMaxPairs; ++i) p.axis[i] = i < p.pairs ? rope->axis[i] : 0;
    p.lanes = lanes_of(columns);
    // Few tokens: several warps share one's heads, down to two heads each, until there are
    // eight warps an SM.
    const int64_t groups = warps_of(p.lanes);
    const int heads = p.hq + 2 * p.hkv;
    p.shares = (int)std::max<int64_t>(1, std::min<int64_t>(heads / 2, kFull / groups));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const unsigned grid = (unsigned)((groups * p.shares + kThreads / 32 - 1) / (kThreads / 32));
    auto launch = [&](auto type, auto half) {
        using ST = decltype(type);
        constexpr int H = decltype(half)::value;
        if (a->norm) prep_kernel<ST, true, H><<<grid, kThreads, 0, st>>>(p);
        else prep_kernel<ST, false, H><<<grid, kThreads, 0, st>>>(p);
    };
    const auto four = std::integral_constant<int, 4>();
    const auto eight = std::integral_constant<int, 8>();
    if (a->src_dtype == DA_F32) launch(0.f, four);
    else if (a->src_dtype == DA_F16 && wide) launch(__half(), eight);
    else if (a->src_dtype == DA_F16) launch(__half(), four);
    else if (wide) launch(__nv_bfloat16(), eight);
    else launch(__nv_bfloat16(), four);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return skv::set_error(DA_ELAUNCH, "rope_append", cudaGetErrorString(e));
    return DA_OK;
}
