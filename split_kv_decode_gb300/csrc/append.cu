// decode_attn_append_8bit: quantise new K/V rows into the pages of an 8-bit cache.
//
// For the new rows of one (block, head), keys or values:
//     a = max |x| over the finite new values, s = 2^e with the least e >= -100
//     for which a <= MAX * 2^e, and at least the block's scale if it has older
//     rows; code = rn(x / s), saturating; older codes c become rn(c * s_old / s)
//     when s > s_old.
// MAX = 1.75 * 2^top (top = 8 for e4m3, 15 for e5m2), so e follows from a's
// exponent and whether its mantissa exceeds 1.75: no division, no logarithm.
#include <algorithm>
#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "internal.h"
#include "ptx.cuh"

namespace skv {
int set_error(int code, const char *phase, const char *msg); // api.cpp
}

using skv::griddep_launch_dependents;
using skv::griddep_wait;
using skv::named_bar_sync;

namespace {

// CTAs of 8 warps for groups of 8, four an SM (64 registers; 36 against 38 us for 32k rows of
// 4 x 256 f16 in pages of 64); otherwise of 4 warps, seven an SM (72 registers), so that
// short calls spread over the SMs and long ones keep 28 warps' loads in flight (126k rows of
// 8 x 128 bf16 in pages of 16: 128 us; five or eight CTAs: 135 and 134 us)
constexpr int warps_of(int G) { return G == 8 ? 8 : 4; }

struct Side { // keys or values; strides in elements
    const void *src;
    uint8_t *pool;
    float *scale;
    int64_t src_stride, src_head, block, pos, head, scale_block, scale_head;
    int32_t units; // 16-element units of a row
};
struct AppendParams {
    Side side[2];
    const int64_t *slot_map;
    int32_t tokens, heads, block_size, shift, num_blocks; // shift: log2 of block_size, or -1
    int32_t chunk;                                        // tokens a group looks after
};

// 16 elements as they are stored
template <typename ST> struct Unit {
    static constexpr int V = sizeof(ST); // 16-byte vectors: 2 or 4
    uint4 v[V];
};
template <typename ST> constexpr int kUnits = 8 / sizeof(ST); // units a thread holds: 128 bytes

// (streamed: rows are read once, and codes of a long prompt are not read back soon;
// evict-first loads and stores took 126k rows of 8 heads from 161 to 151 us)
template <typename ST> __device__ __forceinline__ void load_unit(Unit<ST> &u, const ST *p)
{
#pragma unroll
    for (int i = 0; i < Unit<ST>::V; ++i) u.v[i] = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
}

// Running maximum of |x|, one or two values a word. A maximum drops NaN; an infinity
// stays and sends the run to the slow path.
template <typename ST> struct Top;
template <> struct Top<float> {
    float m = 0.f;
    __device__ __forceinline__ void add(uint32_t w) { m = fmaxf(m, fabsf(__uint_as_float(w))); }
    __device__ __forceinline__ float value() const { return m; }
};
template <> struct Top<__half> {
    __half2 m = __half2(__half(0.f), __half(0.f));
    __device__ __forceinline__ void add(uint32_t w)
    {
        m = __hmax2(m, __habs2(*reinterpret_cast<__half2 *>(&w)));
    }
    __device__ __forceinline__ float value() const
    {
        return fmaxf(__low2float(m), __high2float(m));
    }
};
template <> struct Top<__nv_bfloat16> {
    __nv_bfloat162 m = __nv_bfloat162(__nv_bfloat16(0.f), __nv_bfloat16(0.f));
    __device__ __forceinline__ void add(uint32_t w)
    {
        m = __hmax2(m, __habs2(*reinterpret_cast<__nv_bfloat162 *>(&w)));
    }
    __device__ __forceinline__ float value() const
    {
        return fmaxf(__low2float(m), __high2float(m));
    }
};
template <typename ST> __device__ __forceinline__ void add_unit(Top<ST> &m, const Unit<ST> &u)
{
#pragma unroll
    for (int i = 0; i < Unit<ST>::V; ++i) {
        m.add(u.v[i].x);
        m.add(u.v[i].y);
        m.add(u.v[i].z);
        m.add(u.v[i].w);
    }
}

// a unit's elements in f32
__device__ __forceinline__ void widen(const Unit<float> &u, float *f)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[4 * i] = __uint_as_float(u.v[i].x);
        f[4 * i + 1] = __uint_as_float(u.v[i].y);
        f[4 * i + 2] = __uint_as_float(u.v[i].z);
        f[4 * i + 3] = __uint_as_float(u.v[i].w);
    }
}
__device__ __forceinline__ void widen2(uint32_t w, float *f, __half)
{
    const float2 x = __half22float2(*reinterpret_cast<__half2 *>(&w));
    f[0] = x.x;
    f[1] = x.y;
}
__device__ __forceinline__ void widen2(uint32_t w, float *f, __nv_bfloat16)
{
    f[0] = __uint_as_float(w << 16);
    f[1] = __uint_as_float(w & 0xffff0000u);
}
template <typename ST> __device__ __forceinline__ void widen(const Unit<ST> &u, float *f)
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        widen2(u.v[i].x, f + 8 * i, ST());
        widen2(u.v[i].y, f + 8 * i + 2, ST());
        widen2(u.v[i].z, f + 8 * i + 4, ST());
        widen2(u.v[i].w, f + 8 * i + 6, ST());
    }
}

// the largest finite |x| of a unit (the rare path: something was not finite)
template <typename ST> __device__ __noinline__ float top_finite(Unit<ST> u, float m)
{
    float f[16];
    widen(u, f);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float a = fabsf(f[i]);
        if (a <= 3.402823466e38f) m = fmaxf(m, a);
    }
    return m;
}

// 16 f32 -> 16 codes, saturating, round to nearest even
template <__nv_fp8_interpretation_t F> __device__ __forceinline__ uint4 encode16(const float *f)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i], f[4 * i + 1]),
                                                    __NV_SATFINITE, F);
        const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i + 2], f[4 * i + 3]),
                                                    __NV_SATFINITE, F);
        w[i] = a | (b << 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The codes of a unit under a power-of-two scale (inv: its inverse). f16 is scaled in its own
// type, two elements at a time, where inv is an f16: exact, but for results below 2^-14,
// rounded to 2^-24, which e4m3, whose least step is 2^-9, does not see (e5m2's steps of 2^-16
// could, so it goes through f32).
template <__nv_fp8_interpretation_t F, typename ST>
__device__ __forceinline__ uint4 encode_unit(const Unit<ST> &u, float inv)
{
    constexpr bool kHalf = std::is_same<ST, __half>::value;
    if constexpr (kHalf && F == __NV_E4M3) {
        if (inv >= 6.103515625e-5f && inv <= 32768.f) {
            const __half2 s = __float2half2_rn(inv);
            uint32_t c[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t w = (&u.v[i / 4].x)[i % 4];
                const __half2 y = __hmul2(*reinterpret_cast<const __half2 *>(&w), s);
                c[i] = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(y), __NV_SATFINITE, F);
            }
            return make_uint4(c[0] | (c[1] << 16), c[2] | (c[3] << 16), c[4] | (c[5] << 16),
                              c[6] | (c[7] << 16));
        }
    }
    float f[16];
    widen(u, f);
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] *= inv;
    return encode16<F>(f);
}

// the same under a scale that is no power of two (rare: a page that another quantiser began)
template <__nv_fp8_interpretation_t F, typename ST>
__device__ __noinline__ uint4 encode_divided(Unit<ST> u, float sc)
{
    float f[16];
    widen(u, f);
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] /= sc;
    return encode16<F>(f);
}

template <__nv_fp8_interpretation_t F> __device__ __forceinline__ void decode16(uint4 c, float *f)
{
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const __half2 h(__nv_cvt_fp8x2_to_halfraw2(
            (__nv_fp8x2_storage_t)(w[i / 2] >> (16 * (i & 1))), F));
        const float2 x = __half22float2(h);
        f[2 * i] = x.x;
        f[2 * i + 1] = x.y;
    }
}

// the least e >= -100 with a <= 1.75 * 2^(top + e), as 2^e (a >= 0, finite)
__device__ __forceinline__ float scale_for(float a, int top)
{
    const uint32_t u = __float_as_uint(a);
    const int e = (int)(u >> 23) - 127 - top + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float((uint32_t)(max(e, -100) + 127) << 23);
}

// A group of G warps looks after `chunk` tokens of one head, keys or values: it finds the
// runs that begin among them and writes each (a run is a page's new rows, so nobody else
// touches that page and head). A page that fits the group's registers is read once:
// G follows from the page's size. Every warp of a group finds the runs for itself.
template <typename ST, __nv_fp8_interpretation_t F, int G>
__global__ void __launch_bounds__(32 * warps_of(G), G == 8 ? 4 : 7)
    append_kernel(const __grid_constant__ AppendParams p)
{
    griddep_wait();
    // The attention that follows may set itself up meanwhile. Not before the wait: the kernel
    // after that could then run beside what came before this one.
    griddep_launch_dependents();
    constexpr int TG = 32 * G, kWarps = warps_of(G);
    __shared__ float red[2][kWarps], red_finite[2][kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = warp / G, gt = threadIdx.x - group * TG; // thread of the group
    const int P = p.block_size, T = p.tokens;
    // tasks: head fastest, then keys and values, then chunks
    const uint32_t task = blockIdx.x * (kWarps / G) + group, pair = task / (uint32_t)p.heads;
    const int h = (int)(task - pair * p.heads), kv = (int)(pair & 1);
    const int64_t c0 = (int64_t)(pair >> 1) * p.chunk;
    if (c0 >= T) return; // the whole group
    const int c1 = (int)min((int64_t)T, c0 + p.chunk);
    const Side &sd = p.side[kv];
    const ST *src0 = static_cast<const ST *>(sd.src) + (int64_t)h * sd.src_head;
    const int64_t slots = (int64_t)p.num_blocks * P;
    int parity = 0; // of the reduction buffers

    for (int w0 = (int)c0; w0 < c1; w0 += 32) {
        const int t = w0 + lane;
        const int64_t s = t < T ? p.slot_map[t] : -1;
        int64_t prev = __shfl_up_sync(0xffffffffu, s, 1);
        if (lane == 0) prev = t > 0 ? p.slot_map[t - 1] : -2;
        const bool in = s >= 0 && s < slots;
        const int64_t blk = in ? (p.shift >= 0 ? s >> p.shift : s / P) : 0;
        const int off = (int)(s - blk * P);
        unsigned heads = __ballot_sync(0xffffffffu, t < c1 && in && (off == 0 || prev != s - 1));
        while (heads) {
            const int f = __ffs(heads) - 1;
            heads &= heads - 1;
            // the run: rows at consecutive slots, up to the page's end
            const int t0 = w0 + f, p0 = __shfl_sync(0xffffffffu, off, f);
            const int64_t s0 = __shfl_sync(0xffffffffu, s, f), b0 = __shfl_sync(0xffffffffu, blk, f);
            const int most = min(P - p0, T - t0);
            int n = 0;
            for (;;) {
                const int i = n + lane;
                const bool cont = i < most && p.slot_map[t0 + i] == s0 + i;
                const unsigned stop = ~__ballot_sync(0xffffffffu, cont);
                if (stop) {
                    n += __ffs(stop) - 1;
                    break;
                }
                n += 32;
            }
            float *sp = sd.scale + b0 * sd.scale_block + h * sd.scale_head;
            const float was = p0 > 0 ? *sp : 0.f;
            const ST *src = src0 + (int64_t)t0 * sd.src_stride;
            uint8_t *page = sd.pool + b0 * sd.block + h * sd.head;
            // thread gt takes units gt, gt + TG, ... of the run's n * units
            const int U = sd.units, dr = TG / U, dc = TG - dr * U;
            const int row_first = gt / U, col_first = gt - row_first * U;
            Unit<ST> u[kUnits<ST>];
            Top<ST> most_abs;
            int r = row_first, c = col_first;
            auto step = [&] {
                r += dr;
                c += dc;
                if (c >= U) {
                    c -= U;
                    ++r;
                }
            };
#pragma unroll
            for (int k = 0; k < kUnits<ST>; ++k) {
                if (r < n) load_unit(u[k], src + (int64_t)r * sd.src_stride + 16 * c);
                else
                    for (int i = 0; i < Unit<ST>::V; ++i) u[k].v[i] = make_uint4(0, 0, 0, 0);
                step();
            }
#pragma unroll
            for (int k = 0; k < kUnits<ST>; ++k) add_unit(most_abs, u[k]);
            const int r_rest = r, c_rest = c; // what does not fit the registers
            for (; r < n; step()) {
                Unit<ST> x;
                load_unit(x, src + (int64_t)r * sd.src_stride + 16 * c);
                add_unit(most_abs, x);
            }
            auto reduce = [&](float m, float *buf) { // over the group (magnitudes order as integers)
                m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
                if constexpr (G > 1) {
                    if (lane == 0) buf[warp] = m;
                    named_bar_sync(1 + group, TG);
#pragma unroll
                    for (int w = 0; w < G; ++w) m = fmaxf(m, buf[group * G + w]);
                }
                return m;
            };
            float amax = reduce(most_abs.value(), red[parity]);
            if (amax > 3.402823466e38f) { // an infinity (the same for the whole group)
                amax = 0.f;
#pragma unroll
                for (int k = 0; k < kUnits<ST>; ++k) amax = top_finite(u[k], amax);
                for (r = r_rest, c = c_rest; r < n; step()) {
                    Unit<ST> x;
                    load_unit(x, src + (int64_t)r * sd.src_stride + 16 * c);
                    amax = top_finite(x, amax);
                }
                amax = reduce(amax, red_finite[parity]);
            }
            parity ^= 1;
            const float sc = fmaxf(scale_for(amax, F == __NV_E4M3 ? 8 : 15), was);
            // sc is a power of two, unless it is the scale that another quantiser gave the
            // page's older rows
            const bool pow2 = (__float_as_uint(sc) & 0x7fffffu) == 0;
            const float inv = 1.f / sc;
            auto put = [&](const Unit<ST> &x, int row, int col) {
                __stcs(reinterpret_cast<uint4 *>(page + (int64_t)(p0 + row) * sd.pos + 16 * col),
                       pow2 ? encode_unit<F>(x, inv) : encode_divided<F>(x, sc));
            };
            r = row_first;
            c = col_first;
#pragma unroll
            for (int k = 0; k < kUnits<ST>; ++k) {
                if (r < n) put(u[k], r, c);
                step();
            }
            for (; r < n; step()) {
                Unit<ST> x;
                load_unit(x, src + (int64_t)r * sd.src_stride + 16 * c);
                put(x, r, c);
            }
            if (p0 > 0 && sc > was) { // the older rows move to the new scale
                const float ratio = was / sc;
#pragma unroll 4
                for (int i = gt; i < p0 * U; i += TG) {
                    uint4 *at = reinterpret_cast<uint4 *>(page + (int64_t)(i / U) * sd.pos +
                                                          16 * (i % U));
                    float y[16];
                    decode16<F>(*at, y);
#pragma unroll
                    for (int k = 0; k < 16; ++k) y[k] *= ratio;
                    *at = encode16<F>(y);
                }
            }
            if (gt == 0 && sc != was) *sp = sc;
        }
    }
}

int bad(const char *msg) { return skv::set_error(DA_EINVAL, "args", msg); }
bool off16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 != 0; }

template <typename ST, __nv_fp8_interpretation_t F, int G>
cudaError_t launch_g(AppendParams &p, cudaStream_t st)
{
    // Few rows: a group per row, so that runs go side by side (a decode step's are one row
    // each). Many rows (over two waves of warps): a group per page's worth of rows, which
    // hold one or two runs.
    constexpr int kWarps = warps_of(G);
    const int64_t lanes = (int64_t)p.heads * 2;
    p.chunk = (int64_t)p.tokens * lanes * G > 2 * 152 * 64 ? p.block_size : 1;
    const int64_t tasks = (p.tokens + (int64_t)p.chunk - 1) / p.chunk * lanes;
    const int64_t grid = (tasks * G + kWarps - 1) / kWarps;
    if (tasks + kWarps > INT32_MAX) return cudaErrorInvalidValue; // 32-bit task numbers
    return skv::launch_after(append_kernel<ST, F, G>, (unsigned)grid, 32 * kWarps, st, p);
}

template <typename ST, __nv_fp8_interpretation_t F>
cudaError_t launch_f(AppendParams &p, cudaStream_t st)
{
    // warps whose registers hold a page of one head (4 KB each)
    const int64_t page = (int64_t)p.block_size * std::max(p.side[0].units, p.side[1].units) * 16;
    constexpr int64_t warp = 32 * kUnits<ST> * 16;
    if (page <= warp) return launch_g<ST, F, 1>(p, st);
    if (page <= 4 * warp) return launch_g<ST, F, 4>(p, st);
    return launch_g<ST, F, 8>(p, st);
}

template <typename ST> cudaError_t launch(AppendParams &p, int code, cudaStream_t st)
{
    return code == DA_E4M3 ? launch_f<ST, __NV_E4M3>(p, st) : launch_f<ST, __NV_E5M2>(p, st);
}

} // namespace

extern "C" int decode_attn_append_8bit(const da_append_t *a, const void *k_new, const void *v_new,
                                       const int64_t *slot_map, void *k_pool, void *v_pool,
                                       float *k_scale, float *v_scale, da_stream_t stream)
{
    if (!a) return bad("shapes is NULL");
    if (a->n_tokens < 0 || a->n_tokens > 1 << 30 || a->n_kv_heads < 1 || a->n_kv_heads > 65535)
        return bad("n_tokens must be in [0, 2^30] and n_kv_heads in [1, 65535]");
    for (int d : {a->head_dim, a->v_dim})
        if (d < 16 || d > 1024 || d % 16)
            return bad("head_dim and v_dim must be multiples of 16 in [16, 1024]");
    if (a->block_size < 1 || a->num_blocks < 1) return bad("block_size and num_blocks must be >= 1");
    if ((int64_t)a->block_size * std::max(a->head_dim, a->v_dim) > INT32_MAX)
        return bad("block_size * head_dim must be below 2^31");
    if (a->src_dtype != DA_F32 && a->src_dtype != DA_F16 && a->src_dtype != DA_BF16)
        return bad("src_dtype must be DA_F32, DA_F16 or DA_BF16");
    if (a->code_dtype != DA_E4M3 && a->code_dtype != DA_E5M2)
        return bad("code_dtype must be DA_E4M3 or DA_E5M2");
    const int es = a->src_dtype == DA_F32 ? 4 : 2;
    for (int64_t s : {a->k_src_stride, a->k_src_head_stride, a->v_src_stride, a->v_src_head_stride})
        if (s < 0 || (s * es) % 16) return bad("source strides must be multiples of 16 bytes, >= 0");
    for (int64_t s : {a->k_block_stride, a->k_pos_stride, a->k_head_stride, a->v_block_stride,
                      a->v_pos_stride, a->v_head_stride})
        if (s < 1 || s % 16) return bad("pool strides must be positive multiples of 16 bytes");
    for (int64_t s : {a->k_scale_block_stride, a->k_scale_head_stride, a->v_scale_block_stride,
                      a->v_scale_head_stride})
        if (s < 1) return bad("scale strides must be positive");
    if (a->n_tokens == 0) return DA_OK;
    if (!k_new || !v_new || !slot_map || !k_pool || !v_pool || !k_scale || !v_scale)
        return bad("a tensor pointer is NULL");
    if (off16(k_new) || off16(v_new) || off16(k_pool) || off16(v_pool))
        return bad("new rows and pools must be 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(slot_map) % 8 || reinterpret_cast<uintptr_t>(k_scale) % 4 ||
        reinterpret_cast<uintptr_t>(v_scale) % 4)
        return bad("slot_map and scales must be aligned to their elements");
    const cudaError_t pre = cudaGetLastError();
    if (pre != cudaSuccess) return skv::set_error(DA_ECUDA, "before append", cudaGetErrorString(pre));
    AppendParams p;
    p.side[0] = {k_new, static_cast<uint8_t *>(k_pool), k_scale, a->k_src_stride,
                 a->k_src_head_stride, a->k_block_stride, a->k_pos_stride, a->k_head_stride,
                 a->k_scale_block_stride, a->k_scale_head_stride, a->head_dim / 16};
    p.side[1] = {v_new, static_cast<uint8_t *>(v_pool), v_scale, a->v_src_stride,
                 a->v_src_head_stride, a->v_block_stride, a->v_pos_stride, a->v_head_stride,
                 a->v_scale_block_stride, a->v_scale_head_stride, a->v_dim / 16};
    p.slot_map = slot_map;
    p.tokens = a->n_tokens;
    p.heads = a->n_kv_heads;
    p.block_size = a->block_size;
    p.num_blocks = a->num_blocks;
    p.shift = -1;
    for (int s = 0; s < 31; ++s)
        if (a->block_size == 1 << s) p.shift = s;
    p.chunk = 1;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = a->src_dtype == DA_F32   ? launch<float>(p, a->code_dtype, st)
                          : a->src_dtype == DA_F16 ? launch<__half>(p, a->code_dtype, st)
                                                   : launch<__nv_bfloat16>(p, a->code_dtype, st);
    if (e != cudaSuccess) return skv::set_error(DA_ELAUNCH, "append", cudaGetErrorString(e));
    return DA_OK;
}
