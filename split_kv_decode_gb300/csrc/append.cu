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
#include <cstdio>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "internal.h"

namespace skv {
int set_error(int code, const char *phase, const char *msg); // api.cpp
}

namespace {

constexpr int kThreads = 128;

struct AppendParams {
    da_append_t a;
    const void *src[2];
    const int64_t *slot_map;
    uint8_t *pool[2];
    float *scale[2];
    int64_t src_stride[2], src_head_stride[2];
    int64_t block_stride[2], pos_stride[2], head_stride[2];
    int64_t scale_block_stride[2], scale_head_stride[2];
    int32_t dim[2];
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

template <__nv_fp8_interpretation_t F> __device__ __forceinline__ uint8_t encode(float x)
{
    return __nv_cvt_float_to_fp8(x, __NV_SATFINITE, F);
}
template <__nv_fp8_interpretation_t F> __device__ __forceinline__ float decode(uint8_t c)
{
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, F)));
}

// the least e >= -100 with a <= 1.75 * 2^(top + e), as the bits of 2^e (a >= 0, finite)
__device__ __forceinline__ float scale_for(float a, int top)
{
    const uint32_t u = __float_as_uint(a);
    int e = (int)(u >> 23) - 127 - top + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = max(e, -100);
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

template <typename ST, __nv_fp8_interpretation_t F>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams p)
{
    const int t = blockIdx.x, h = blockIdx.y, kv = blockIdx.z;
    const int P = p.a.block_size, T = p.a.n_tokens, dim = p.dim[kv];
    const int64_t slot = p.slot_map[t];
    if (slot < 0 || slot / P >= p.a.num_blocks) return;
    const int p0 = (int)(slot % P);
    if (t > 0 && p0 > 0 && p.slot_map[t - 1] == slot - 1) return; // not a run's first row
    // the run's length: rows at consecutive slots up to the block's end
    __shared__ int n_s;
    __shared__ float red[kThreads / 32];
    if (threadIdx.x == 0) n_s = min(P - p0, T - t);
    __syncthreads();
    for (int i = threadIdx.x; i < min(P - p0, T - t); i += kThreads)
        if (p.slot_map[t + i] != slot + i) {
            atomicMin(&n_s, i);
            break;
        }
    __syncthreads();
    const int n = n_s;
    const int64_t blk = slot / P;
    const ST *src = static_cast<const ST *>(p.src[kv]) + (size_t)t * p.src_stride[kv] +
                    (size_t)h * p.src_head_stride[kv];
    uint8_t *page = p.pool[kv] + blk * p.block_stride[kv] + h * p.head_stride[kv];
    float *sp = p.scale[kv] + blk * p.scale_block_stride[kv] + h * p.scale_head_stride[kv];
    const float was = *sp;

    float amax = 0.f;
    for (int i = threadIdx.x; i < n * dim; i += kThreads) {
        const float a = fabsf(to_f(src[(size_t)(i / dim) * p.src_stride[kv] + i % dim]));
        if (a <= 3.402823466e38f) amax = fmaxf(amax, a);
    }
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
    __syncthreads();
    for (int w = 0; w < kThreads / 32; ++w) amax = fmaxf(amax, red[w]);
    float s = scale_for(amax, F == __NV_E4M3 ? 8 : 15);
    if (p0 > 0) s = fmaxf(s, was);
    if (p0 > 0 && s > was) { // the older rows move to the new scale
        const float f = was / s;
        for (int i = threadIdx.x; i < p0 * dim; i += kThreads) {
            uint8_t *c = page + (int64_t)(i / dim) * p.pos_stride[kv] + i % dim;
            *c = encode<F>(decode<F>(*c) * f);
        }
    }
    // s is a power of two, unless it is the scale that another quantiser gave the
    // block's older rows
    const bool pow2 = (__float_as_uint(s) & 0x7fffffu) == 0;
    const float inv = 1.f / s;
    auto scaled = [&](float x) { return pow2 ? x * inv : x / s; };
    for (int i = threadIdx.x; i < n * dim; i += kThreads)
        page[(int64_t)(p0 + i / dim) * p.pos_stride[kv] + i % dim] =
            encode<F>(scaled(to_f(src[(size_t)(i / dim) * p.src_stride[kv] + i % dim])));
    if (threadIdx.x == 0) *sp = s;
}

int bad(const char *msg) { return skv::set_error(DA_EINVAL, "args", msg); }
bool off16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 != 0; }

template <typename ST> void launch(const AppendParams &p, cudaStream_t st)
{
    const dim3 grid(p.a.n_tokens, p.a.n_kv_heads, 2);
    if (p.a.code_dtype == DA_E4M3) append_kernel<ST, __NV_E4M3><<<grid, kThreads, 0, st>>>(p);
    else append_kernel<ST, __NV_E5M2><<<grid, kThreads, 0, st>>>(p);
}

} // namespace

extern "C" int decode_attn_append_8bit(const da_append_t *a, const void *k_new, const void *v_new,
                                       const int64_t *slot_map, void *k_pool, void *v_pool,
                                       float *k_scale, float *v_scale, da_stream_t stream)
{
    if (!a) return bad("shapes is NULL");
    if (a->n_tokens < 0 || a->n_kv_heads < 1 || a->n_kv_heads > 65535)
        return bad("n_tokens must be >= 0 and n_kv_heads in [1, 65535]");
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
    p.a = *a;
    p.slot_map = slot_map;
    p.src[0] = k_new;
    p.src[1] = v_new;
    p.pool[0] = static_cast<uint8_t *>(k_pool);
    p.pool[1] = static_cast<uint8_t *>(v_pool);
    p.scale[0] = k_scale;
    p.scale[1] = v_scale;
    p.src_stride[0] = a->k_src_stride;
    p.src_stride[1] = a->v_src_stride;
    p.src_head_stride[0] = a->k_src_head_stride;
    p.src_head_stride[1] = a->v_src_head_stride;
    p.block_stride[0] = a->k_block_stride;
    p.block_stride[1] = a->v_block_stride;
    p.pos_stride[0] = a->k_pos_stride;
    p.pos_stride[1] = a->v_pos_stride;
    p.head_stride[0] = a->k_head_stride;
    p.head_stride[1] = a->v_head_stride;
    p.scale_block_stride[0] = a->k_scale_block_stride;
    p.scale_block_stride[1] = a->v_scale_block_stride;
    p.scale_head_stride[0] = a->k_scale_head_stride;
    p.scale_head_stride[1] = a->v_scale_head_stride;
    p.dim[0] = a->head_dim;
    p.dim[1] = a->v_dim;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (a->src_dtype == DA_F32) launch<float>(p, st);
    else if (a->src_dtype == DA_F16) launch<__half>(p, st);
    else launch<__nv_bfloat16>(p, st);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return skv::set_error(DA_ELAUNCH, "append", cudaGetErrorString(e));
    return DA_OK;
}
