// Scored attention (gqa_scored.cuh): bf16 caches, f32 outputs.
#include "gqa_scored.cuh"

namespace skv {

cudaError_t launch_gqa_scored_bf16_f32(int head_dim, int grid, int smem, cudaStream_t st,
                                     const CUtensorMap &km, const CUtensorMap &vm,
                                     const ScoredParams &p)
{
    return launch_d<__nv_bfloat16, 3>(head_dim, grid, smem, st, km, vm, p);
}

} // namespace skv
