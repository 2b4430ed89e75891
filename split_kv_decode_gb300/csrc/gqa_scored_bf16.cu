// Scored attention (gqa_scored.cuh): bf16 caches, 16-bit outputs.
#include "gqa_scored.cuh"

namespace skv {

cudaError_t launch_gqa_scored_bf16(int head_dim, int grid, int smem, cudaStream_t st,
                                     const CUtensorMap &km, const CUtensorMap &vm,
                                     const ScoredParams &p)
{
    return launch_d<__nv_bfloat16, 2>(head_dim, grid, smem, st, km, vm, p);
}

} // namespace skv
