// Scored attention (gqa_scored.cuh): f16 caches.
#include "gqa_scored.cuh"

namespace skv {

cudaError_t launch_gqa_scored_f16(int head_dim, int grid, int smem, cudaStream_t st,
                                     const CUtensorMap &km, const CUtensorMap &vm,
                                     const ScoredParams &p)
{
    return launch_d<__half, 2>(head_dim, grid, smem, st, km, vm, p);
}

} // namespace skv
