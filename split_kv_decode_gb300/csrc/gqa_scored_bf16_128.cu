// Scored attention (gqa_scored.cuh): bf16 caches, 128 columns.
#include "gqa_scored.cuh"

namespace skv {

SKV_SCORED_LAUNCH(launch_gqa_scored_bf16_128)
{
    return launch_kind<__nv_bfloat16, 128, 2>(grid, smem, st, km, vm, p);
}

} // namespace skv
