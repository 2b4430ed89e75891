// Scored attention (gqa_scored.cuh): bf16 caches, 256 columns.
#include "gqa_scored.cuh"

namespace skv {

SKV_SCORED_LAUNCH(launch_gqa_scored_bf16_256)
{
    return launch_kind<__nv_bfloat16, 256, 2>(grid, smem, st, km, vm, p);
}

} // namespace skv
