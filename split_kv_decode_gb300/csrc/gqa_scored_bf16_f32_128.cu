// Scored attention (gqa_scored.cuh): bf16 caches, f32 outputs, 128 columns.
#include "gqa_scored.cuh"

namespace skv {

SKV_SCORED_LAUNCH(launch_gqa_scored_bf16_f32_128)
{
    return launch_kind<__nv_bfloat16, 128, 3>(grid, smem, st, km, vm, p);
}

} // namespace skv
