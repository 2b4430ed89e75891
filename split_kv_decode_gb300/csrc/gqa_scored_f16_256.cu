// Scored attention (gqa_scored.cuh): f16 caches, 256 columns.
#include "gqa_scored.cuh"

namespace skv {

SKV_SCORED_LAUNCH(launch_gqa_scored_f16_256)
{
    return launch_kind<__half, 256, 2>(grid, smem, st, km, vm, p);
}

} // namespace skv
