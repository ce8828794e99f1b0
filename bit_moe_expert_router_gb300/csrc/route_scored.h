// Internal arguments and launcher of routing by scores (host side; the C ABI in
// api.cu validates everything before calling it).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

struct RouteScoredArgs {
    const void* logits;
    const float* bias;   // [E] or null
    int32_t* ids;        // [T][k]
    float* wts;
    int64_t T, E, stride;
    int k, dtype;        // dtype: MOE_LOGITS_*
    int sigmoid, n_groups, topk_groups, group_top, renormalise;
    float scale;
    // set by the launcher: lanes of a group (a power of two, n_groups of them make 32), experts of a group and of a lane
    int lanes_log2, group_size, per_lane, vec;
};

// n_groups: a power of two up to 32 that divides E <= 1024; k <= 32.
cudaError_t launch_route_scored(RouteScoredArgs a, cudaStream_t st);

}  // namespace moe
