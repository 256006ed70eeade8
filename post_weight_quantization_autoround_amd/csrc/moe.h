// Mixture of experts on either side of the grouped products: the router and
// the weighted sum of the experts' outputs (moe_kernels.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ar {

constexpr int32_t kMoeMaxExperts = 1024;       // a wavefront holds a token's scores, 16 a lane
constexpr int32_t kMoeMaxChoices = 64;         // one a lane
constexpr int64_t kMoeMaxSlots = 1 << 24;      // tokens times choices, rows of a grouped product

struct MoeRouteArgs {
    const void* logits; bool bf16;             // [T, E]
    int64_t T;
    int32_t E, k;
    bool sigmoid, normalize;
    const float* bias;                         // [E], nullable
    float weight_scale;
    int32_t* expert; float* weight;            // [T, k]
    int32_t* offsets;                          // [E + 1]
    int32_t* token;                            // [T k]
    int32_t* pos;                              // [T, k]
};
hipError_t launch_moe_route(const MoeRouteArgs& a, hipStream_t stream);

struct MoeCombineArgs {
    const void* z; bool z_bf16;                // [P, N]
    int64_t P, N;
    const int32_t* pos; const float* weight;   // [T, k]
    int64_t T;
    int32_t k;
    const void* res; bool res_bf16;            // [T, N], nullable; may be y with the same type
    void* y; bool y_bf16;                      // [T, N]
};
hipError_t launch_moe_combine(const MoeCombineArgs& a, hipStream_t stream);

}  // namespace ar
