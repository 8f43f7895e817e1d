// Structures shared between the host API (api.hip) and the routing kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace dlm {

constexpr int kRouteMaxExperts = 512;
constexpr int kRouteMaxK = 16;
constexpr int kRouteSoftmax = 0, kRouteSigmoid = 1;

struct RouteArgs {
    const void* logits;  // [T] rows of E, ld elements apart
    int64_t ld;
    const float* bias;   // [E] or nullptr
    int64_t T;
    int32_t E, k, score, renorm;
    float scale;
    int32_t n_groups, group_size, keep_groups, group_top;
    uint32_t gs_magic;     // e / group_size = (e * gs_magic) >> 20 for e < 512
    int32_t vec, vec_out;  // rows of logits / dlogits take 16-byte accesses
    int32_t vec_bias;      // so does the bias, and E is a multiple of 4
    int32_t need_scores;   // every expert's score is needed, not only the chosen ones'
    int32_t scores_order;  // keys are scores plus bias; else the logits order the experts
    int32_t group_lanes;   // lanes a group spans when groups are whole runs of them, else 0 (the launcher sets it)
    int32_t lds_groups;    // byte offset of the groups' part of the dynamic LDS
    int32_t* idx;          // [T][k] out
    float* g;              // [T][k] out
    int32_t* counts;       // [E], added to, or nullptr
    // gradient
    const int32_t* in_idx; // [T][k]
    const float* dg;       // [T][k]
    void* dlogits;         // [T] rows of E, ldd elements apart
    int64_t ldd;
};

hipError_t launch_route(const RouteArgs& a, int dtype, hipStream_t s);
hipError_t launch_route_grad(const RouteArgs& a, int dtype, hipStream_t s);

}  // namespace dlm
