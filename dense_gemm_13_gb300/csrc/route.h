// route.h -- routing to experts: sizes, arguments and launcher.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "gemm13.h"

namespace g13 {

constexpr int kRouteMaxExperts = 512, kRouteMaxTopK = 32, kRouteMaxGroups = 32;

struct RouteArgs {
    gemm_route_desc_t d;
    const void* logits;
    const float* bias;  // or null
    int32_t* ids;
    float* weights;
};

cudaError_t launch_route(const RouteArgs& a, int num_sms, cudaStream_t st);

}  // namespace g13
