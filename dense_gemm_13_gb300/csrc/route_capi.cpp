// route_capi.cpp -- the C entry point of routing to experts.
#include "route.h"

#include <cmath>
#include <cstring>

#include "device.h"
#include "dispatch.h"
#include "internal.h"

using namespace g13;

extern "C" {

void gemm_route_desc_init(gemm_route_desc_t* d) {
    if (!d) return;
    std::memset(d, 0, sizeof(*d));
    d->dtype = GEMM_F32;
    d->scores = GEMM_ROUTE_SOFTMAX;
    d->groups = 1;
    d->top_groups = 1;
    d->group_score = GEMM_ROUTE_GROUP_MAX;
    d->normalize = 1;
    d->scale = 1.0f;
}

int gemm_route(const gemm_route_desc_t* desc, const void* logits, const float* bias, int32_t* expert_ids,
               float* expert_weights, void* stream) {
    if (!desc) return GEMM_ERR_INVALID_ARG;
    RouteArgs a{};
    a.d = *desc;
    gemm_route_desc_t& d = a.d;
    if (dtype_size(d.dtype) == 0) return GEMM_ERR_INVALID_ARG;
    if ((d.scores != GEMM_ROUTE_SOFTMAX && d.scores != GEMM_ROUTE_SIGMOID) ||
        (d.group_score != GEMM_ROUTE_GROUP_MAX && d.group_score != GEMM_ROUTE_GROUP_TOP2) ||
        (d.normalize != 0 && d.normalize != 1) || !std::isfinite(d.scale))
        return GEMM_ERR_INVALID_ARG;
    if (d.T < 0 || d.E < 1 || d.top_k < 1 || d.groups < 1 || d.top_groups < 1) return GEMM_ERR_INVALID_ARG;
    if (d.groups > d.E || d.E % d.groups != 0 || d.top_groups > d.groups || d.top_k > d.E / d.groups * d.top_groups)
        return GEMM_ERR_INVALID_ARG;
    if (d.E > kRouteMaxExperts || d.top_k > kRouteMaxTopK || d.groups > kRouteMaxGroups || d.T > (int64_t(1) << 40))
        return GEMM_ERR_UNSUPPORTED;
    if (d.ld == 0) d.ld = d.E;
    if (d.ld < d.E) return GEMM_ERR_INVALID_ARG;
    if (d.ld > (int64_t(1) << 20)) return GEMM_ERR_UNSUPPORTED;
    if (d.T == 0) return GEMM_OK;
    if (!logits || !expert_ids || !expert_weights) return GEMM_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(logits) % dtype_size(d.dtype) != 0 || reinterpret_cast<uintptr_t>(bias) % 4 != 0 ||
        reinterpret_cast<uintptr_t>(expert_ids) % 4 != 0 || reinterpret_cast<uintptr_t>(expert_weights) % 4 != 0)
        return GEMM_ERR_MISALIGNED;
    int sms = 0;
    if (!usable_device(&sms)) return GEMM_ERR_NO_DEVICE;
    a.logits = logits;
    a.bias = bias;
    a.ids = expert_ids;
    a.weights = expert_weights;
    return cuda_status(launch_route(a, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
