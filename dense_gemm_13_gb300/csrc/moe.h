// moe.h -- the mixture-of-experts layer: sizes, workspace and launcher.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "gemm13.h"

namespace g13 {

constexpr int kMoeMaxTokens = 64, kMoeMaxExperts = 512, kMoeMaxTopK = 32, kMoeMaxH = 16384;
constexpr int kMoeWarps = 16;
constexpr int kMoeBlock = 64;  // output columns that the down product's CTAs share or cut

// Byte offsets of the parts of a run's workspace (FP16: behind h, as large, its values beyond FP16's range).
struct MoeWorkspace {
    int64_t bar, counters, logits, x, h, partial, flushed, bytes;
    int64_t hp, ip;  // row lengths of the padded copies of x and of h (multiples of 64)
};
MoeWorkspace moe_workspace(const gemm_moe_desc_t& d, int grid);

struct MoeArgs {
    gemm_moe_desc_t d;
    MoeWorkspace w;
    const void* x;
    const void* router;
    const void* w1;
    const void* w2;
    void* y;
    int32_t* ids;
    float* weights;
    char* ws;
    unsigned* status;
    uint64_t timeout_ns;
};

// Routing kernel, then the experts' kernel on a cooperative grid of `grid` CTAs.
cudaError_t launch_moe(const MoeArgs& a, int grid, cudaStream_t st);

}  // namespace g13
