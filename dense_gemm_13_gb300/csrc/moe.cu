// moe.cu -- the mixture-of-experts layer with its router, and the workspace.
#include "moe_kernel.cuh"

namespace g13 {

MoeWorkspace moe_workspace(const gemm_moe_desc_t& d, int grid) {
    MoeWorkspace w{};
    w.hp = round_up(d.H, 64);
    w.ip = round_up(d.I, 64);
    w.bar = 0;
    w.counters = 256;
    w.logits = w.counters + round_up((d.H + kMoeBlock - 1) / kMoeBlock * 4, 256);
    w.x = w.logits + round_up(d.T * d.E * 4, 256);
    w.h = w.x + round_up(d.T * w.hp * 2, 256);
    w.partial = w.h + round_up(d.T * d.top_k * (d.dtype == GEMM_F16 ? 4 : 2) * w.ip * 2, 256);
    w.flushed = w.partial + static_cast<int64_t>(grid) * 2 * kMoeBlock * d.T * 4;
    w.bytes = w.flushed + static_cast<int64_t>(grid) * kMoeTeams * kMoeBlock * d.T * 4;
    return w;
}

cudaError_t launch_moe(const MoeArgs& a, int grid, cudaStream_t st) {
    return a.given_ids ? launch_moe_given(a, grid, st) : launch_moe_kernels<false>(a, grid, st);
}

}  // namespace g13
