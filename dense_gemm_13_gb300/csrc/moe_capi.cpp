// moe_capi.cpp -- the C entry points of the mixture-of-experts layer.
#include "moe.h"

#include <algorithm>
#include <cstring>
#include <mutex>
#include <new>
#include <unordered_set>

#include "device.h"
#include "internal.h"

using namespace g13;

struct gemm_moe_plan_s {
    gemm_moe_desc_t d{};
    MoeWorkspace w{};
    int device = 0;
    int grid = 0;
    unsigned* d_status = nullptr;
};

namespace {

std::mutex g_live_mu;
std::unordered_set<const gemm_moe_plan_s*> g_live;

bool alive(const gemm_moe_plan_s* p) {
    if (!p) return false;
    std::lock_guard<std::mutex> lk(g_live_mu);
    return g_live.count(p) != 0;
}

int check_desc(gemm_moe_desc_t& d) {
    if (d.dtype != GEMM_F32 && d.dtype != GEMM_F16 && d.dtype != GEMM_BF16) return GEMM_ERR_INVALID_ARG;
    if (d.act != GEMM_MOE_GELU && d.act != GEMM_MOE_RELU && d.act != GEMM_MOE_SWIGLU)
        return GEMM_ERR_INVALID_ARG;
    if ((d.normalize != 0 && d.normalize != 1) || (d.flags & ~GEMM_FLAG_TEST_STALL)) return GEMM_ERR_INVALID_ARG;
    if (d.T < 0 || d.E < 1 || d.H < 1 || d.I < 1 || d.top_k < 1 || d.top_k > d.E) return GEMM_ERR_INVALID_ARG;
    if (d.dtype == GEMM_F32 || d.T > kMoeMaxTokens || d.E > kMoeMaxExperts || d.top_k > kMoeMaxTopK ||
        d.H > kMoeMaxH || d.I > (int64_t(1) << 20))
        return GEMM_ERR_UNSUPPORTED;
    const int64_t rows = d.act == GEMM_MOE_SWIGLU ? 2 * d.I : d.I;
    if (d.ldx == 0) d.ldx = d.H;
    if (d.ld_router == 0) d.ld_router = d.H;
    if (d.ld_w1 == 0) d.ld_w1 = d.H;
    if (d.ld_w2 == 0) d.ld_w2 = d.I;
    if (d.ldy == 0) d.ldy = d.H;
    // a bound that keeps every product below in 64 bits
    const int64_t lim = int64_t(1) << 40;
    if (d.ldx < d.H || d.ld_router < d.H || d.ld_w1 < d.H || d.ld_w2 < d.I || d.ldy < d.H) return GEMM_ERR_INVALID_ARG;
    if (d.ldx > lim || d.ld_router > lim || d.ld_w1 > lim || d.ld_w2 > lim || d.ldy > lim) return GEMM_ERR_UNSUPPORTED;
    if (d.stride_w1 == 0) d.stride_w1 = rows * d.ld_w1;
    if (d.stride_w2 == 0) d.stride_w2 = d.H * d.ld_w2;
    if (d.stride_w1 < 0 || d.stride_w2 < 0) return GEMM_ERR_INVALID_ARG;
    if (d.stride_w1 > (int64_t(1) << 52) || d.stride_w2 > (int64_t(1) << 52)) return GEMM_ERR_UNSUPPORTED;
    // the kernel counts pieces of 16 rows x 64 elements in 32 bits
    if (d.E * ((rows + 15) / 16 + 1) * ((d.H + 63) / 64) >= (int64_t(1) << 30) ||
        d.E * ((d.H + 15) / 16) * ((d.I + 63) / 64) >= (int64_t(1) << 30))
        return GEMM_ERR_UNSUPPORTED;
    if (d.timeout_ms == 0) d.timeout_ms = 2000;
    return GEMM_OK;
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// A layer with a router (Wr), or with a choice made beforehand (given_ids, given_weights).
int run_layer(const gemm_moe_plan_s* plan, const void* X, const void* Wr, const int32_t* given_ids,
              const float* given_weights, const void* W1, const void* W2, void* Y, int32_t* expert_ids,
              float* expert_weights, void* workspace, void* stream) {
    if (!X || !W1 || !W2 || !Y || !workspace) return GEMM_ERR_INVALID_ARG;
    if (!aligned(X, 2) || !aligned(Wr, 2) || !aligned(W1, 2) || !aligned(W2, 2) || !aligned(Y, 2) ||
        !aligned(expert_ids, 4) || !aligned(expert_weights, 4) || !aligned(given_ids, 4) ||
        !aligned(given_weights, 4) || !aligned(workspace, 256))
        return GEMM_ERR_MISALIGNED;
    int cur = -1;
    if (cudaGetDevice(&cur) != cudaSuccess || cur != plan->device) return GEMM_ERR_INVALID_ARG;
    MoeArgs a{};
    a.d = plan->d;
    a.w = plan->w;
    a.x = X;
    a.router = Wr;
    a.w1 = W1;
    a.w2 = W2;
    a.y = Y;
    a.ids = expert_ids;
    a.weights = expert_weights;
    a.given_ids = given_ids;
    a.given_weights = given_weights;
    a.ws = static_cast<char*>(workspace);
    a.status = plan->d_status;
    a.timeout_ns = static_cast<uint64_t>(plan->d.timeout_ms) * 1000000ull;
    return cuda_status(launch_moe(a, plan->grid, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

void gemm_moe_desc_init(gemm_moe_desc_t* d) {
    if (!d) return;
    std::memset(d, 0, sizeof(*d));
    d->dtype = GEMM_BF16;
    d->act = GEMM_MOE_SWIGLU;
    d->normalize = 1;
}

int gemm_moe_plan(const gemm_moe_desc_t* desc, gemm_moe_plan_t* out_plan) {
    if (!out_plan) return GEMM_ERR_INVALID_ARG;
    *out_plan = nullptr;
    if (!desc) return GEMM_ERR_INVALID_ARG;
    gemm_moe_desc_t d = *desc;
    const int rc = check_desc(d);
    if (rc != GEMM_OK) return rc;
    int dev = 0, major = 0, minor = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || major != 10 ||
        minor != 3)
        return GEMM_ERR_NO_DEVICE;
    // a warp's share of the down product (a quarter of a CTA's) touches at most two output
    // blocks: that needs fewer than four blocks per CTA
    if ((d.H + kMoeBlock - 1) / kMoeBlock > int64_t(3) * sms) return GEMM_ERR_UNSUPPORTED;
    gemm_moe_plan_s* pl = new (std::nothrow) gemm_moe_plan_s();
    if (!pl) return GEMM_ERR_OUT_OF_MEMORY;
    pl->d = d;
    pl->device = dev;
    pl->grid = sms;
    pl->w = moe_workspace(d, sms);
    cudaError_t ce = cudaMalloc(reinterpret_cast<void**>(&pl->d_status), sizeof(unsigned));
    if (ce == cudaSuccess) ce = cudaMemset(pl->d_status, 0, sizeof(unsigned));
    if (ce != cudaSuccess) {
        if (pl->d_status) cudaFree(pl->d_status);
        delete pl;
        return cuda_status(ce);
    }
    try {
        std::lock_guard<std::mutex> lk(g_live_mu);
        g_live.insert(pl);
    } catch (...) {
        cudaFree(pl->d_status);
        delete pl;
        return GEMM_ERR_OUT_OF_MEMORY;
    }
    *out_plan = pl;
    return GEMM_OK;
}

int64_t gemm_moe_workspace_bytes(gemm_moe_plan_t plan) { return alive(plan) ? plan->w.bytes : 0; }

int gemm_moe_run(gemm_moe_plan_t plan, const void* X, const void* Wr, const void* W1, const void* W2,
                 void* Y, int32_t* expert_ids, float* expert_weights, void* workspace, void* stream) {
    if (!alive(plan)) return GEMM_ERR_BAD_PLAN;
    if (plan->d.T == 0) return GEMM_OK;
    if (!Wr) return GEMM_ERR_INVALID_ARG;
    return run_layer(plan, X, Wr, nullptr, nullptr, W1, W2, Y, expert_ids, expert_weights, workspace, stream);
}

int gemm_moe_run_routed(gemm_moe_plan_t plan, const void* X, const int32_t* expert_ids, const float* expert_weights,
                        const void* W1, const void* W2, void* Y, void* workspace, void* stream) {
    if (!alive(plan)) return GEMM_ERR_BAD_PLAN;
    if (plan->d.T == 0) return GEMM_OK;
    if (!expert_ids || !expert_weights) return GEMM_ERR_INVALID_ARG;
    return run_layer(plan, X, nullptr, expert_ids, expert_weights, W1, W2, Y, nullptr, nullptr, workspace, stream);
}

int gemm_moe_status(gemm_moe_plan_t plan) {
    if (!alive(plan)) return GEMM_ERR_BAD_PLAN;
    if (cudaDeviceSynchronize() != cudaSuccess) return GEMM_ERR_CUDA;
    unsigned v = 0;
    if (cudaMemcpy(&v, plan->d_status, sizeof v, cudaMemcpyDeviceToHost) != cudaSuccess)
        return GEMM_ERR_CUDA;
    return (v & 1u) ? GEMM_ERR_DEVICE_TIMEOUT : GEMM_OK;
}

void gemm_moe_destroy(gemm_moe_plan_t plan) {
    {
        std::lock_guard<std::mutex> lk(g_live_mu);
        if (!plan || !g_live.erase(plan)) return;
    }
    free_plan_memory(plan->d_status);
    delete plan;
}

}  // extern "C"
