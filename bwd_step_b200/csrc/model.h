// The model handle behind the C ABI (nanochat_b200.h): config, flat parameter
// layout, device status word, streams and the per-launch profiler.
#pragma once
#include "nanochat_b200.h"
#include "kernels.h"

#include <string>
#include <vector>

struct ParamEntry { std::string name; int64_t offset; int rows, cols; };

struct nc_model {
    nc_config cfg;
    nc_precision prec;
    int device = 0;
    int* status = nullptr;  // device int[64]: [0] = status flags, [1] = loss scratch for the host variant
    std::vector<ParamEntry> layout;
    int64_t nparams = 0;
    int V, d, L, H, nkv, hd, F, Nqkv;
    nc::DType at;  // weight / activation type
    bool tc = false;  // tcgen05 path available (bf16 on sm_100)
    // LM head: fused (logits never stored; tensor-core path only) or materialised
    // logit chunks with a separate cross-entropy pass; rows per chunk (0 = default)
    int lm_mode = NC_LM_HEAD_FUSED;
    int lm_rows = 0;
    // activations recomputed in the backward instead of saved (NC_RECOMPUTE_*)
    int recompute = NC_RECOMPUTE_NONE;
    // caller-owned events recorded when each gradient bucket is final (may be empty)
    std::vector<cudaEvent_t> grad_events;
    // the backward's weight-gradient GEMMs run on this second stream, overlapping the
    // input-gradient chain on the caller's stream; kSideEvents order the two (null: off)
    static constexpr int kSideEvents = 6;
    cudaStream_t side = nullptr;
    cudaEvent_t sev[kSideEvents] = {};
    // profiler: CUDA events around every launch while enabled
    struct Rec { int cls; cudaEvent_t a, b; double flops, bytes; long long launches; };
    bool prof_on = false;
    std::vector<cudaEvent_t> ev_pool;
    size_t ev_next = 0;
    std::vector<Rec> recs;
    cudaEvent_t event() {
        if (ev_next == ev_pool.size()) {
            cudaEvent_t e = nullptr;
            if (cudaEventCreate(&e) != cudaSuccess) return nullptr;
            ev_pool.push_back(e);
        }
        return ev_pool[ev_next++];
    }
};

namespace nc {
// The model's device must be current: its buffers are that device's memory,
// and kernels launched on another device would reach them as peer memory.
inline bool on_model_device(const nc_model* m) {
    int dev = -1;
    return cudaGetDevice(&dev) == cudaSuccess && dev == m->device;
}
}  // namespace nc
