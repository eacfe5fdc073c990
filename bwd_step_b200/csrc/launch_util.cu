// Host-side launch helpers shared by the kernels' launchers: per-device
// function attributes and device properties.
#include "kernels.h"

#include <atomic>
#include <mutex>
#include <set>
#include <utility>

namespace nc {

namespace {
std::mutex g_attr_mu;
std::set<std::pair<const void*, int>> g_attr_done;  // (kernel, device) pairs already raised
}  // namespace

cudaError_t ensure_smem_limit(const void* func, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(g_attr_mu);
    if (g_attr_done.count({func, dev})) return cudaSuccess;
    e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) g_attr_done.insert({func, dev});
    return e;
}

int device_sm_count() {
    static std::atomic<int> known[64];  // per device: asked once
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 148;
    if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 148;
    if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

}  // namespace nc
