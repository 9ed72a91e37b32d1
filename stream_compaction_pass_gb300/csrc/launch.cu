// launch.cu -- launch set-up shared by the kernel launchers: the dynamic
// shared-memory limit of a kernel and the number of its CTAs an SM holds,
// kept per (kernel, device).  The shared-memory attribute belongs to the
// device it was set on, so a process that launches on several devices sets
// it once on each; the table is locked so that host threads that launch at
// the same time on a new device set it up once.
#include <map>
#include <mutex>
#include <utility>

#include "internal.h"

namespace ss {

namespace {
std::mutex g_setup_mu;
std::map<std::pair<const void*, int>, KernelSetup> g_setup;
struct ClusterKey {
    const void* kern;
    int dev, ranks;
    bool operator<(const ClusterKey& o) const {
        return kern != o.kern ? kern < o.kern : dev != o.dev ? dev < o.dev : ranks < o.ranks;
    }
};
std::map<ClusterKey, int> g_clusters;
}  // namespace

cudaError_t kernel_setup(const void* kern, int threads, size_t max_smem, KernelSetup* out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lk(g_setup_mu);
    const auto key = std::make_pair(kern, dev);
    auto it = g_setup.find(key);
    if (it != g_setup.end()) {
        *out = it->second;
        return cudaSuccess;
    }
    KernelSetup k;
    if (max_smem > 0) {  // also at 48 KB and below: static shared memory counts against the default limit
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)max_smem);
        if (e != cudaSuccess) return e;
    }
    e = cudaDeviceGetAttribute(&k.sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    int b = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&b, kern, threads, max_smem);
    if (e != cudaSuccess) return e;
    k.sms = k.sms > 0 ? k.sms : 1;
    k.blocks_per_sm = b > 0 ? b : 1;
    g_setup[key] = k;
    *out = k;
    return cudaSuccess;
}

cudaError_t cluster_limit(const void* kern, int threads, size_t smem, int ranks, int* clusters) {
    ClusterKey key{kern, 0, ranks};
    cudaError_t e = cudaGetDevice(&key.dev);
    if (e != cudaSuccess) return e;
    {
        std::lock_guard<std::mutex> lk(g_setup_mu);
        auto it = g_clusters.find(key);
        if (it != g_clusters.end()) {
            *clusters = it->second;
            return cudaSuccess;
        }
    }
    KernelSetup su;
    e = kernel_setup(kern, threads, smem, &su);
    if (e != cudaSuccess) return e;
    int n = su.sms * su.blocks_per_sm;
    if (ranks > 1) {
        cudaLaunchAttribute at;
        at.id = cudaLaunchAttributeClusterDimension;
        at.val.clusterDim.x = (unsigned)ranks;
        at.val.clusterDim.y = at.val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(ranks * su.sms));
        cfg.blockDim = dim3((unsigned)threads);
        cfg.dynamicSmemBytes = smem;
        cfg.attrs = &at;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
        if (e != cudaSuccess) return e;
    }
    std::lock_guard<std::mutex> lk(g_setup_mu);
    g_clusters[key] = n;
    *clusters = n;
    return cudaSuccess;
}

}  // namespace ss
