// What the host has asked of a device or set for a kernel on it, kept by device: a function's attribute that was set with one device
// current is not set on another.  Plain C++ over the runtime's interface, without device code.
#pragma once

#include <cuda_runtime_api.h>

#include <map>
#include <mutex>
#include <tuple>
#include <utility>

namespace tq {

// Multiprocessors of the current device; the GB300's where none can be asked.
inline int device_sms() {
    static std::mutex mu;
    static std::map<int, int> known;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 152;
    std::lock_guard<std::mutex> lock(mu);
    int& n = known[dev];
    if (n <= 0 && cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) n = 0;
    return n > 0 ? n : 152;
}

// Raise a kernel's dynamic shared-memory limit once for each device (not on every
// launch, so launches can be captured into CUDA graphs without extra API calls).
inline cudaError_t ensure_smem(const void* kernel, size_t bytes) {
    static std::mutex mu;
    static std::map<std::pair<int, const void*>, size_t> done;
    if (bytes <= 48 * 1024) return cudaSuccess;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    size_t& cur = done[{dev, kernel}];
    if (cur >= bytes) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) cur = bytes;
    return e;
}

// May clusters of `size` CTAs of this kernel be launched on the current device?  Up to 8 always; more have to be allowed to the
// kernel, and the device may have no place for one (fewer multiprocessors behind one crossbar, or some of them given away).  The
// kernel's shared-memory limit is to be raised before.
inline bool clusters_fit(const void* kernel, int size, int threads, size_t smem) {
    static std::mutex mu;
    static std::map<std::tuple<int, const void*, int, int, size_t>, bool> known;
    if (size <= 8) return true;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    std::lock_guard<std::mutex> lock(mu);
    const auto key = std::make_tuple(dev, kernel, size, threads, smem);
    const auto at = known.find(key);
    if (at != known.end()) return at->second;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)size);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)size;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    const bool fit = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                     cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess && n > 0;
    if (!fit) cudaGetLastError();  // (a refusal here is an answer, not an error of the call)
    if (known.size() > 4096) known.clear();
    return known[key] = fit;
}

}  // namespace tq
