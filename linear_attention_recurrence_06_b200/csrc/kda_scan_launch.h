// kda_scan_launch.h -- how the tiled kernels of the element-wise scan are launched.
#pragma once
#include <atomic>

#include "kda_scan.h"
#include "kda_scan_tile.cuh"

namespace kda {

// The widest copy that every input's address and token stride allow.
inline int scan_width(const void* const* in, const int64_t* ld, int n, bool bf16) {
    uintptr_t all = 0;
    for (int i = 0; i < n; ++i) all |= reinterpret_cast<uintptr_t>(in[i]) | (uintptr_t)(ld[i] * (bf16 ? 2 : 4));
    return all % 16 == 0 ? 16 : (all % 4 == 0 ? 4 : 2);
}

// Splits and cluster: 2 CTAs fit on an SM.  Splitting the batch costs nothing, splitting time
// costs an exchange per tile, so time is only split where the batch leaves SMs without work.
// Packed sequences may be one long one: they are split only where 8 CTAs in time would not do.
struct ScanGrid {
    int groups, splits, cluster;
};
inline ScanGrid scan_grid(const ScanArgs& a, int tile, int sms) {
    ScanGrid g{(a.D + SC_CH - 1) / SC_CH, 1, 1};
    const int64_t tokens = a.cu ? a.T : (int64_t)a.B * a.T;
    const int slots = 2 * sms;
    auto clamp = [](int64_t v, int64_t hi) { return (int)(v < 1 ? 1 : (v > hi ? hi : v)); };
    const int want = clamp(slots / g.groups, 65535);
    if (!a.cu) {
        g.splits = clamp(want, a.B);
    } else if (want > SC_MAX_CLUSTER) {
        g.splits = clamp(want / SC_MAX_CLUSTER, a.n_seqs);
    }
    g.cluster = clamp(want / g.splits, SC_MAX_CLUSTER);
    const int64_t tiles = (tokens / g.splits + tile) / tile;  // one at least
    g.cluster = clamp(g.cluster, tiles);
    return g;
}

template <auto KERNEL>
cudaError_t scan_launch(int smem, int tile, const ScanArgs& a, int width, cudaStream_t stream) {
    static std::atomic<uint64_t> ready{0};  // devices on which this kernel may use its shared memory
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
        if ((e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
        if (dev < 64) ready.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
    }
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    const ScanGrid g = scan_grid(a, tile, sms);
    if ((int64_t)g.groups * g.cluster > INT32_MAX) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(g.groups * g.cluster), (unsigned)g.splits);
    cfg.blockDim = dim3(SC_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = g.cluster;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = g.cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, KERNEL, a, g.cluster, width);
}

}  // namespace kda
