// kda_scan_launch.h -- how the tiled kernels of the element-wise scan are launched.
#pragma once
#include <string.h>

#include <atomic>

#include "kda_scan.h"
#include "kda_scan_tile.cuh"

namespace kda {

// __VA_ARGS__ with the constants G (a gate) and W (normalize)
#define KDA_SCAN_GN(GATE, NORM, ...)                                     \
    do {                                                                 \
        if (GATE) {                                                      \
            if (NORM) { constexpr bool G = true, W = true; __VA_ARGS__; }       \
            else      { constexpr bool G = true, W = false; __VA_ARGS__; }      \
        } else {                                                         \
            if (NORM) { constexpr bool G = false, W = true; __VA_ARGS__; }      \
            else      { constexpr bool G = false, W = false; __VA_ARGS__; }     \
        }                                                                \
    } while (0)

// [rows, cols] tensor, rows `ld` elements apart, box of a warp's tokens, zeros outside
bool make_scan_map(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t ld, int box_rows, bool bf16);

// The widest copy that every input's address and token stride allow (16: TMA), and the tensor
// maps for it.
inline cudaError_t scan_maps(const ScanArgs& a, const void* const* in, const int64_t* ld, int n, int box_rows,
                             ScanMaps* maps, int* width) {
    memset(maps, 0, sizeof(*maps));
    const int64_t tokens = a.cu ? a.T : (int64_t)a.B * a.T;
    uintptr_t all = 0;
    for (int i = 0; i < n; ++i) all |= reinterpret_cast<uintptr_t>(in[i]) | (uintptr_t)(ld[i] * (a.in_bf16 ? 2 : 4));
    *width = all % 16 == 0 ? 16 : (all % 4 == 0 ? 4 : 2);
    if (*width == 16 && tokens > 0)
        for (int i = 0; i < n; ++i)
            if (!make_scan_map(&maps->m[i], in[i], tokens, a.D, ld[i], box_rows, a.in_bf16)) return cudaErrorInvalidValue;
    return cudaSuccess;
}

// Splits and cluster, for `per_sm` CTAs on an SM with clusters of up to 4 (one with more).  Splitting
// the batch costs nothing, splitting time costs an exchange per tile, so time is only split
// where the batch leaves SMs without work.  Of packed sequences one may be long: time first,
// by 4, then the sequences.
struct ScanGrid {
    int groups, splits, cluster;
};
inline ScanGrid scan_grid(const ScanArgs& a, int sms, int per_sm, int tile) {
    ScanGrid g{(a.D + SC_CH - 1) / SC_CH, 1, 1};
    const int64_t tokens = a.cu ? a.T : (int64_t)a.B * a.T;
    auto clamp = [](int64_t v, int64_t hi) { return (int)(v < 1 ? 1 : (v > hi ? hi : v)); };
    const int want = clamp(per_sm * sms / g.groups, 65535);
    g.splits = a.cu ? clamp(want / 4, a.n_seqs) : clamp(want, a.B);
    const int64_t tiles = (tokens / g.splits + tile) / tile;  // one at least
    const bool few = (int64_t)g.groups * g.splits * SC_MAX_CLUSTER <= sms;
    g.cluster = clamp(clamp(want / g.splits, few ? SC_MAX_CLUSTER : 4), tiles);
    return g;
}

template <auto KERNEL>
cudaError_t scan_launch(int (*smem)(int), int tile, const ScanArgs& a, const ScanMaps& maps, int width,
                        cudaStream_t stream) {
    static std::atomic<uint64_t> ready{0};  // devices on which this kernel may use its shared memory
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
        if ((e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, smem(SC_MAX_CLUSTER))) !=
            cudaSuccess)
            return e;
        if (dev < 64) ready.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
    }
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    const ScanGrid g = scan_grid(a, sms, 2 * (smem(4) + 1024) <= 228 * 1024 ? 2 : 1, tile);
    if ((int64_t)g.groups * g.cluster > INT32_MAX) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(g.groups * g.cluster), (unsigned)g.splits);
    cfg.blockDim = dim3(SC_THREADS);
    cfg.dynamicSmemBytes = smem(g.cluster);
    cfg.stream = stream;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = g.cluster;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = g.cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, KERNEL, a, maps, g.cluster, width);
}

}  // namespace kda
