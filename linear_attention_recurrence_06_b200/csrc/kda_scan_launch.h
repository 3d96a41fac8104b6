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

// The widest copy that every input's address and token stride allow (16: TMA, where D is even), and
// the tensor maps for it.
inline cudaError_t scan_maps(const ScanArgs& a, const void* const* in, const int64_t* ld, int n, int box_rows,
                             ScanMaps* maps, int* width) {
    memset(maps, 0, sizeof(*maps));
    const int64_t tokens = a.cu ? a.T : (int64_t)a.B * a.T;
    uintptr_t all = 0;
    for (int i = 0; i < n; ++i) all |= reinterpret_cast<uintptr_t>(in[i]) | (uintptr_t)(ld[i] * (a.in_bf16 ? 2 : 4));
    *width = all % 16 == 0 && a.D % 2 == 0 ? 16 : (all % 4 == 0 ? 4 : 2);
    if (*width == 16 && tokens > 0)
        for (int i = 0; i < n; ++i)
            if (!make_scan_map(&maps->m[i], in[i], tokens, a.D, ld[i], box_rows, a.in_bf16)) return cudaErrorInvalidValue;
    return cudaSuccess;
}

// dependent: the kernel ahead is one of the scan's (the check of cu_seqlens, or the forward that writes
// the chunk states), which lets this one start beside it: launch, set-up and first loads of the call's
// inputs, which were complete when that one began, overlap its end.
//
// Splits of the batch and cluster.  Splitting the batch costs nothing, splitting time costs an
// exchange per tile, so time is only split where the batch leaves SMs without work; of packed
// sequences one may be long, so there time comes first, by up to 4, but not by more than
// half of what the GPU takes (scan_span).  The cluster is then the largest of which all run at
// once: a second wave doubles the time (16 clusters of 8, of which not all find room,
// took 67 us for 8192 x 1024 values; as clusters of 7, 42 us).
// Work that fills the GPU is cut finer, into up to 4 times as many splits, so that SMs which
// have done their part find more (14 % off 16 x 8192 x 4096, 21 % off 6 x 4096 x 4096, 23 % off 125,841
// tokens in 16 packed sequences x 4096, in 8 splits of 2 instead of 1 of 4), as long as a CTA
// has 2,048 tokens, about 20 us: its start costs several (4,620 tokens x 1000 take a fifth longer
// in splits of 144 than of 288).
constexpr int64_t SC_PART_TOKENS = 2048;
template <auto KERNEL>
cudaError_t scan_launch(int (*smem)(int), int tile, const ScanArgs& a, const ScanMaps& maps, int width,
                        bool dependent, cudaStream_t stream) {
    static std::atomic<uint64_t> ready{0};           // devices on which this kernel may use its shared memory
    static std::atomic<int> active[64][SC_MAX_CLUSTER + 1];  // clusters of a size that run at once, + 1
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64) return cudaErrorInvalidDevice;
    if (!(ready.load(std::memory_order_relaxed) >> dev & 1)) {
        if ((e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, smem(SC_MAX_CLUSTER))) !=
            cudaSuccess)
            return e;
        ready.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
    }
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;

    auto clamp = [](int64_t v, int64_t hi) { return (int)(v < 1 ? 1 : (v > hi ? hi : v)); };
    const int groups = (a.D + SC_CH - 1) / SC_CH;
    const int64_t tokens = a.cu ? a.T : (int64_t)a.B * a.T;
    const int per_sm = 2 * (smem(4) + 1024) <= 228 * 1024 ? 2 : 1;
    const int want = clamp(per_sm * sms / groups, 65535);
    const int at_once = a.cu ? clamp(want / clamp(want / 2, 4), a.n_seqs) : clamp(want, a.B);
    int cluster = clamp(clamp(want / at_once, SC_MAX_CLUSTER), (tokens / at_once + tile) / tile);
    int splits = clamp(tokens / (SC_PART_TOKENS * cluster), a.cu ? a.n_seqs : a.B);
    splits = splits < at_once ? at_once : clamp(splits, 4 * (int64_t)at_once);
    if (!a.cu) {
        const int each = (a.B + splits - 1) / splits;  // sequences of a split
        splits = (a.B + each - 1) / each;
    }

    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(SC_THREADS);
    cfg.stream = stream;
    cudaLaunchAttribute at[2] = {};
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    for (;; --cluster) {
        cfg.gridDim = dim3((unsigned)(groups * cluster), (unsigned)splits);
        cfg.dynamicSmemBytes = smem(cluster);
        cfg.numAttrs = cluster > 1 ? 1 : 0;
        at[0].val.clusterDim.x = cluster;
        if (cluster == 1) break;
        int n = active[dev][cluster].load(std::memory_order_relaxed) - 1;
        if (n < 0) {
            if ((e = cudaOccupancyMaxActiveClusters(&n, KERNEL, &cfg)) != cudaSuccess) return e;
            active[dev][cluster].store(n + 1, std::memory_order_relaxed);
        }
        if ((int64_t)groups * at_once <= n) break;
    }
    if (dependent) cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, KERNEL, a, maps, cluster, width);
}

}  // namespace kda
