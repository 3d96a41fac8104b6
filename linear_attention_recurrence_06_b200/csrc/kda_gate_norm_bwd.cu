// kda_gate_norm_bwd.cu -- gradients of the per-head RMSNorm and sigmoid output
// gate (include/kda.h, kda_gate_norm_bwd).  HBM-bound: three rows in, two out.
#include "kda_launch.h"
#include "kda_sm100.cuh"

namespace kda {

namespace {

constexpr int D = 128;
constexpr int GNB_WARPS = 8;

KDA_DEV float warp_sum(float v) {
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

// A warp per row, 4 channels (lane + 32 j) per lane; d_norm_weight: every warp sums its
// rows in registers, a CTA its warps through shared memory, and the second kernel the
// CTAs, each in a fixed order.
template <bool IN_BF16, bool OUT_BF16>
__global__ void __launch_bounds__(GNB_WARPS * 32)
gate_norm_bwd_kernel(const void* o, const void* g, const void* dy, const float* w, float eps, void* d_o, void* d_g,
                     float* partial, int64_t rows) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float wv[4], dw[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 4; ++j) wv[j] = w ? w[lane + 32 * j] : 1.f;
    for (int64_t row = (int64_t)blockIdx.x * GNB_WARPS + warp; row < rows; row += (int64_t)gridDim.x * GNB_WARPS) {
        float ov[4], s[4], y[4], ss = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const size_t i = (size_t)row * D + lane + 32 * j;
            ov[j] = ld_in<IN_BF16>(o, i);
            y[j] = ld_in<IN_BF16>(dy, i);
            s[j] = __fdividef(1.f, 1.f + __expf(-ld_in<IN_BF16>(g, i)));
            ss += ov[j] * ov[j];
        }
        const float r = rsqrtf(warp_sum(ss) * (1.f / D) + eps);
        float dot = 0.f, dn[4], nv[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            nv[j] = ov[j] * r;
            const float ys = y[j] * s[j];
            dn[j] = ys * wv[j];
            dot += dn[j] * nv[j];
            dw[j] += ys * nv[j];
        }
        dot = warp_sum(dot) * (1.f / D);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const size_t i = (size_t)row * D + lane + 32 * j;
            st_out<OUT_BF16>(d_o, i, r * (dn[j] - nv[j] * dot));
            st_out<OUT_BF16>(d_g, i, dn[j] * nv[j] * (1.f - s[j]));
        }
    }
    if (!partial) return;
    __shared__ float sh[GNB_WARPS][D];
#pragma unroll
    for (int j = 0; j < 4; ++j) sh[warp][lane + 32 * j] = dw[j];
    __syncthreads();
    if (threadIdx.x < D) {
        float t = 0.f;
        for (int k = 0; k < GNB_WARPS; ++k) t += sh[k][threadIdx.x];
        partial[(size_t)blockIdx.x * D + threadIdx.x] = t;
    }
}

__global__ void __launch_bounds__(D) gate_norm_dw_kernel(const float* partial, int n, float* dw) {
    float t = 0.f;
    for (int k = 0; k < n; ++k) t += partial[(size_t)k * D + threadIdx.x];
    dw[threadIdx.x] = t;
}

}  // namespace

int gate_norm_bwd_blocks(int64_t rows) {
    const int64_t need = (rows + GNB_WARPS - 1) / GNB_WARPS, cap = 148 * 4;
    return (int)(need < cap ? need : cap);
}

cudaError_t launch_gate_norm_bwd(const void* o, const void* g, const void* dy, const float* w, float eps, void* d_o,
                                 void* d_g, float* dw, int64_t rows, bool in_bf16, bool out_bf16, float* partial,
                                 cudaStream_t stream) {
    const int blocks = gate_norm_bwd_blocks(rows);
    if (!dw) partial = nullptr;
    if (blocks > 0) {
#define KDA_GNB(IB, OB) \
    gate_norm_bwd_kernel<IB, OB><<<blocks, GNB_WARPS * 32, 0, stream>>>(o, g, dy, w, eps, d_o, d_g, partial, rows)
        if (in_bf16) { if (out_bf16) KDA_GNB(true, true); else KDA_GNB(true, false); }
        else         { if (out_bf16) KDA_GNB(false, true); else KDA_GNB(false, false); }
#undef KDA_GNB
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (dw) gate_norm_dw_kernel<<<1, D, 0, stream>>>(partial, blocks, dw);
    return cudaGetLastError();
}

}  // namespace kda
