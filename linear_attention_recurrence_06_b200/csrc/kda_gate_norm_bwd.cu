// kda_gate_norm_bwd.cu -- gradients of the per-head RMSNorm and sigmoid output
// gate (include/kda.h, kda_gate_norm_bwd).  HBM-bound: three rows in, two out.
//
// Half a warp per row of 128 (8 channels per lane, 16 bytes of bf16), as the forward; both
// row sums (o^2, then dn n) by shuffles, everything else in registers.  A row's loads are on their
// way while the row before it is worked on, which 8 registers for the weights would not leave
// room for (those come from shared memory).  d_norm_weight is summed in a fixed order: each lane over
// the rows of its half warp, a CTA's half warps through shared memory, the CTAs by a second
// kernel, whose launch overlaps the first's end.
// 262,144 rows in bf16: 54 us, 6.2 TB/s of the 6.5 that a copy reaches (8 us more without the loads
// ahead), 2 us of it the second kernel; fp32 122 us, 5.5 TB/s (592 CTAs where 444 run at once; those kernels spill
// 28 bytes, bf16 inputs with fp32 gradients 12); 602 rows: 3.6 us, most of it the two launches.
#include <float.h>

#include "kda_launch.h"
#include "kda_sm100.cuh"

namespace kda {

namespace {

constexpr int D = 128;
constexpr int GNB_THREADS = 256, GNB_HALVES = GNB_THREADS / 16;
constexpr int GNB_MAX_BLOCKS = 148 * 4;

// 8 values as they lie in memory, so that a row can be on its way while the one before it is worked on
template <bool BF16>
struct Raw8 {
    uint4 w[BF16 ? 1 : 2];
    KDA_DEV void load(const void* base, size_t i, bool in) {
        const uint4* const p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + i * (BF16 ? 2 : 4));
#pragma unroll
        for (int k = 0; k < (BF16 ? 1 : 2); ++k) w[k] = in ? __ldg(p + k) : make_uint4(0u, 0u, 0u, 0u);
    }
    KDA_DEV void get(float* v) const {
#pragma unroll
        for (int k = 0; k < (BF16 ? 1 : 2); ++k) {
            const uint32_t ww[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                if constexpr (BF16) {
                    v[2 * p] = __uint_as_float(ww[p] << 16);
                    v[2 * p + 1] = __uint_as_float(ww[p] & 0xFFFF0000u);
                } else {
                    v[4 * k + p] = __uint_as_float(ww[p]);
                }
            }
        }
    }
};
template <bool BF16>
KDA_DEV void store8(void* base, size_t i, const float* v) {
    if constexpr (BF16) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + i) =
            make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    } else {
        float4* const p = reinterpret_cast<float4*>(static_cast<float*>(base) + i);
        p[0] = make_float4(v[0], v[1], v[2], v[3]);
        p[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
}
KDA_DEV float half_warp_sum(float v) {
#pragma unroll
    for (int m = 8; m >= 1; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

template <bool IN_BF16, bool OUT_BF16>
__global__ void __launch_bounds__(GNB_THREADS, IN_BF16 ? 4 : 3)
gate_norm_bwd_kernel(const void* __restrict__ o, const void* __restrict__ g, const void* __restrict__ dy,
                     const float* __restrict__ w, float eps, void* __restrict__ d_o, void* __restrict__ d_g,
                     float* __restrict__ partial, int64_t rows) {
    pdl_trigger();
    const int sub = threadIdx.x & 15, half = threadIdx.x >> 4;
    __shared__ float sw[D];  // 8 registers per thread that a row on its way needs more
    if (threadIdx.x < D) sw[threadIdx.x] = w ? __ldg(w + threadIdx.x) : 1.f;
    float dw[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    // pairs of rows, so that both halves of a warp take the same number of turns
    const int64_t step = (int64_t)gridDim.x * GNB_HALVES;
    int64_t row = (int64_t)blockIdx.x * GNB_HALVES + half;
    Raw8<IN_BF16> ro, rg, ry;
    auto fetch = [&](int64_t r) {
        const size_t i = (size_t)r * D + sub * 8;
        const bool in = r < rows;
        ro.load(o, i, in);
        rg.load(g, i, in);
        ry.load(dy, i, in);
    };
    fetch(row);
    __syncthreads();
    for (; row - (half & 1) < rows; row += step) {
        const bool in = row < rows;
        const size_t i = (size_t)row * D + sub * 8;
        float ov[8], s[8], y[8];
        ro.get(ov);
        rg.get(s);
        ry.get(y);
        fetch(row + step);
        float ss = 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            ss += ov[c] * ov[c];
            s[c] = __expf(-s[c]);
        }
        ss = half_warp_sum(ss);
        // a row past the end is all zeros and adds nothing to dw, with eps = 0 too
        const float r = in ? rsqrtf(ss * (1.f / D) + eps) : 0.f;
        float dot = 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const float sig = __fdividef(1.f, 1.f + s[c]);
            ov[c] *= r;                // n
            y[c] *= sig;               // dy s
            s[c] = fminf(s[c], FLT_MAX) * sig;  // 1 - s = e^-g s keeps its digits where s is next to 1 (s = 0: times 0)
            dw[c] += y[c] * ov[c];
            y[c] *= sw[sub * 8 + c];   // dn
            dot += y[c] * ov[c];
        }
        dot = half_warp_sum(dot) * (1.f / D);
        if (!in) continue;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            s[c] = y[c] * ov[c] * s[c];
            y[c] = r * (y[c] - ov[c] * dot);
        }
        store8<OUT_BF16>(d_o, i, y);
        store8<OUT_BF16>(d_g, i, s);
    }
    if (!partial) return;
    __shared__ float sh[GNB_HALVES][D];
#pragma unroll
    for (int c = 0; c < 8; ++c) sh[half][sub * 8 + c] = dw[c];
    __syncthreads();
    if (threadIdx.x < D) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < GNB_HALVES; ++k) t += sh[k][threadIdx.x];
        partial[(size_t)blockIdx.x * D + threadIdx.x] = t;
    }
}

// 16 CTAs of 8 columns: 32 partial sums over the rows of `partial`, then their sum.
__global__ void __launch_bounds__(256) gate_norm_dw_kernel(const float* __restrict__ partial, int n, float* dw) {
    __shared__ float sh[32][8];
    const int c = threadIdx.x & 7, k = threadIdx.x >> 3, col = blockIdx.x * 8 + c;
    pdl_wait();
    float v[GNB_MAX_BLOCKS / 32 + 1], t = 0.f;  // all on their way at once
#pragma unroll
    for (int i = 0; i <= GNB_MAX_BLOCKS / 32; ++i) v[i] = k + 32 * i < n ? partial[(size_t)(k + 32 * i) * D + col] : 0.f;
#pragma unroll
    for (int i = 0; i <= GNB_MAX_BLOCKS / 32; ++i) t += v[i];
    sh[k][c] = t;
    __syncthreads();
    if (threadIdx.x < 8) {
        t = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) t += sh[i][c];
        dw[col] = t;
    }
}

}  // namespace

int gate_norm_bwd_blocks(int64_t rows) {
    const int64_t need = (rows + GNB_HALVES - 1) / GNB_HALVES;
    return (int)(need < GNB_MAX_BLOCKS ? need : GNB_MAX_BLOCKS);
}

cudaError_t launch_gate_norm_bwd(const void* o, const void* g, const void* dy, const float* w, float eps, void* d_o,
                                 void* d_g, float* dw, int64_t rows, bool in_bf16, bool out_bf16, float* partial,
                                 cudaStream_t stream) {
    const int blocks = gate_norm_bwd_blocks(rows);
    if (!dw) partial = nullptr;
    if (blocks > 0) {
#define KDA_GNB(IB, OB) \
    gate_norm_bwd_kernel<IB, OB><<<blocks, GNB_THREADS, 0, stream>>>(o, g, dy, w, eps, d_o, d_g, partial, rows)
        if (in_bf16) { if (out_bf16) KDA_GNB(true, true); else KDA_GNB(true, false); }
        else         { if (out_bf16) KDA_GNB(false, true); else KDA_GNB(false, false); }
#undef KDA_GNB
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (!dw) return cudaSuccess;
    if (blocks == 0) return cudaMemsetAsync(dw, 0, D * sizeof(float), stream);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(D / 8);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gate_norm_dw_kernel, (const float*)partial, blocks, dw);
}

}  // namespace kda
