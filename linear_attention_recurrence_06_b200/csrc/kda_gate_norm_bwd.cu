// kda_gate_norm_bwd.cu -- gradients of the per-head RMSNorm and sigmoid output
// gate (include/kda.h, kda_gate_norm_bwd).  HBM-bound: three rows in, two out.
//
// Half a warp per row of 128 (8 channels per lane, 16 bytes of bf16), as the forward; both
// row sums (o^2, then dn n) by shuffles, everything else in registers.  d_norm_weight is summed in
// a fixed order: each lane over the rows of its half warp, a CTA's half warps through shared
// memory, the CTAs by a second kernel, whose launch overlaps the first's end.
#include "kda_launch.h"
#include "kda_sm100.cuh"

namespace kda {

namespace {

constexpr int D = 128;
constexpr int GNB_THREADS = 256, GNB_HALVES = GNB_THREADS / 16;
constexpr int GNB_MAX_BLOCKS = 148 * 4;

template <bool BF16>
KDA_DEV void load8(const void* base, size_t i, float* v) {
    if constexpr (BF16) {
        const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i);
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            v[2 * p] = __uint_as_float(ww[p] << 16);
            v[2 * p + 1] = __uint_as_float(ww[p] & 0xFFFF0000u);
        }
    } else {
        const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
        const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + i + 4);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
}
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
__global__ void __launch_bounds__(GNB_THREADS, 4)
gate_norm_bwd_kernel(const void* __restrict__ o, const void* __restrict__ g, const void* __restrict__ dy,
                     const float* __restrict__ w, float eps, void* __restrict__ d_o, void* __restrict__ d_g,
                     float* __restrict__ partial, int64_t rows) {
    pdl_trigger();
    const int sub = threadIdx.x & 15, half = threadIdx.x >> 4;
    float wv[8], dw[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        wv[c] = w ? __ldg(w + sub * 8 + c) : 1.f;
        dw[c] = 0.f;
    }
    // pairs of rows, so that both halves of a warp take the same number of turns
    for (int64_t pair = (int64_t)blockIdx.x * (GNB_HALVES / 2) + (half >> 1); 2 * pair < rows;
         pair += (int64_t)gridDim.x * (GNB_HALVES / 2)) {
        const int64_t row = 2 * pair + (half & 1);
        const bool in = row < rows;
        const size_t i = (size_t)row * D + sub * 8;
        float ov[8], s[8], y[8];
        if (in) {
            load8<IN_BF16>(o, i, ov);
            load8<IN_BF16>(g, i, s);
            load8<IN_BF16>(dy, i, y);
        } else {
#pragma unroll
            for (int c = 0; c < 8; ++c) ov[c] = s[c] = y[c] = 0.f;
        }
        float ss = 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            ss += ov[c] * ov[c];
            s[c] = __fdividef(1.f, 1.f + __expf(-s[c]));
        }
        const float r = rsqrtf(half_warp_sum(ss) * (1.f / D) + eps);
        float dot = 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            ov[c] *= r;                // n
            y[c] *= s[c];              // dy s
            dw[c] += y[c] * ov[c];
            y[c] *= wv[c];             // dn
            dot += y[c] * ov[c];
        }
        dot = half_warp_sum(dot) * (1.f / D);
        if (!in) continue;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            s[c] = y[c] * ov[c] * (1.f - s[c]);
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
    float t = 0.f;
#pragma unroll 4
    for (int i = k; i < n; i += 32) t += partial[(size_t)i * D + col];
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
