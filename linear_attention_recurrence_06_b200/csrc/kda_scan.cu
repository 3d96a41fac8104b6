// kda_scan.cu -- element-wise gated scan (include/kda.h, kda_scan_fwd), forward
// and single tokens.
#include "kda_row_slot.cuh"
#include "kda_scan.h"
#include "kda_scan.cuh"

namespace kda {

namespace {

template <bool GATE, bool NORM>
__global__ void __launch_bounds__(128) scan_fwd_kernel(ScanArgs a) {
    const int ch = blockIdx.x * 128 + threadIdx.x, n = blockIdx.y;
    if (ch >= a.D) return;
    int64_t first, end;
    scan_range(a.cu, n, a.T, &first, &end);
    float h = a.init ? a.init[(size_t)n * a.D + ch] : 0.f;
    for (int64_t t = first; t < end; ++t) {
        if (a.chunk_states && t % SCAN_CHUNK == 0) a.chunk_states[(size_t)(t / SCAN_CHUNK) * a.D + ch] = h;
        const size_t ix = (size_t)t * a.ld_x + ch, il = (size_t)t * a.ld_l + ch, ig = (size_t)t * a.ld_g + ch;
        const float x = a.in_bf16 ? ld_in<true>(a.x, ix) : ld_in<false>(a.x, ix);
        const float l = a.in_bf16 ? ld_in<true>(a.log_alpha, il) : ld_in<false>(a.log_alpha, il);
        const float g = !GATE ? 0.f : a.in_bf16 ? ld_in<true>(a.gate, ig) : ld_in<false>(a.gate, ig);
        const ScanTerm r = scan_term<GATE, NORM>(x, l, g);
        h = scan_step(r.p, h, r.u);
        if (a.h) {
            const size_t io = (size_t)t * a.D + ch;
            if (a.out_bf16) st_out<true>(a.h, io, h);
            else st_out<false>(a.h, io, h);
        }
    }
    if (a.final_state) a.final_state[(size_t)n * a.D + ch] = h;
}

__global__ void scan_check_cu_kernel(const int32_t* cu, int n_seqs, int64_t T, uint32_t* status) {
    bool bad = threadIdx.x == 0 && cu[0] != 0;
    for (int i = threadIdx.x; i < n_seqs; i += blockDim.x) bad |= cu[i + 1] < cu[i] || cu[i + 1] > T;
    if (__syncthreads_or(bad) && threadIdx.x == 0) *status = 2u;
}

template <bool GATE, bool NORM>
__global__ void __launch_bounds__(128)
scan_decode_kernel(float* state, const void* x, const void* log_alpha, const void* gate, void* hout,
                   const int32_t* slots, int n_slots, int n_steps, int Bd, int D, bool in_bf16, bool out_bf16,
                   float* step_states) {
    const int ch = blockIdx.x * 128 + threadIdx.x, b = blockIdx.y;
    const int slot = slots ? row_slot(slots, n_slots, b) : b;
    if (ch >= D) return;
    float h = slot >= 0 ? state[(size_t)slot * D + ch] : 0.f;
    for (int t = 0; t < n_steps; ++t) {
        const size_t i = ((size_t)t * Bd + b) * D + ch;
        if (slot >= 0) {
            const float xv = in_bf16 ? ld_in<true>(x, i) : ld_in<false>(x, i);
            const float l = in_bf16 ? ld_in<true>(log_alpha, i) : ld_in<false>(log_alpha, i);
            const float g = !GATE ? 0.f : in_bf16 ? ld_in<true>(gate, i) : ld_in<false>(gate, i);
            const ScanTerm r = scan_term<GATE, NORM>(xv, l, g);
            h = scan_step(r.p, h, r.u);
        }
        if (out_bf16) st_out<true>(hout, i, h);
        else st_out<false>(hout, i, h);
        if (step_states) step_states[i] = h;
    }
    if (slot >= 0) state[(size_t)slot * D + ch] = h;
}

}  // namespace

#define KDA_SCAN_GN(GATE, NORM, CALL)                                    \
    do {                                                                 \
        if (GATE) {                                                      \
            if (NORM) { constexpr bool G = true, W = true; CALL; }       \
            else      { constexpr bool G = true, W = false; CALL; }      \
        } else {                                                         \
            if (NORM) { constexpr bool G = false, W = true; CALL; }      \
            else      { constexpr bool G = false, W = false; CALL; }     \
        }                                                                \
    } while (0)

cudaError_t launch_scan_check(const ScanArgs& a, cudaStream_t stream) {
    cudaError_t e = cudaMemsetAsync(a.status, 0, sizeof(uint32_t), stream);
    if (e != cudaSuccess || !a.cu) return e;
    scan_check_cu_kernel<<<1, 256, 0, stream>>>(a.cu, a.n_seqs, a.T, a.status);
    return cudaGetLastError();
}

cudaError_t launch_scan_fwd(const ScanArgs& a, cudaStream_t stream) {
    if (a.status) {
        const cudaError_t e = launch_scan_check(a, stream);
        if (e != cudaSuccess) return e;
    }
    const dim3 grid((a.D + 127) / 128, a.n_seqs);
    KDA_SCAN_GN(a.gate != nullptr, a.normalize, (scan_fwd_kernel<G, W><<<grid, 128, 0, stream>>>(a)));
    return cudaGetLastError();
}

cudaError_t launch_scan_decode(float* state, const void* x, const void* log_alpha, const void* gate, void* h,
                               const int32_t* slots, int n_slots, int n_steps, int Bd, int D, bool in_bf16,
                               bool out_bf16, bool normalize, float* step_states, cudaStream_t stream) {
    const dim3 grid((D + 127) / 128, Bd);
    KDA_SCAN_GN(gate != nullptr, normalize,
                (scan_decode_kernel<G, W><<<grid, 128, 0, stream>>>(state, x, log_alpha, gate, h, slots, n_slots,
                                                                    n_steps, Bd, D, in_bf16, out_bf16, step_states)));
    return cudaGetLastError();
}

}  // namespace kda
