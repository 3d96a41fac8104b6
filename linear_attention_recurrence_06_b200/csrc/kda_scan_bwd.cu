// kda_scan_bwd.cu -- gradients of the element-wise gated scan (include/kda.h,
// kda_scan_bwd).  The states inside a chunk of 64 tokens are computed again from
// the state before it; then the gradient G_t = dh_t + a_{t+1} G_{t+1} walks back.
#include "kda_scan.h"
#include "kda_scan.cuh"

namespace kda {

namespace {

template <bool GATE, bool NORM>
__global__ void __launch_bounds__(128) scan_bwd_kernel(ScanArgs a) {
    const int ch = blockIdx.x * 128 + threadIdx.x, n = blockIdx.y;
    if (ch >= a.D) return;
    int64_t first, end;
    scan_range(a.cu, n, a.T, &first, &end);
    const float h0 = a.init ? a.init[(size_t)n * a.D + ch] : 0.f;
    float c = a.d_final ? a.d_final[(size_t)n * a.D + ch] : 0.f;  // a_{t+1} G_{t+1}
    auto in = [&](const void* p, int64_t t, int64_t ld) {
        const size_t i = (size_t)t * ld + ch;
        return a.in_bf16 ? ld_in<true>(p, i) : ld_in<false>(p, i);
    };
    auto out = [&](void* p, int64_t t, float v) {
        const size_t i = (size_t)t * a.D + ch;
        if (a.out_bf16) st_out<true>(p, i, v);
        else st_out<false>(p, i, v);
    };
    float hp[SCAN_CHUNK];  // the state before each token of the chunk
    for (int64_t ce = end; ce > first;) {
        int64_t cs = (ce - 1) / SCAN_CHUNK * SCAN_CHUNK;
        float h = cs > first ? a.chunk_states[(size_t)(cs / SCAN_CHUNK) * a.D + ch] : h0;
        if (cs < first) cs = first;
        for (int64_t t = cs; t < ce; ++t) {
            hp[t - cs] = h;
            const ScanTerm r = scan_term<GATE, NORM>(in(a.x, t, a.ld_x), in(a.log_alpha, t, a.ld_l),
                                                     GATE ? in(a.gate, t, a.ld_g) : 0.f);
            h = scan_step(r.p, h, r.u);
        }
        for (int64_t t = ce - 1; t >= cs; --t) {
            const float l = in(a.log_alpha, t, a.ld_l);
            const ScanTerm r = scan_term<GATE, NORM>(in(a.x, t, a.ld_x), l, GATE ? in(a.gate, t, a.ld_g) : 0.f);
            const float G = in(a.d_h, t, a.ld_dh) + c;
            out(a.dx, t, G * r.ws);
            float dl = scan_a(r.p) * hp[t - cs];
            if (NORM) dl += scan_du_dl(r);
            out(a.dl, t, l > 0.f ? 0.f : G * dl);
            if (GATE) out(a.dg, t, G * r.u * (1.f - r.s));
            c = scan_step(r.p, G, 0.f);
        }
        ce = cs;
    }
    if (a.d_init) a.d_init[(size_t)n * a.D + ch] = c;
}

}  // namespace

cudaError_t launch_scan_bwd(const ScanArgs& a, bool own_states, cudaStream_t stream) {
    cudaError_t e;
    if (own_states) {
        ScanArgs f = a;
        f.h = nullptr, f.final_state = nullptr;
        if ((e = launch_scan_fwd(f, stream)) != cudaSuccess) return e;
    } else if (a.status && (e = launch_scan_check(a, stream)) != cudaSuccess) {
        return e;
    }
    const dim3 grid((a.D + 127) / 128, a.n_seqs);
    if (a.gate) {
        if (a.normalize) scan_bwd_kernel<true, true><<<grid, 128, 0, stream>>>(a);
        else scan_bwd_kernel<true, false><<<grid, 128, 0, stream>>>(a);
    } else {
        if (a.normalize) scan_bwd_kernel<false, true><<<grid, 128, 0, stream>>>(a);
        else scan_bwd_kernel<false, false><<<grid, 128, 0, stream>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace kda
