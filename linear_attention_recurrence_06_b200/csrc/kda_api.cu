// kda_api.cu -- the extern "C" boundary of libkda (declared in include/kda.h).
// Host-side argument checks happen before any launch; every entry point is
// asynchronous on the caller's stream except kda_query_status.
#include <cuda_runtime.h>
#include <stdint.h>

#include <string.h>

#include <vector>

#include "../../include/kda.h"
#include "kda_launch.h"
#include "kda_profile.h"
#include "kda_scan.h"


namespace kda {
namespace {
struct ProfRec {
    int kind;
    cudaEvent_t start, stop;
};
bool g_prof_on = false;
std::vector<ProfRec> g_prof_open;     // begun, not yet ended (at most one per kind)
std::vector<ProfRec> g_prof_done;     // waiting to be read
std::vector<cudaEvent_t> g_event_pool;

cudaEvent_t pool_event() {
    if (!g_event_pool.empty()) {
        cudaEvent_t e = g_event_pool.back();
        g_event_pool.pop_back();
        return e;
    }
    cudaEvent_t e = nullptr;
    cudaEventCreate(&e);
    return e;
}
}  // namespace

bool prof_enabled() { return g_prof_on; }

void prof_begin(int kind, cudaStream_t stream) {
    if (!g_prof_on) return;
    ProfRec r{kind, pool_event(), pool_event()};
    cudaEventRecord(r.start, stream);
    g_prof_open.push_back(r);
}

void prof_end(int kind, cudaStream_t stream) {
    if (!g_prof_on) return;
    for (size_t i = g_prof_open.size(); i-- > 0;) {
        if (g_prof_open[i].kind == kind) {
            cudaEventRecord(g_prof_open[i].stop, stream);
            g_prof_done.push_back(g_prof_open[i]);
            g_prof_open.erase(g_prof_open.begin() + (long)i);
            return;
        }
    }
}
}  // namespace kda

namespace {

constexpr int kSupportedD = 128;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }  // vectors of slots
bool dtype_ok(int d) { return d == KDA_F32 || d == KDA_BF16; }

int num_sms_cached() {
    static int sms = 0;
    if (sms == 0) {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
            sms = 148;
    }
    return sms;
}

kda_status from_cuda(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

}  // namespace

extern "C" {

const char* kda_status_string(int status) {
    switch (status) {
        case KDA_OK: return "KDA_OK";
        case KDA_ERR_INVALID_ARG: return "KDA_ERR_INVALID_ARG: null pointer, bad size or bad dtype";
        case KDA_ERR_UNSUPPORTED: return "KDA_ERR_UNSUPPORTED: only dk = dv = 128 is implemented";
        case KDA_ERR_MISALIGNED: return "KDA_ERR_MISALIGNED: pointers must be 16-byte aligned";
        case KDA_ERR_WORKSPACE: return "KDA_ERR_WORKSPACE: workspace missing or too small";
        case KDA_ERR_CUDA: return "KDA_ERR_CUDA: a CUDA call or kernel launch failed";
        case KDA_ERR_TIMEOUT: return "KDA_ERR_TIMEOUT: a bounded device-side wait gave up";
        case KDA_ERR_DEVICE_ARG: return "KDA_ERR_DEVICE_ARG: cu_seqlens inconsistent with T or max_seqlen";
        default: return "KDA_ERR_UNKNOWN";
    }
}

int kda_version(void) { return 100; }

kda_status kda_chunk_fwd_workspace_size(int64_t T, int H, int dk, int dv, int n_seqs, int64_t max_seqlen,
                                        size_t* bytes_min, size_t* bytes_full) {
    if (T < 0 || H <= 0 || n_seqs < 0 || max_seqlen < 0 || (!bytes_min && !bytes_full)) return KDA_ERR_INVALID_ARG;
    if (dk != kSupportedD || dv != kSupportedD) return KDA_ERR_UNSUPPORTED;
    // the carry is only needed when final_state is NULL; report the size that
    // covers both cases
    const size_t fixed = kda::chunk_fixed_bytes(n_seqs, H, true);
    const size_t per_wc = (size_t)n_seqs * H * kda::chunk_slot_bytes();
    const int64_t nchunks = (max_seqlen + 63) / 64;
    const size_t head = (fixed + 1023) & ~(size_t)1023;
    if (bytes_min) *bytes_min = head + per_wc + 1024;
    if (bytes_full) *bytes_full = head + per_wc * (size_t)(nchunks > 0 ? nchunks : 1) + 1024;
    return KDA_OK;
}

kda_status kda_chunk_fwd_segmented_workspace_size(int64_t T, int H, int dk, int dv, int n_seqs, int64_t max_seqlen,
                                                  int segments, size_t* bytes) {
    if (segments < 1 || !bytes) return KDA_ERR_INVALID_ARG;
    size_t full = 0;
    const kda_status st = kda_chunk_fwd_workspace_size(T, H, dk, dv, n_seqs, max_seqlen, nullptr, &full);
    if (st != KDA_OK) return st;
    *bytes = full + (segments > 1 ? kda::chunk_seg_bytes(n_seqs, H, segments) : 0);
    return KDA_OK;
}

static kda_status chunk_fwd_impl(const void* q, const void* k, const void* v, const void* log_alpha,
                                 const void* beta, const float* init_state, void* o, float* final_state, int B,
                                 int64_t T, int H, int dk, int dv, const int32_t* cu_seqlens, int n_seqs,
                                 int64_t max_seqlen, kda_dtype in_dtype, kda_dtype out_dtype, float scale,
                                 const void* gate, const float* norm_weight, float eps, float* checkpoints,
                                 int64_t ckpt_tokens, int segments, void* workspace, size_t workspace_bytes,
                                 void* stream, int kcp_mode = kda::KCP_NONE, float* transition = nullptr) {
    // the finishing half of the cross-device form reads no token inputs, the
    // transition half writes no outputs; with no tokens at all (an empty segment
    // of a sequence split over devices) the token buffers may be NULL
    const bool has_tokens = B > 0 && T > 0;
    if (has_tokens && kcp_mode != kda::KCP_FINISH && (!q || !k || !v || !log_alpha || !beta))
        return KDA_ERR_INVALID_ARG;
    if (has_tokens && kcp_mode != kda::KCP_TRANSITION && !o) return KDA_ERR_INVALID_ARG;
    if (kcp_mode == kda::KCP_TRANSITION && !transition) return KDA_ERR_INVALID_ARG;
    if (B <= 0 || T < 0 || H <= 0 || !dtype_ok(in_dtype) || !dtype_ok(out_dtype)) return KDA_ERR_INVALID_ARG;
    if (dk != kSupportedD || dv != kSupportedD) return KDA_ERR_UNSUPPORTED;
    if (H > 65535 || (cu_seqlens ? n_seqs : B) > 65535) return KDA_ERR_UNSUPPORTED;  // grid y / z extents
    if (cu_seqlens) {
        if (B != 1 || n_seqs <= 0 || max_seqlen < 0 || max_seqlen > T) return KDA_ERR_INVALID_ARG;
        if (T > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    } else {
        n_seqs = B;
        max_seqlen = T;
    }
    if ((int64_t)B * T * H * 128 / 128 != (int64_t)B * T * H) return KDA_ERR_INVALID_ARG;
    if (eps < 0.f) return KDA_ERR_INVALID_ARG;
    if (checkpoints && (ckpt_tokens <= 0 || ckpt_tokens % 64 != 0)) return KDA_ERR_INVALID_ARG;
    if (segments < 1) return KDA_ERR_INVALID_ARG;
    const void* ptrs[] = {q, k, v, log_alpha, beta, init_state, o, final_state, cu_seqlens, gate, norm_weight, workspace,
                          checkpoints, transition};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_MISALIGNED;
    if (!workspace) return KDA_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return KDA_ERR_MISALIGNED;
    size_t need_min = 0;
    const int64_t tot = T * (cu_seqlens ? 1 : B);
    const kda_status wst =
        segments > 1 ? kda_chunk_fwd_segmented_workspace_size(tot, H, dk, dv, n_seqs, max_seqlen, segments, &need_min)
        : kcp_mode != kda::KCP_NONE
            ? kda_chunk_fwd_workspace_size(tot, H, dk, dv, n_seqs, max_seqlen, nullptr, &need_min)
            : kda_chunk_fwd_workspace_size(tot, H, dk, dv, n_seqs, max_seqlen, &need_min, nullptr);
    if (wst != KDA_OK) return KDA_ERR_INVALID_ARG;
    if (workspace_bytes < need_min) return KDA_ERR_WORKSPACE;

    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool in_bf16 = in_dtype == KDA_BF16, out_bf16 = out_dtype == KDA_BF16;
    bool fused = false;
    cudaError_t e = kda::chunk_fwd_launch(q, k, v, log_alpha, beta, init_state, o, final_state, B, T, H, cu_seqlens,
                                          n_seqs, max_seqlen, in_bf16, out_bf16, scale, gate, norm_weight, eps,
                                          checkpoints, ckpt_tokens, segments, kcp_mode, transition, workspace,
                                          workspace_bytes, st, nullptr,
                                          &fused);
    if (e != cudaSuccess) return KDA_ERR_CUDA;
    if (gate && !fused && kcp_mode != kda::KCP_TRANSITION) {
        const int64_t rows = (int64_t)B * T * H;
        // y overwrites o in place (o already holds out_dtype values)
        kda::prof_begin(kda::PROF_GATE_NORM, st);
        e = kda::launch_gate_norm(o, gate, norm_weight, eps, o, rows, out_bf16, in_bf16, out_bf16, num_sms_cached(),
                                  st);
        kda::prof_end(kda::PROF_GATE_NORM, st);
        if (e != cudaSuccess) return KDA_ERR_CUDA;
    }
    return KDA_OK;
}

kda_status kda_chunk_fwd_ckpt(const void* q, const void* k, const void* v, const void* log_alpha, const void* beta,
                              const float* init_state, void* o, float* final_state, int B, int64_t T, int H, int dk,
                              int dv, const int32_t* cu_seqlens, int n_seqs, int64_t max_seqlen, kda_dtype in_dtype,
                              kda_dtype out_dtype, float scale, const void* gate, const float* norm_weight, float eps,
                              float* checkpoints, int64_t ckpt_tokens, void* workspace, size_t workspace_bytes,
                              void* stream) {
    return chunk_fwd_impl(q, k, v, log_alpha, beta, init_state, o, final_state, B, T, H, dk, dv, cu_seqlens, n_seqs,
                          max_seqlen, in_dtype, out_dtype, scale, gate, norm_weight, eps, checkpoints, ckpt_tokens, 1,
                          workspace, workspace_bytes, stream);
}

kda_status kda_chunk_fwd_segmented(const void* q, const void* k, const void* v, const void* log_alpha,
                                   const void* beta, const float* init_state, void* o, float* final_state, int B,
                                   int64_t T, int H, int dk, int dv, const int32_t* cu_seqlens, int n_seqs,
                                   int64_t max_seqlen, kda_dtype in_dtype, kda_dtype out_dtype, float scale,
                                   const void* gate, const float* norm_weight, float eps, int segments,
                                   void* workspace, size_t workspace_bytes, void* stream) {
    return chunk_fwd_impl(q, k, v, log_alpha, beta, init_state, o, final_state, B, T, H, dk, dv, cu_seqlens, n_seqs,
                          max_seqlen, in_dtype, out_dtype, scale, gate, norm_weight, eps, nullptr, 0, segments,
                          workspace, workspace_bytes, stream);
}

kda_status kda_chunk_fwd(const void* q, const void* k, const void* v, const void* log_alpha, const void* beta,
                         const float* init_state, void* o, float* final_state, int B, int64_t T, int H, int dk,
                         int dv, const int32_t* cu_seqlens, int n_seqs, int64_t max_seqlen, kda_dtype in_dtype,
                         kda_dtype out_dtype, float scale, const void* gate, const float* norm_weight, float eps,
                         void* workspace, size_t workspace_bytes, void* stream) {
    return kda_chunk_fwd_ckpt(q, k, v, log_alpha, beta, init_state, o, final_state, B, T, H, dk, dv, cu_seqlens, n_seqs,
                              max_seqlen, in_dtype, out_dtype, scale, gate, norm_weight, eps, nullptr, 0, workspace,
                              workspace_bytes, stream);
}

kda_status kda_kcp_workspace_size(int64_t T, int H, int dk, int dv, int n_seqs, int64_t max_seqlen, size_t* bytes) {
    if (!bytes) return KDA_ERR_INVALID_ARG;
    return kda_chunk_fwd_workspace_size(T, H, dk, dv, n_seqs, max_seqlen, nullptr, bytes);
}

kda_status kda_kcp_transition(const void* q, const void* k, const void* v, const void* log_alpha, const void* beta,
                              int B, int64_t T, int H, int dk, int dv, const int32_t* cu_seqlens, int n_seqs,
                              int64_t max_seqlen, kda_dtype in_dtype, float scale, float* transition,
                              void* workspace, size_t workspace_bytes, void* stream) {
    return chunk_fwd_impl(q, k, v, log_alpha, beta, nullptr, nullptr, nullptr, B, T, H, dk, dv, cu_seqlens, n_seqs,
                          max_seqlen, in_dtype, in_dtype, scale, nullptr, nullptr, 0.f, nullptr, 0, 1, workspace,
                          workspace_bytes, stream, kda::KCP_TRANSITION, transition);
}

kda_status kda_kcp_compose(const float* transitions, int n_prev, const float* init_state, float* state_in,
                           int n_seqs, int H, int dk, int dv, void* stream) {
    if (!state_in || n_prev < 0 || (n_prev > 0 && !transitions) || n_seqs < 0 || H <= 0) return KDA_ERR_INVALID_ARG;
    if (dk != kSupportedD || dv != kSupportedD) return KDA_ERR_UNSUPPORTED;
    if (H > 65535 || n_seqs > 65535) return KDA_ERR_UNSUPPORTED;
    const void* ptrs[] = {transitions, init_state, state_in};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_MISALIGNED;
    return from_cuda(kda::launch_kcp_compose(transitions, n_prev, init_state, state_in, n_seqs, H,
                                             reinterpret_cast<cudaStream_t>(stream)));
}

kda_status kda_kcp_finish(const float* state_in, void* o, float* final_state, int B, int64_t T, int H, int dk, int dv,
                          const int32_t* cu_seqlens, int n_seqs, int64_t max_seqlen, kda_dtype in_dtype,
                          kda_dtype out_dtype, const void* gate, const float* norm_weight, float eps,
                          void* workspace, size_t workspace_bytes, void* stream) {
    return chunk_fwd_impl(nullptr, nullptr, nullptr, nullptr, nullptr, state_in, o, final_state, B, T, H, dk, dv,
                          cu_seqlens, n_seqs, max_seqlen, in_dtype, out_dtype, 1.f, gate, norm_weight, eps, nullptr, 0,
                          1, workspace, workspace_bytes, stream, kda::KCP_FINISH, nullptr);
}

kda_status kda_chunk_bwd_workspace_size(int64_t T, int H, int dk, int dv, int n_seqs, int64_t max_seqlen,
                                       size_t* bytes) {
    if (!bytes) return KDA_ERR_INVALID_ARG;
    size_t full = 0;
    const kda_status st = kda_chunk_fwd_workspace_size(T, H, dk, dv, n_seqs, max_seqlen, nullptr, &full);
    if (st != KDA_OK) return st;
    *bytes = full + kda::chunk_bwd_extra_bytes(n_seqs, H, max_seqlen);
    return KDA_OK;
}

kda_status kda_chunk_bwd(const void* q, const void* k, const void* v, const void* log_alpha, const void* beta,
                         const float* init_state, const void* d_o, const float* d_final_state, float* dq, float* dk,
                         float* dv, float* dlog_alpha, float* dbeta, float* d_init_state, int B, int64_t T, int H,
                         int dk_dim, int dv_dim, const int32_t* cu_seqlens, int n_seqs, int64_t max_seqlen,
                         kda_dtype in_dtype, float scale, void* workspace, size_t workspace_bytes, void* stream) {
    if (B <= 0 || T < 0 || H <= 0 || !dtype_ok(in_dtype)) return KDA_ERR_INVALID_ARG;
    if (dk_dim != kSupportedD || dv_dim != kSupportedD) return KDA_ERR_UNSUPPORTED;
    if (H > 65535 || (cu_seqlens ? n_seqs : B) > 65535) return KDA_ERR_UNSUPPORTED;
    const bool has_tokens = T > 0;
    if (has_tokens && (!q || !k || !v || !log_alpha || !beta || !d_o || !dq || !dk || !dv || !dlog_alpha || !dbeta))
        return KDA_ERR_INVALID_ARG;
    if (cu_seqlens) {
        if (B != 1 || n_seqs <= 0 || max_seqlen < 0 || max_seqlen > T) return KDA_ERR_INVALID_ARG;
        if (T > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    } else {
        n_seqs = B;
        max_seqlen = T;
    }
    const void* ptrs[] = {q,  k,  v,  log_alpha, beta,  init_state, d_o,          d_final_state, dq,
                          dk, dv, dlog_alpha, dbeta, d_init_state, cu_seqlens, workspace};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_MISALIGNED;
    if (!workspace) return KDA_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return KDA_ERR_MISALIGNED;
    const int64_t tot = T * (cu_seqlens ? 1 : B);
    size_t fwd_full = 0, need = 0;
    if (kda_chunk_fwd_workspace_size(tot, H, dk_dim, dv_dim, n_seqs, max_seqlen, nullptr, &fwd_full) != KDA_OK ||
        kda_chunk_bwd_workspace_size(tot, H, dk_dim, dv_dim, n_seqs, max_seqlen, &need) != KDA_OK)
        return KDA_ERR_INVALID_ARG;
    if (workspace_bytes < need) return KDA_ERR_WORKSPACE;
    const cudaError_t e = kda::chunk_bwd_launch(q, k, v, log_alpha, beta, init_state, d_o, d_final_state, dq, dk, dv,
                                                dlog_alpha, dbeta, d_init_state, B, T, H, cu_seqlens, n_seqs,
                                                max_seqlen, in_dtype == KDA_BF16, scale, workspace, fwd_full,
                                                reinterpret_cast<cudaStream_t>(stream));
    return from_cuda(e);
}

static kda_status decode_steps_impl(float* state, const int32_t* slots, int n_slots, const void* q, const void* k,
                                    const void* v, const void* log_alpha, const void* beta, void* o, int n_steps,
                                    int Bd, int H, int dk, int dv, kda_dtype in_dtype, kda_dtype out_dtype,
                                    float scale, const void* gate, const float* norm_weight, float eps,
                                    float* step_states, void* stream) {
    const bool no_pages = slots && n_slots == 0;  // all rows are padding
    if ((!state && !no_pages) || !q || !k || !v || !log_alpha || !beta || !o) return KDA_ERR_INVALID_ARG;
    if (n_steps < 0 || Bd < 0 || H <= 0 || !dtype_ok(in_dtype) || !dtype_ok(out_dtype) || eps < 0.f)
        return KDA_ERR_INVALID_ARG;
    if (dk != kSupportedD || dv != kSupportedD) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)Bd * H > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    const void* ptrs[] = {state, q, k, v, log_alpha, beta, o, gate, norm_weight, step_states};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_MISALIGNED;
    if (!aligned4(slots)) return KDA_ERR_MISALIGNED;
    if (Bd == 0 || n_steps == 0) return KDA_OK;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    kda::prof_begin(kda::PROF_DECODE, st);
    const cudaError_t e =
        slots ? kda::launch_decode_paged(state, slots, n_slots, q, k, v, log_alpha, beta, o, Bd, H,
                                         in_dtype == KDA_BF16, out_dtype == KDA_BF16, scale, gate, norm_weight, eps,
                                         n_steps, step_states, st)
              : kda::launch_decode_step(state, q, k, v, log_alpha, beta, o, Bd, H, in_dtype == KDA_BF16,
                                        out_dtype == KDA_BF16, scale, gate, norm_weight, eps, n_steps, step_states,
                                        st);
    kda::prof_end(kda::PROF_DECODE, st);
    return from_cuda(e);
}

kda_status kda_decode_steps(float* state, const void* q, const void* k, const void* v, const void* log_alpha,
                            const void* beta, void* o, int n_steps, int Bd, int H, int dk, int dv,
                            kda_dtype in_dtype, kda_dtype out_dtype, float scale, const void* gate,
                            const float* norm_weight, float eps, float* step_states, void* stream) {
    return decode_steps_impl(state, nullptr, 0, q, k, v, log_alpha, beta, o, n_steps, Bd, H, dk, dv, in_dtype,
                             out_dtype, scale, gate, norm_weight, eps, step_states, stream);
}

kda_status kda_decode_steps_paged(float* state, const int32_t* slots, int n_slots, const void* q, const void* k,
                                  const void* v, const void* log_alpha, const void* beta, void* o, int n_steps, int Bd,
                                  int H, int dk, int dv, kda_dtype in_dtype, kda_dtype out_dtype, float scale,
                                  const void* gate, const float* norm_weight, float eps, float* step_states,
                                  void* stream) {
    if (n_slots < 0) return KDA_ERR_INVALID_ARG;
    if ((Bd == 0 && n_steps >= 0) || (n_steps == 0 && Bd >= 0)) return KDA_OK;  // empty tensors may have no address
    if (!slots) return KDA_ERR_INVALID_ARG;
    return decode_steps_impl(state, slots, n_slots, q, k, v, log_alpha, beta, o, n_steps, Bd, H, dk, dv, in_dtype,
                             out_dtype, scale, gate, norm_weight, eps, step_states, stream);
}

kda_status kda_decode_step(float* state, const void* q, const void* k, const void* v, const void* log_alpha,
                           const void* beta, void* o, int Bd, int H, int dk, int dv, kda_dtype in_dtype,
                           kda_dtype out_dtype, float scale, const void* gate, const float* norm_weight, float eps,
                           void* stream) {
    return kda_decode_steps(state, q, k, v, log_alpha, beta, o, 1, Bd, H, dk, dv, in_dtype, out_dtype, scale, gate,
                            norm_weight, eps, nullptr, stream);
}

kda_status kda_gate_norm(const void* o, const void* gate, const float* norm_weight, float eps, void* y, int64_t rows,
                         int dv, kda_dtype in_dtype, kda_dtype out_dtype, void* stream) {
    if (!o || !gate || !y || rows < 0 || !dtype_ok(in_dtype) || !dtype_ok(out_dtype) || eps < 0.f)
        return KDA_ERR_INVALID_ARG;
    if (dv != kSupportedD) return KDA_ERR_UNSUPPORTED;
    if (y == o && in_dtype != out_dtype) return KDA_ERR_INVALID_ARG;  // in place needs equal element sizes
    const void* ptrs[] = {o, gate, norm_weight, y};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_MISALIGNED;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    kda::prof_begin(kda::PROF_GATE_NORM, st);
    const cudaError_t e = kda::launch_gate_norm(o, gate, norm_weight, eps, y, rows, in_dtype == KDA_BF16,
                                                in_dtype == KDA_BF16, out_dtype == KDA_BF16, num_sms_cached(), st);
    kda::prof_end(kda::PROF_GATE_NORM, st);
    return from_cuda(e);
}

}  // extern "C"

namespace {

// token strides: 0 stands for D
bool scan_strides(int D, int64_t* a, int64_t* b, int64_t* c, int64_t* d) {
    int64_t* const all[] = {a, b, c, d};
    for (int64_t* s : all) {
        if (!s) continue;
        if (*s == 0) *s = D;
        if (*s < D) return false;
    }
    return true;
}

bool element_aligned(const void* p, kda_dtype t) {
    return (reinterpret_cast<uintptr_t>(p) & (t == KDA_BF16 ? 1u : 3u)) == 0;
}

// The checks that the scan's two directions share.  Fills in n_seqs for a batch of equal lengths.
kda_status scan_check(const kda::ScanArgs& a, kda_dtype in_dtype, kda_dtype out_dtype, int* n_seqs, size_t ws_need,
                      const void* workspace, size_t workspace_bytes) {
    if (a.B <= 0 || a.T < 0 || a.D <= 0 || !dtype_ok(in_dtype) || !dtype_ok(out_dtype)) return KDA_ERR_INVALID_ARG;
    if (a.T > 0 && (!a.x || !a.log_alpha)) return KDA_ERR_INVALID_ARG;
    if (a.cu) {
        if (a.B != 1 || *n_seqs <= 0) return KDA_ERR_INVALID_ARG;
    } else {
        *n_seqs = a.B;
    }
    if (a.T > kda::SCAN_MAX_TOKENS / a.B || a.D > kda::SCAN_MAX_D) return KDA_ERR_UNSUPPORTED;
    const void* in[] = {a.x, a.log_alpha, a.gate, a.d_h};
    for (const void* p : in)
        if (p && !element_aligned(p, in_dtype)) return KDA_ERR_MISALIGNED;
    const void* ptrs[] = {a.init, a.h, a.final_state, a.chunk_states, a.d_final, a.dx, a.dl, a.dg, a.d_init};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_MISALIGNED;
    if (!aligned4(a.cu)) return KDA_ERR_MISALIGNED;
    if (workspace || ws_need) {
        if (!workspace || workspace_bytes < (ws_need ? ws_need : KDA_STATUS_BYTES)) return KDA_ERR_WORKSPACE;
        if (!aligned16(workspace)) return KDA_ERR_MISALIGNED;
    }
    return KDA_OK;
}

}  // namespace

extern "C" {

kda_status kda_scan_fwd(const void* x, const void* log_alpha, const void* gate, const float* init_state, void* h,
                        float* final_state, float* chunk_states, int B, int64_t T, int D, int64_t x_stride,
                        int64_t log_alpha_stride, int64_t gate_stride, const int32_t* cu_seqlens, int n_seqs,
                        kda_dtype in_dtype, kda_dtype out_dtype, int normalize, void* workspace,
                        size_t workspace_bytes, void* stream) {
    if (!scan_strides(D, &x_stride, &log_alpha_stride, &gate_stride, nullptr)) return KDA_ERR_INVALID_ARG;
    kda::ScanArgs a{};
    a.x = x, a.log_alpha = log_alpha, a.gate = gate;
    a.ld_x = x_stride, a.ld_l = log_alpha_stride, a.ld_g = gate_stride;
    a.init = init_state, a.cu = cu_seqlens, a.B = B, a.D = D, a.T = T;
    a.in_bf16 = in_dtype == KDA_BF16, a.out_bf16 = out_dtype == KDA_BF16, a.normalize = normalize != 0;
    a.status = static_cast<uint32_t*>(workspace);
    a.h = h, a.final_state = final_state, a.chunk_states = chunk_states;
    const kda_status st = scan_check(a, in_dtype, out_dtype, &n_seqs, 0, workspace, workspace_bytes);
    if (st != KDA_OK) return st;
    if (T > 0 && !h) return KDA_ERR_INVALID_ARG;
    a.n_seqs = n_seqs;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    kda::prof_begin(kda::PROF_SCAN, s);
    const cudaError_t e = kda::launch_scan_fwd(a, s);
    kda::prof_end(kda::PROF_SCAN, s);
    return from_cuda(e);
}

kda_status kda_scan_bwd_workspace_size(int B, int64_t T, int D, size_t* bytes) {
    if (B <= 0 || T < 0 || D <= 0 || !bytes) return KDA_ERR_INVALID_ARG;
    if (T > kda::SCAN_MAX_TOKENS / B || D > kda::SCAN_MAX_D) return KDA_ERR_UNSUPPORTED;
    const size_t chunks = (size_t)(((int64_t)B * T + KDA_SCAN_CHUNK - 1) / KDA_SCAN_CHUNK);
    *bytes = KDA_STATUS_BYTES + chunks * (size_t)D * sizeof(float);
    return KDA_OK;
}

kda_status kda_scan_bwd(const void* x, const void* log_alpha, const void* gate, const float* init_state,
                        const void* d_h, const float* d_final_state, const float* chunk_states, void* dx,
                        void* dlog_alpha, void* dgate, float* d_init_state, int B, int64_t T, int D, int64_t x_stride,
                        int64_t log_alpha_stride, int64_t gate_stride, int64_t d_h_stride, const int32_t* cu_seqlens,
                        int n_seqs, kda_dtype in_dtype, kda_dtype grad_dtype, int normalize, void* workspace,
                        size_t workspace_bytes, void* stream) {
    if (!scan_strides(D, &x_stride, &log_alpha_stride, &gate_stride, &d_h_stride)) return KDA_ERR_INVALID_ARG;
    kda::ScanArgs a{};
    a.x = x, a.log_alpha = log_alpha, a.gate = gate, a.d_h = d_h;
    a.ld_x = x_stride, a.ld_l = log_alpha_stride, a.ld_g = gate_stride, a.ld_dh = d_h_stride;
    a.init = init_state, a.cu = cu_seqlens, a.B = B, a.D = D, a.T = T;
    a.in_bf16 = in_dtype == KDA_BF16, a.out_bf16 = grad_dtype == KDA_BF16, a.normalize = normalize != 0;
    a.status = static_cast<uint32_t*>(workspace);
    a.chunk_states = const_cast<float*>(chunk_states);
    a.d_final = d_final_state, a.dx = dx, a.dl = dlog_alpha, a.dg = dgate, a.d_init = d_init_state;
    size_t need = 0;
    const bool own_states = !chunk_states && T > 0;  // (no tokens: no states)
    if (B > 0 && D > 0 && own_states) {
        const kda_status st = kda_scan_bwd_workspace_size(B, T, D, &need);
        if (st != KDA_OK) return st;
    }
    const kda_status st = scan_check(a, in_dtype, grad_dtype, &n_seqs, need, workspace, workspace_bytes);
    if (st != KDA_OK) return st;
    if (T > 0 && (!d_h || !dx || !dlog_alpha || (gate != nullptr) != (dgate != nullptr))) return KDA_ERR_INVALID_ARG;
    a.n_seqs = n_seqs;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (own_states)
        a.chunk_states = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + KDA_STATUS_BYTES);
    kda::prof_begin(kda::PROF_SCAN_BWD, s);
    const cudaError_t e = kda::launch_scan_bwd(a, own_states, s);
    kda::prof_end(kda::PROF_SCAN_BWD, s);
    return from_cuda(e);
}

kda_status kda_scan_decode_steps(float* state, const void* x, const void* log_alpha, const void* gate, void* h,
                                 const int32_t* slots, int n_slots, int n_steps, int Bd, int D, kda_dtype in_dtype,
                                 kda_dtype out_dtype, int normalize, float* step_states, void* stream) {
    if (n_steps < 0 || Bd < 0 || D <= 0 || n_slots < 0 || !dtype_ok(in_dtype) || !dtype_ok(out_dtype))
        return KDA_ERR_INVALID_ARG;
    if (Bd == 0 || n_steps == 0) return KDA_OK;
    const bool no_pages = slots && n_slots == 0;  // all rows are padding
    if ((!state && !no_pages) || !x || !log_alpha || !h || (!slots && n_slots < Bd)) return KDA_ERR_INVALID_ARG;
    if (Bd > 65535 || D > kda::SCAN_MAX_D) return KDA_ERR_UNSUPPORTED;  // grid y extent
    const void* ptrs[] = {state, x, log_alpha, gate, h, step_states};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_MISALIGNED;
    if (!aligned4(slots)) return KDA_ERR_MISALIGNED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    kda::prof_begin(kda::PROF_SCAN_DECODE, s);
    const cudaError_t e =
        kda::launch_scan_decode(state, x, log_alpha, gate, h, slots, n_slots, n_steps, Bd, D, in_dtype == KDA_BF16,
                                out_dtype == KDA_BF16, normalize != 0, step_states, s);
    kda::prof_end(kda::PROF_SCAN_DECODE, s);
    return from_cuda(e);
}

kda_status kda_gate_norm_bwd_workspace_size(int64_t rows, int dv, size_t* bytes) {
    if (rows < 0 || !bytes) return KDA_ERR_INVALID_ARG;
    if (dv != kSupportedD) return KDA_ERR_UNSUPPORTED;
    *bytes = (size_t)kda::gate_norm_bwd_blocks(rows) * dv * sizeof(float);
    return KDA_OK;
}

kda_status kda_gate_norm_bwd(const void* o, const void* gate, const void* d_y, const float* norm_weight, float eps,
                             void* d_o, void* d_gate, float* d_norm_weight, int64_t rows, int dv, kda_dtype in_dtype,
                             kda_dtype grad_dtype, void* workspace, size_t workspace_bytes, void* stream) {
    if (rows < 0 || !dtype_ok(in_dtype) || !dtype_ok(grad_dtype) || !(eps >= 0.f)) return KDA_ERR_INVALID_ARG;
    if (rows > 0 && (!o || !gate || !d_y || !d_o || !d_gate)) return KDA_ERR_INVALID_ARG;
    if (dv != kSupportedD) return KDA_ERR_UNSUPPORTED;
    const void* ptrs[] = {o, gate, d_y, norm_weight, d_o, d_gate, d_norm_weight, workspace};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_MISALIGNED;
    size_t need = 0;
    const kda_status st = kda_gate_norm_bwd_workspace_size(rows, dv, &need);
    if (st != KDA_OK) return st;
    if (d_norm_weight && need > 0 && (!workspace || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    kda::prof_begin(kda::PROF_GATE_NORM_BWD, s);
    const cudaError_t e = kda::launch_gate_norm_bwd(o, gate, d_y, norm_weight, eps, d_o, d_gate, d_norm_weight, rows,
                                                    in_dtype == KDA_BF16, grad_dtype == KDA_BF16,
                                                    static_cast<float*>(workspace), s);
    kda::prof_end(kda::PROF_GATE_NORM_BWD, s);
    return from_cuda(e);
}

kda_status kda_state_copy(void* dst, const void* src, int layers, int64_t page_bytes, int dst_pages, int src_pages,
                          int64_t dst_layer_bytes, int64_t src_layer_bytes, const int32_t* dst_slots,
                          const int32_t* src_slots, int n, void* stream) {
    if (layers < 0 || n < 0 || page_bytes <= 0 || page_bytes % 4 != 0 || dst_pages < 0 || src_pages < 0)
        return KDA_ERR_INVALID_ARG;
    if (n == 0 || layers == 0 || dst_pages == 0) return KDA_OK;
    if (!dst || !dst_slots || !src_slots || (!src && src_pages > 0)) return KDA_ERR_INVALID_ARG;
    if (layers > 65535 || n > 65535 || page_bytes > (int64_t(1) << 40)) return KDA_ERR_UNSUPPORTED;  // grid extents
    if (!aligned16(dst) || !aligned16(src) || !aligned4(dst_slots) || !aligned4(src_slots)) return KDA_ERR_MISALIGNED;
    const int64_t d_size = page_bytes * dst_pages, s_size = page_bytes * src_pages;
    if (layers == 1) dst_layer_bytes = d_size, src_layer_bytes = s_size;
    if (dst_layer_bytes < d_size || src_layer_bytes < s_size || dst_layer_bytes % 4 != 0 || src_layer_bytes % 4 != 0)
        return KDA_ERR_INVALID_ARG;
    if (src_pages > 0) {
        // one pool twice, or two that share no byte
        const uintptr_t d0 = (uintptr_t)dst, s0 = (uintptr_t)src;
        const uintptr_t d1 = d0 + (uintptr_t)(dst_layer_bytes * (layers - 1) + d_size);
        const uintptr_t s1 = s0 + (uintptr_t)(src_layer_bytes * (layers - 1) + s_size);
        const bool one = d0 == s0 && (layers == 1 || dst_layer_bytes == src_layer_bytes);
        if (!one && d0 < s1 && s0 < d1) return KDA_ERR_INVALID_ARG;
    }
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    kda::prof_begin(kda::PROF_PAGES, s);
    const cudaError_t e = kda::launch_state_copy(dst, src, layers, page_bytes, dst_pages, src_pages, dst_layer_bytes,
                                                 src_layer_bytes, dst_slots, src_slots, n, s);
    kda::prof_end(kda::PROF_PAGES, s);
    return from_cuda(e);
}

kda_status kda_state_alloc(uint8_t* live, int n_pages, int32_t* slots, int n, void* stream) {
    if (n < 0 || n_pages < 0) return KDA_ERR_INVALID_ARG;
    if (n == 0) return KDA_OK;
    if ((!live && n_pages > 0) || !slots) return KDA_ERR_INVALID_ARG;
    if (!aligned4(slots)) return KDA_ERR_MISALIGNED;
    return from_cuda(kda::launch_state_alloc(live, n_pages, slots, n, reinterpret_cast<cudaStream_t>(stream)));
}

kda_status kda_state_free(uint8_t* live, int n_pages, const int32_t* slots, int n, void* stream) {
    if (n < 0 || n_pages < 0) return KDA_ERR_INVALID_ARG;
    if (n == 0 || n_pages == 0) return KDA_OK;
    if (!live || !slots) return KDA_ERR_INVALID_ARG;
    if (!aligned4(slots)) return KDA_ERR_MISALIGNED;
    return from_cuda(kda::launch_state_free(live, n_pages, slots, n, reinterpret_cast<cudaStream_t>(stream)));
}

kda_status kda_state_compact(uint8_t* live, int n_pages, int32_t* dst_slots, int32_t* src_slots, int32_t* new_slots,
                             int32_t* n_live, void* stream) {
    if (n_pages < 0 || !n_live) return KDA_ERR_INVALID_ARG;
    if (n_pages > 0 && (!live || !dst_slots || !src_slots || !new_slots)) return KDA_ERR_INVALID_ARG;
    const void* ptrs[] = {dst_slots, src_slots, new_slots, n_live};
    for (const void* p : ptrs)
        if (!aligned4(p)) return KDA_ERR_MISALIGNED;
    return from_cuda(kda::launch_state_compact(live, n_pages, dst_slots, src_slots, new_slots, n_live,
                                               reinterpret_cast<cudaStream_t>(stream)));
}

kda_status kda_profile_enable(int on) {
    kda::g_prof_on = on != 0;
    return KDA_OK;
}

kda_status kda_profile_read(kda_kernel_time* out, int max_entries, int* n_entries) {
    static const char* names[kda::PROF_KINDS] = {"intra",      "chain",    "gate_norm",
                                                 "decode",     "check_cu", "kcp_compose",
                                                 "chain_bwd",  "intra_bwd", "scan",
                                                 "scan_bwd",   "scan_decode", "gate_norm_bwd",
                                                 "pages"};
    int launches[kda::PROF_KINDS] = {0};
    double ms[kda::PROF_KINDS] = {0};
    kda_status st = KDA_OK;
    for (auto& r : kda::g_prof_done) {
        float t = 0.f;
        if (cudaEventSynchronize(r.stop) != cudaSuccess || cudaEventElapsedTime(&t, r.start, r.stop) != cudaSuccess)
            st = KDA_ERR_CUDA;
        launches[r.kind] += 1;
        ms[r.kind] += t;
        kda::g_event_pool.push_back(r.start);
        kda::g_event_pool.push_back(r.stop);
    }
    kda::g_prof_done.clear();
    int n = 0;
    for (int k = 0; k < kda::PROF_KINDS; ++k) {
        if (launches[k] == 0) continue;
        if (out && n < max_entries) {
            memset(out[n].name, 0, sizeof(out[n].name));
            strncpy(out[n].name, names[k], sizeof(out[n].name) - 1);
            out[n].launches = launches[k];
            out[n].ms = ms[k];
        }
        ++n;
    }
    if (n_entries) *n_entries = n;
    return st;
}

kda_status kda_test_drop_tile_load(unsigned long long wait_limit_ns) {
    if (wait_limit_ns != 0 && (wait_limit_ns < 1000ull || wait_limit_ns > 1000000000ull)) return KDA_ERR_INVALID_ARG;
    kda::set_test_tile_drop(wait_limit_ns);
    return KDA_OK;
}

kda_status kda_query_status(void* workspace, void* stream) {
    if (!workspace) return KDA_ERR_INVALID_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    uint32_t word = 0;
    if (cudaMemcpyAsync(&word, workspace, sizeof(word), cudaMemcpyDeviceToHost, st) != cudaSuccess)
        return KDA_ERR_CUDA;
    if (cudaStreamSynchronize(st) != cudaSuccess) return KDA_ERR_CUDA;
    if (cudaMemsetAsync(workspace, 0, sizeof(word), st) != cudaSuccess) return KDA_ERR_CUDA;
    if (cudaStreamSynchronize(st) != cudaSuccess) return KDA_ERR_CUDA;
    if (word & 1u) return KDA_ERR_TIMEOUT;
    if (word & 2u) return KDA_ERR_DEVICE_ARG;
    return KDA_OK;
}

}  // extern "C"
