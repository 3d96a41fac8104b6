/*
 * kda.h -- C ABI of libkda, a B200 (sm_100a) library for the Kimi Delta
 * Attention (KDA) gated delta-rule recurrence.
 *
 * The operation (sources: the K3 article summaries on the xhh.club tag page,
 * items "KDA recurrence form", "chunkwise parallel algorithm" and "3:1
 * hybrid"; section 6 of the nlpx.cn K3 paper walkthrough).  Each head keeps a
 * dk x dv fp32 state S (row = key channel).  For every token t of a sequence:
 *
 *     l_t = max(log_alpha_t, -5)                     per key channel
 *     S_t = (I - beta_t k_t k_t^T) Diag(exp(l_t)) S_{t-1} + beta_t k_t v_t^T
 *     o_t = scale * S_t^T q_t
 *
 * optionally followed by the per-head RMSNorm and full-rank sigmoid gate
 *     y_t = o_t / sqrt(mean_j o_tj^2 + eps) * w * sigmoid(g_t).
 * Prefill runs the chunkwise form (64-token chunks: matrix products inside a
 * chunk, a recurrence between chunks); decode runs the recurrent form.
 *
 * Conventions for every entry point:
 *  - Pointers are DEVICE pointers owned by the caller, unless stated.  The
 *    library never allocates, frees or keeps them past the call.
 *  - Element layout is token-major, head-minor: [B, T, H, d] (contiguous).
 *    beta is [B, T, H].  States are fp32 [N, H, dk, dv], row = key channel.
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *    stream).  Every call is asynchronous on that stream and never
 *    synchronises, except kda_query_status.
 *  - Arguments are checked on the host before any launch; a rejected call
 *    launches nothing and returns a negative kda_status.  A failed launch
 *    returns KDA_ERR_CUDA (cudaGetLastError is cleared into the return code).
 *    Errors detected on the device (a bounded wait that expired, cu_seqlens
 *    that contradict T or max_seqlen) are recorded in a status word inside
 *    the workspace and read back with kda_query_status.
 *  - Supported shapes: dk = dv = 128 (the element-wise scan: any D).  Supported dtypes: inputs KDA_F32 or
 *    KDA_BF16 (all of q, k, v, log_alpha, beta, gate share in_dtype);
 *    outputs KDA_F32 or KDA_BF16.  Every pointer must be 16-byte aligned.
 *  - Outputs must not alias inputs, except where stated (in-place states).
 */
#ifndef KDA_H_
#define KDA_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define KDA_API __attribute__((visibility("default")))
#else
#define KDA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    KDA_OK = 0,
    KDA_ERR_INVALID_ARG = -1, /* null pointer, bad size, bad dtype */
    KDA_ERR_UNSUPPORTED = -2, /* shape outside what the kernels implement */
    KDA_ERR_MISALIGNED = -3,  /* a pointer is not 16-byte aligned */
    KDA_ERR_WORKSPACE = -4,   /* workspace missing or smaller than required */
    KDA_ERR_CUDA = -5,        /* a CUDA runtime call or launch failed */
    KDA_ERR_TIMEOUT = -6,     /* device: a bounded wait gave up */
    KDA_ERR_DEVICE_ARG = -7   /* device: cu_seqlens inconsistent with T / max_seqlen */
} kda_status;

typedef enum { KDA_F32 = 0, KDA_BF16 = 1 } kda_dtype;

/* Human-readable name of a kda_status value (static string, never NULL). */
KDA_API const char* kda_status_string(int status);

/* Library ABI version (major * 10000 + minor * 100 + patch). */
KDA_API int kda_version(void);

/*
 * kda_chunk_fwd_workspace_size -- bytes of device workspace kda_chunk_fwd needs.
 *
 *   T, H, dk, dv   as for kda_chunk_fwd (T = tokens per sequence for fixed
 *                  length, total packed tokens for varlen)
 *   n_seqs         number of sequences N (B for fixed length)
 *   max_seqlen     longest sequence (T for fixed length)
 *   bytes_min      out: the smallest workspace accepted (one 64-token chunk
 *                  of every sequence per pass)
 *   bytes_full     out: the workspace that lets one pass cover every chunk
 *                  of every sequence (fewest launches)
 * Any size in [bytes_min, inf) works; larger workspaces need fewer passes.
 */
KDA_API kda_status kda_chunk_fwd_workspace_size(int64_t T, int H, int dk, int dv, int n_seqs,
                                        int64_t max_seqlen, size_t* bytes_min,
                                        size_t* bytes_full);

/*
 * kda_chunk_fwd -- chunkwise prefill / training forward of the KDA recurrence.
 * Defined by the "chunkwise parallel algorithm" item of the K3 article
 * summaries (xhh.club tag page): 64-token chunks, state recurrence between
 * chunks, matrix products inside a chunk, per-step log-decay bounded below by
 * -5, 16-token diagonal tiles in BF16 matrix multiplies.
 *
 *   q, k, log_alpha  [B, T, H, dk]   in_dtype
 *   v                [B, T, H, dv]   in_dtype
 *   beta             [B, T, H]       in_dtype, values in [0, 1]
 *   init_state       [N, H, dk, dv]  fp32, NULL = zero state
 *   o                [B, T, H, dv]   out_dtype: o, or y when gate != NULL
 *   final_state      [N, H, dk, dv]  fp32, NULL = not returned.  May alias
 *                                    init_state (updated in place).
 *   B, T             batch and tokens per sequence; for varlen B = 1 and T
 *                    = total packed tokens
 *   H, dk, dv        heads and head dims (dk = dv = 128)
 *   cu_seqlens       device int32 [n_seqs + 1] (cu[0] = 0, non-decreasing,
 *                    cu[n_seqs] = T), or NULL for B fixed-length sequences
 *   n_seqs           number of sequences when cu_seqlens != NULL (else B)
 *   max_seqlen       host upper bound on any sequence length (T when
 *                    cu_seqlens == NULL); lengths above it are a device error
 *   scale            output scale (1.0 for the plain recurrence)
 *   gate             [B, T, H, dv] in_dtype, or NULL: when given, the per-head
 *                    RMSNorm (over dv) and sigmoid gate are applied and y is
 *                    written to o
 *   norm_weight      [dv] fp32 RMSNorm weight shared by heads, NULL = ones
 *   eps              RMSNorm epsilon
 *   workspace        device buffer of workspace_bytes >=
 *                    kda_chunk_fwd_workspace_size(...).bytes_min, 256-byte
 *                    aligned.  Holds the per-chunk intermediates and the
 *                    device status word; its contents on entry are ignored.
 *   stream           cudaStream_t as void*
 * Zero-length sequences are allowed (final state = initial state).
 */
KDA_API kda_status kda_chunk_fwd(const void* q, const void* k, const void* v, const void* log_alpha,
                         const void* beta, const float* init_state, void* o,
                         float* final_state, int B, int64_t T, int H, int dk, int dv,
                         const int32_t* cu_seqlens, int n_seqs, int64_t max_seqlen,
                         kda_dtype in_dtype, kda_dtype out_dtype, float scale,
                         const void* gate, const float* norm_weight, float eps,
                         void* workspace, size_t workspace_bytes, void* stream);

/*
 * kda_chunk_fwd_ckpt -- kda_chunk_fwd that also emits state checkpoints for a
 * prefix cache (the "training and inference systems" item of the K3 article
 * summaries: states cached at 512-token boundaries).  Arguments as
 * kda_chunk_fwd, plus:
 *
 *   checkpoints  NULL (then identical to kda_chunk_fwd), or fp32
 *                [n_seqs, n_ckpt, H, dk, dv] with n_ckpt = max_seqlen /
 *                ckpt_tokens (fixed length: T / ckpt_tokens), 16-byte aligned.
 *                Checkpoint j of sequence n is the state after that sequence's
 *                first (j + 1) * ckpt_tokens tokens (initial state included);
 *                checkpoints beyond a sequence's length are not written.
 *   ckpt_tokens  checkpoint spacing in tokens, a positive multiple of 64
 *                (the chunk length); KDA_ERR_INVALID_ARG otherwise.
 */
KDA_API kda_status kda_chunk_fwd_ckpt(const void* q, const void* k, const void* v, const void* log_alpha,
                              const void* beta, const float* init_state, void* o,
                              float* final_state, int B, int64_t T, int H, int dk, int dv,
                              const int32_t* cu_seqlens, int n_seqs, int64_t max_seqlen,
                              kda_dtype in_dtype, kda_dtype out_dtype, float scale,
                              const void* gate, const float* norm_weight, float eps,
                              float* checkpoints, int64_t ckpt_tokens,
                              void* workspace, size_t workspace_bytes, void* stream);

/*
 * kda_chunk_fwd_segmented -- kda_chunk_fwd with every sequence cut into
 * `segments` segments of whole chunks that are walked in parallel: the
 * segment-parallel (associative scan) form of the prefill ("training and
 * inference systems" item of the K3 article summaries: context parallelism as a
 * prefix scan of segment transitions; the nlpx.cn walkthrough, §6: KCP).
 * Pass 1 computes, per (sequence, segment, head), the segment's affine state
 * map S -> M S + B; pass 2 walks each segment from the initial state folded
 * through the maps of the segments before it.  Useful when n_seqs * H is small
 * next to the GPU (the plain walk has 4 * n_seqs * H independent chains).
 * Arguments as kda_chunk_fwd plus `segments` (>= 1; 1 is kda_chunk_fwd); the
 * workspace must hold kda_chunk_fwd_segmented_workspace_size bytes (every chunk
 * at once plus the segment maps).  Results equal kda_chunk_fwd's up to bf16
 * rounding of the segment maps.
 */
KDA_API kda_status kda_chunk_fwd_segmented(const void* q, const void* k, const void* v,
                                   const void* log_alpha, const void* beta,
                                   const float* init_state, void* o, float* final_state,
                                   int B, int64_t T, int H, int dk, int dv,
                                   const int32_t* cu_seqlens, int n_seqs, int64_t max_seqlen,
                                   kda_dtype in_dtype, kda_dtype out_dtype, float scale,
                                   const void* gate, const float* norm_weight, float eps,
                                   int segments, void* workspace, size_t workspace_bytes,
                                   void* stream);

/*
 * kda_chunk_fwd_segmented_workspace_size -- workspace bytes for
 * kda_chunk_fwd_segmented (arguments as kda_chunk_fwd_workspace_size plus
 * segments).
 */
KDA_API kda_status kda_chunk_fwd_segmented_workspace_size(int64_t T, int H, int dk, int dv, int n_seqs,
                                                  int64_t max_seqlen, int segments,
                                                  size_t* bytes);

/*
 * Context parallelism across devices (KCP: the nlpx.cn K3 walkthrough, §6; the
 * "training and inference systems" item of the K3 article summaries: context
 * parallelism as a prefix scan of segment transitions).  Every sequence is cut
 * into consecutive token segments, segment r on device r.  Segment r's effect
 * on the state is affine, S -> M_r S + B_r, so each device
 *   1. kda_kcp_transition: runs the chunk-local work over its segment, keeps it
 *      in the workspace and writes (M_r, B_r) in fp32;
 *   2. exchanges the maps (an all-gather in device order; the library does no
 *      communication);
 *   3. kda_kcp_compose: folds the maps of devices 0 .. r-1 over the sequences'
 *      initial state into its own initial state;
 *   4. kda_kcp_finish: walks its kept chunks from that state, with outputs.
 * Device r's outputs then equal those of kda_chunk_fwd over the whole
 * sequence (up to fp32 rounding of the composition and bf16 rounding of the
 * map's state image inside the walk), and the last device's final state is
 * the sequence's.  Arguments as kda_chunk_fwd, for this device's segment.
 *
 * kda_kcp_workspace_size -- bytes of the workspace that steps 1 and 4 share
 * (every chunk's slot at once: kda_chunk_fwd_workspace_size's bytes_full).
 */
KDA_API kda_status kda_kcp_workspace_size(int64_t T, int H, int dk, int dv, int n_seqs, int64_t max_seqlen,
                                          size_t* bytes);

/*
 * kda_kcp_transition -- step 1.  Inputs as kda_chunk_fwd (q and scale are used:
 * the kept chunk work includes the output terms).
 *
 *   transition  [2, N, H, dk, dk] fp32, device, caller-owned: [0] = M (dk x dk),
 *               [1] = B (dk x dv) with S_out = M S_in + B per (sequence, head);
 *               an empty segment gives M = I, B = 0
 *   workspace   >= kda_kcp_workspace_size bytes, 256-byte aligned; it holds the
 *               chunk slots until kda_kcp_finish has run on the same stream
 *
 * Errors as kda_chunk_fwd (device-side ones land in the workspace status word).
 */
KDA_API kda_status kda_kcp_transition(const void* q, const void* k, const void* v, const void* log_alpha,
                                      const void* beta, int B, int64_t T, int H, int dk, int dv,
                                      const int32_t* cu_seqlens, int n_seqs, int64_t max_seqlen,
                                      kda_dtype in_dtype, float scale, float* transition, void* workspace,
                                      size_t workspace_bytes, void* stream);

/*
 * kda_kcp_compose -- step 3:  S = init_state (zero when NULL), then for
 * j = 0 .. n_prev-1:  S = M_j S + B_j;  state_in = S.
 *
 *   transitions [R, 2, N, H, dk, dk] fp32, device: the gathered maps in device
 *               order (R >= n_prev; may be NULL when n_prev == 0)
 *   init_state  [N, H, dk, dv] fp32 or NULL; state_in [N, H, dk, dv] fp32 (output)
 *
 * KDA_ERR_INVALID_ARG for n_prev < 0 or missing buffers, KDA_ERR_MISALIGNED
 * for pointers not 16-byte aligned.
 */
KDA_API kda_status kda_kcp_compose(const float* transitions, int n_prev, const float* init_state,
                                   float* state_in, int n_seqs, int H, int dk, int dv, void* stream);

/*
 * kda_kcp_finish -- step 4: the walk of kda_chunk_fwd over the chunk slots
 * that kda_kcp_transition left in `workspace` (same B, T, H, cu_seqlens,
 * n_seqs, max_seqlen and workspace), starting from state_in (NULL = zero).
 * o, final_state, gate, norm_weight, eps and the dtypes as kda_chunk_fwd;
 * in_dtype is the gate's dtype.  The workspace status word carries step 1's
 * device-side errors too.
 */
KDA_API kda_status kda_kcp_finish(const float* state_in, void* o, float* final_state, int B, int64_t T, int H,
                                  int dk, int dv, const int32_t* cu_seqlens, int n_seqs, int64_t max_seqlen,
                                  kda_dtype in_dtype, kda_dtype out_dtype, const void* gate,
                                  const float* norm_weight, float eps, void* workspace, size_t workspace_bytes,
                                  void* stream);

/*
 * kda_chunk_bwd -- gradients of kda_chunk_fwd (without the gate) with respect
 * to q, k, v, log_alpha, beta and the initial state, given dL/do and dL/d(final
 * state).  The pages give no backward pass; this is the exact gradient of the
 * forward definition, computed chunkwise: the forward walk is recomputed (chunk
 * slots and chunk-boundary states kept in the workspace), a reverse walk forms
 * dL/d(state) at every chunk end, and a chunk-local kernel forms the token
 * gradients.  The clamp l = max(log_alpha, -5) passes the gradient where
 * log_alpha >= -5 and blocks it below.
 *
 *   q, k, v, log_alpha, beta, init_state, B, T, H, cu_seqlens, n_seqs,
 *   max_seqlen, in_dtype, scale   as kda_chunk_fwd
 *   d_o           [B, T, H, dv] in_dtype: dL/do (device)
 *   d_final_state [N, H, dk, dv] fp32 or NULL (zero)
 *   dq, dk, dlog_alpha [B, T, H, dk] fp32; dv [B, T, H, dv] fp32; dbeta [B, T, H]
 *                 fp32 (outputs, caller-owned device memory)
 *   d_init_state  [N, H, dk, dv] fp32 or NULL: dL/d(initial state)
 *   workspace     >= kda_chunk_bwd_workspace_size bytes, 256-byte aligned
 *
 * Errors as kda_chunk_fwd; device-side ones land in the workspace status word.
 */
KDA_API kda_status kda_chunk_bwd(const void* q, const void* k, const void* v, const void* log_alpha,
                                 const void* beta, const float* init_state, const void* d_o,
                                 const float* d_final_state, float* dq, float* dk, float* dv,
                                 float* dlog_alpha, float* dbeta, float* d_init_state, int B, int64_t T,
                                 int H, int dk_dim, int dv_dim, const int32_t* cu_seqlens, int n_seqs,
                                 int64_t max_seqlen, kda_dtype in_dtype, float scale, void* workspace,
                                 size_t workspace_bytes, void* stream);

/*
 * kda_chunk_bwd_workspace_size -- workspace bytes of kda_chunk_bwd: the
 * forward's whole-sequence workspace plus, per chunk and head, the state at the
 * chunk's start and the state gradient at its end, each kept as a bf16 128 x 128
 * operand image (arguments as kda_chunk_fwd_workspace_size).
 */
KDA_API kda_status kda_chunk_bwd_workspace_size(int64_t T, int H, int dk, int dv, int n_seqs, int64_t max_seqlen,
                                                size_t* bytes);

/*
 * kda_decode_step -- one recurrent step for Bd independent sequences
 * ("decode uses the recurrent form", chunkwise-algorithm item of the K3
 * article summaries).  The state is read once and written once, in place.
 *
 *   state        [Bd, H, dk, dv] fp32, updated in place
 *   q, k, log_alpha [Bd, H, dk]; v [Bd, H, dv]; beta [Bd, H]   in_dtype
 *   o            [Bd, H, dv] out_dtype (y when gate != NULL)
 *   gate         [Bd, H, dv] in_dtype or NULL; norm_weight [dv] fp32 or NULL
 */
KDA_API kda_status kda_decode_step(float* state, const void* q, const void* k, const void* v,
                           const void* log_alpha, const void* beta, void* o, int Bd, int H,
                           int dk, int dv, kda_dtype in_dtype, kda_dtype out_dtype,
                           float scale, const void* gate, const float* norm_weight,
                           float eps, void* stream);

/*
 * kda_decode_steps -- n_steps consecutive recurrent steps for Bd independent
 * sequences in one call: verification of n_steps draft tokens in speculative
 * decoding, or plain decode of several tokens.  (Decode runs the recurrent
 * form, chunkwise-algorithm item of the K3 article summaries; speculative
 * decoding with state rollback is the "training and inference systems" item.)
 * Each (sequence, head) state is read once and written once for all steps.
 *
 *   state        [Bd, H, dk, dv] fp32: the state before step 0; on return the
 *                state after the last step
 *   q, k, log_alpha, gate [n_steps, Bd, H, dk]; v [n_steps, Bd, H, dv];
 *   beta [n_steps, Bd, H]          in_dtype (step-major)
 *   o            [n_steps, Bd, H, dv] out_dtype (y when gate != NULL)
 *   step_states  NULL, or [n_steps, Bd, H, dk, dv] fp32: the state after each
 *                step (step_states[n_steps - 1] equals the final state).  To
 *                roll back to "accepted the first a tokens" (1 <= a <= n_steps)
 *                copy step_states[a - 1] into the state; keep a copy of the
 *                incoming state to reject every draft token.
 * Errors as kda_decode_step; n_steps == 0 or Bd == 0 does nothing.
 */
KDA_API kda_status kda_decode_steps(float* state, const void* q, const void* k, const void* v,
                            const void* log_alpha, const void* beta, void* o, int n_steps,
                            int Bd, int H, int dk, int dv, kda_dtype in_dtype,
                            kda_dtype out_dtype, float scale, const void* gate,
                            const float* norm_weight, float eps, float* step_states,
                            void* stream);

/*
 * kda_gate_norm -- per-head RMSNorm over dv followed by the full-rank sigmoid
 * output gate ("KDA recurrence form" and "3:1 hybrid" items of the K3
 * article summaries):  y = o / sqrt(mean(o^2) + eps) * w * sigmoid(g).
 *
 *   o      [rows, dv] in_dtype (rows = B*T*H)
 *   gate   [rows, dv] in_dtype
 *   norm_weight [dv] fp32 or NULL (ones)
 *   y      [rows, dv] out_dtype; may alias o exactly (in place)
 */
KDA_API kda_status kda_gate_norm(const void* o, const void* gate, const float* norm_weight, float eps,
                         void* y, int64_t rows, int dv, kda_dtype in_dtype,
                         kda_dtype out_dtype, void* stream);

/*
 * Element-wise gated scan: the diagonal relative of the recurrence above, one
 * state value per channel (no counterpart on the pages).  For every token t of
 * a sequence and every channel, in fp32:
 *
 *     l_t = min(log_alpha_t, 0)            a_t = exp(l_t)
 *     s_t = sigmoid(gate_t), or 1          w_t = sqrt(1 - a_t^2), or 1
 *     u_t = w_t * s_t * x_t                h_t = a_t * h_{t-1} + u_t
 *
 * log_alpha has no floor here; -inf restarts a channel (a_t = 0).  gate is
 * optional; `normalize` selects w_t = sqrt(1 - a_t^2), which keeps the state's
 * variance at the input's.  States are fp32 [N, D].
 *
 * Token tensors are [B, T, D] (or packed [1, T, D] with cu_seqlens), channels
 * contiguous.  The inputs x, log_alpha, gate and d_h take a token stride in
 * elements (0 = D), so that columns of one wider tensor can be passed as they
 * lie; they need element alignment only (16-byte aligned pointers with strides
 * of whole 16 bytes load fastest).  Here and below, cu_seqlens and vectors of
 * slots need 4-byte alignment, all other pointers 16-byte alignment.  D is any
 * size from 1 to 2^28; B * T is at most 2^31 - 65536 tokens.  What is not finite
 * stays in its channel and sequence, where an infinite state may turn to NaN.
 * A gate below -44 may count as -44 or as -infinity (s is below 1e-19 there).
 *
 *   cu_seqlens   device int32 [n_seqs + 1], cu[0] = 0, non-decreasing,
 *                cu[n_seqs] <= T, or NULL for B sequences of T tokens.  Rows of
 *                tokens at and behind cu[n_seqs] are neither read nor written.
 *   workspace    NULL, or a buffer whose first word receives the device status
 *                (kda_query_status): KDA_ERR_DEVICE_ARG when cu_seqlens breaks
 *                these rules.  Such a call reads and writes nothing out of
 *                range; its outputs are undefined.  KDA_ERR_TIMEOUT when a
 *                bounded wait gave up.  At least KDA_STATUS_BYTES when given.
 *                Without a workspace both leave no trace: the call returns
 *                KDA_OK, its outputs are undefined and nothing says so.
 */
#define KDA_STATUS_BYTES 256u

/* Tokens between two rows of chunk_states below. */
#define KDA_SCAN_CHUNK 8

/*
 * kda_scan_fwd -- h for every token and the last state of every sequence.
 *
 *   x, log_alpha  [B, T, D] in_dtype; gate the same or NULL
 *   init_state    [N, D] fp32, NULL = zero
 *   h             [B, T, D] out_dtype, contiguous
 *   final_state   [N, D] fp32 or NULL; may alias init_state exactly.  The
 *                 initial state's for a sequence without tokens.
 *   chunk_states  NULL, or fp32 [ceil(B * T / KDA_SCAN_CHUNK), D]: row c is the
 *                 state before token c * KDA_SCAN_CHUNK of the B * T tokens in
 *                 a row (unspecified where a sequence starts there, and at or
 *                 behind cu[n_seqs]), which kda_scan_bwd takes
 */
KDA_API kda_status kda_scan_fwd(const void* x, const void* log_alpha, const void* gate, const float* init_state,
                                void* h, float* final_state, float* chunk_states, int B, int64_t T, int D,
                                int64_t x_stride, int64_t log_alpha_stride, int64_t gate_stride,
                                const int32_t* cu_seqlens, int n_seqs, kda_dtype in_dtype, kda_dtype out_dtype,
                                int normalize, void* workspace, size_t workspace_bytes, void* stream);

/*
 * kda_scan_bwd -- gradients of kda_scan_fwd with respect to x, log_alpha, gate
 * and the initial state, given dL/dh and dL/d(final state):
 *
 *     G_t = dh_t + a_{t+1} G_{t+1}   (the last token: + d_final_state)
 *     dx = G w s;   dgate = G u (1 - s);   d_init = a_first G_first
 *     dlog_alpha = G (a h_{t-1} - a^2 s x / w)     (second term: normalize)
 *
 * The gradient of min(log_alpha, 0) passes where log_alpha <= 0.  The second
 * term has no limit at log_alpha = 0 (w = 0) and is left out there.
 *
 *   x .. init_state, B .. n_seqs, normalize   as kda_scan_fwd
 *   d_h            [B, T, D] in_dtype; d_final_state [N, D] fp32 or NULL (zero)
 *   chunk_states   as kda_scan_fwd wrote them for the same arguments, or NULL:
 *                  then they are computed first, into the workspace
 *   dx, dlog_alpha, dgate  [B, T, D] grad_dtype, contiguous (dgate NULL without
 *                  a gate); d_init_state [N, D] fp32 or NULL (for a sequence
 *                  without tokens d_final_state)
 *   workspace      kda_scan_bwd_workspace_size bytes when chunk_states is NULL and
 *                  T > 0; otherwise as for kda_scan_fwd
 */
KDA_API kda_status kda_scan_bwd(const void* x, const void* log_alpha, const void* gate, const float* init_state,
                                const void* d_h, const float* d_final_state, const float* chunk_states, void* dx,
                                void* dlog_alpha, void* dgate, float* d_init_state, int B, int64_t T, int D,
                                int64_t x_stride, int64_t log_alpha_stride, int64_t gate_stride, int64_t d_h_stride,
                                const int32_t* cu_seqlens, int n_seqs, kda_dtype in_dtype, kda_dtype grad_dtype,
                                int normalize, void* workspace, size_t workspace_bytes, void* stream);

/* kda_scan_bwd_workspace_size -- the status word and the chunk states of B * T tokens. */
KDA_API kda_status kda_scan_bwd_workspace_size(int B, int64_t T, int D, size_t* bytes);

/*
 * kda_scan_decode_steps -- n_steps consecutive tokens of Bd sequences, states in
 * place (one token per sequence: n_steps = 1).
 *
 *   state        [n_slots, D] fp32: row slots[b] is sequence b's state; slots
 *                NULL: row b (n_slots >= Bd).  Updated in place.  May be NULL
 *                with slots and n_slots = 0 (every row is padding).
 *   x, log_alpha, gate  [n_steps, Bd, D] in_dtype contiguous, gate or NULL
 *   h            [n_steps, Bd, D] out_dtype
 *   slots        device int32 [Bd] or NULL.  A negative slot, or one of n_slots
 *                and above, marks a row of padding: its outputs are zeros, its
 *                inputs are not used and no state changes.  Of rows that name
 *                the same slot the first is stepped, the others are padding.
 *   step_states  NULL or [n_steps, Bd, D] fp32: the state after every step
 *                (rows of padding: zeros)
 */
KDA_API kda_status kda_scan_decode_steps(float* state, const void* x, const void* log_alpha, const void* gate, void* h,
                                         const int32_t* slots, int n_slots, int n_steps, int Bd, int D,
                                         kda_dtype in_dtype, kda_dtype out_dtype, int normalize, float* step_states,
                                         void* stream);

/*
 * kda_decode_steps_paged -- kda_decode_steps for sequences whose states lie in a
 * pool: state is [n_slots, H, dk, dv] and row b of the batch uses page slots[b]
 * (slots as for kda_scan_decode_steps; padding: zeros in o and step_states).
 * A gated call normalises o in fp32, whatever n_steps is.
 */
KDA_API kda_status kda_decode_steps_paged(float* state, const int32_t* slots, int n_slots, const void* q,
                                          const void* k, const void* v, const void* log_alpha, const void* beta,
                                          void* o, int n_steps, int Bd, int H, int dk, int dv, kda_dtype in_dtype,
                                          kda_dtype out_dtype, float scale, const void* gate,
                                          const float* norm_weight, float eps, float* step_states, void* stream);

/*
 * kda_gate_norm_bwd -- gradients of kda_gate_norm.  With r = (mean(o^2) + eps)^-1/2,
 * n = o r, s = sigmoid(g):
 *
 *     d_gate = dy n w s (1 - s);   d_norm_weight = sum over rows of dy n s
 *     d_o = r (dn - n mean(dn n)),   dn = dy w s
 *
 *   o, gate, d_y  [rows, dv] in_dtype; norm_weight [dv] fp32 or NULL (ones)
 *   d_o, d_gate   [rows, dv] grad_dtype; d_norm_weight [dv] fp32, or NULL (not
 *                 wanted).  Sums run in a fixed order: equal inputs give equal bits.
 *   workspace     kda_gate_norm_bwd_workspace_size bytes, 16-byte aligned; may
 *                 be NULL when d_norm_weight is
 */
KDA_API kda_status kda_gate_norm_bwd(const void* o, const void* gate, const void* d_y, const float* norm_weight,
                                     float eps, void* d_o, void* d_gate, float* d_norm_weight, int64_t rows, int dv,
                                     kda_dtype in_dtype, kda_dtype grad_dtype, void* workspace,
                                     size_t workspace_bytes, void* stream);
KDA_API kda_status kda_gate_norm_bwd_workspace_size(int64_t rows, int dv, size_t* bytes);

/*
 * Pages of recurrent states.  A pool is [layers, n_pages, page_bytes]: one page
 * per sequence slot and layer, the same slot in every layer (prefix cache at
 * fixed token boundaries, state rollback: the "training and inference systems"
 * item of the K3 article summaries).
 *
 * kda_state_copy -- for i = 0 .. n-1, in list order, in every layer:
 *     dst page dst_slots[i] = src page src_slots[i],   or zeros when src_slots[i] < 0
 * with the result of carrying the list out one by one: a page written by one
 * entry and read by a later one is read as written, and of entries that write
 * one page the last stands.  An entry whose destination is negative or not
 * below dst_pages, or whose source is not below src_pages, does nothing.
 *
 *   dst, src      device pools, or the same pool twice; otherwise their address ranges,
 *                 from the first layer's first page to the last layer's last, may not
 *                 overlap, not even where they share no page (page ranges of one wider
 *                 pool with several layers: KDA_ERR_INVALID_ARG).  src may be NULL when
 *                 every entry clears.
 *   page_bytes    a positive multiple of 4; pools 16-byte aligned
 *   *_layer_bytes distance between layers (layers == 1: ignored); a multiple of
 *                 4, at least n_pages * page_bytes
 *   dst_slots, src_slots   device int32 [n], n at most 65535 (as is layers; KDA_ERR_UNSUPPORTED
 *                 above): pass a longer list in pieces, one call behind the other
 *
 * Entries that read or write a page which another entry writes are carried out one after the
 * other, all others side by side.
 */
KDA_API kda_status kda_state_copy(void* dst, const void* src, int layers, int64_t page_bytes, int dst_pages,
                                  int src_pages, int64_t dst_layer_bytes, int64_t src_layer_bytes,
                                  const int32_t* dst_slots, const int32_t* src_slots, int n, void* stream);

/*
 * kda_state_alloc -- takes the n lowest free slots: live[p] (one byte per page,
 * 0 = free) becomes 1 and slots[0 .. n) lists them in rising order, -1 where none
 * was left.   kda_state_free -- live[slots[i]] = 0; slots out of range are ignored.
 */
KDA_API kda_status kda_state_alloc(uint8_t* live, int n_pages, int32_t* slots, int n, void* stream);
KDA_API kda_status kda_state_free(uint8_t* live, int n_pages, const int32_t* slots, int n, void* stream);

/*
 * kda_state_compact -- plans the moves that bring all live pages to the front of
 * the pool: with m live pages, the k-th free slot below m receives the k-th live
 * page at or above m.  The moves themselves are kda_state_copy(dst_slots,
 * src_slots, n = n_pages) for each pool that shares the slots, of which the first n_pages / 2
 * entries hold every move.
 *
 *   live       [n_pages] bytes, on return 1 for the first m and 0 behind them
 *   dst_slots, src_slots  int32 [n_pages]: the moves, then -1
 *   new_slots  int32 [n_pages]: where each old slot's page lies now, -1 if it was free
 *   n_live     int32 [1]: m
 */
KDA_API kda_status kda_state_compact(uint8_t* live, int n_pages, int32_t* dst_slots, int32_t* src_slots,
                                     int32_t* new_slots, int32_t* n_live, void* stream);

/*
 * kda_query_status -- synchronises `stream`, reads the device status word of
 * a kda_chunk_fwd workspace, clears it and returns it (KDA_OK when no device
 * error was recorded).  This is the only call that blocks the host.
 */
KDA_API kda_status kda_query_status(void* workspace, void* stream);

/*
 * kda_test_drop_tile_load -- test hook for the device-side failure path (no
 * counterpart on the pages).  The next kda_chunk_fwd-family call with bf16
 * inputs in this process runs its chunk-local kernel with one change: CTA 0
 * does not issue one of the four tile loads of its first item, and its wait
 * for them gives up after wait_limit_ns (1e3 .. 1e9 ns) instead of the usual
 * second.  That CTA then stops; the call returns KDA_OK, its outputs are
 * undefined, and kda_query_status on its workspace returns KDA_ERR_TIMEOUT.
 * The process and the GPU context stay usable: the next call is normal.
 * wait_limit_ns = 0 cancels a pending drop.  Host-side only; not
 * thread-safe.  KDA_ERR_INVALID_ARG for any other limit outside the range.
 */
KDA_API kda_status kda_test_drop_tile_load(unsigned long long wait_limit_ns);

/*
 * kda_chunk_fwd_noalloc -- kda_chunk_fwd for callers that cannot allocate
 * device memory.  (No counterpart on the pages: it is a packaging of
 * kda_chunk_fwd, not part of the method.)
 *
 * Who needs it: hosts that hand a plugin its inputs and outputs but no way to
 * get device scratch -- e.g. a framework whose memory pool already owns all
 * free device memory, or a runtime that forbids cudaMalloc on its hot path
 * because cudaMalloc can synchronise the device.  Here the scratch is a
 * static array of KDA_NOALLOC_SCRATCH_BYTES inside libkda's own device
 * memory, so there is no workspace argument and the call allocates nothing.
 *
 * Arguments, layouts and results are exactly those of kda_chunk_fwd minus
 * (workspace, workspace_bytes).  The caller still owns every input and output.
 *  - Limit: the problem must fit the static scratch, i.e.
 *    kda_chunk_fwd_workspace_size(...).bytes_min <= KDA_NOALLOC_SCRATCH_BYTES
 *    (roughly n_seqs * H <= 400).  Larger problems
 *    return KDA_ERR_WORKSPACE before any CUDA call; larger scratch than the
 *    minimum only means fewer passes.
 *  - The array is reserved on each GPU that loads this part of the library and
 *    is held until the process exits.  The first call on a device looks up the
 *    array's device address (cudaGetSymbolAddress) with that device current;
 *    make that first call before any stream capture on that device.
 *  - Every call on a device shares the one array, which keeps the previous
 *    call's contents (the call clears the parts that must start at zero
 *    itself).  Calls that overlap on the GPU (different streams without
 *    ordering, or different host threads) race on it: order them.
 *  - Errors the kernels detect on the device (a bounded wait that gave up,
 *    cu_seqlens that contradict T or max_seqlen) are recorded in a status word
 *    at the start of the static array; read them with
 *    kda_chunk_fwd_noalloc_query_status (kda_query_status takes a workspace,
 *    and this entry point has none).  Each call clears the word first, so it
 *    describes the last call on the device.
 *  - The array's device address is cached per device; after a cudaDeviceReset
 *    the module is unloaded and the cached address is stale, so do not call
 *    this entry point again in that process after a reset.
 */
#define KDA_NOALLOC_SCRATCH_BYTES (64u * 1024u * 1024u)

KDA_API kda_status kda_chunk_fwd_noalloc(const void* q, const void* k, const void* v,
                                 const void* log_alpha, const void* beta,
                                 const float* init_state, void* o, float* final_state,
                                 int B, int64_t T, int H, int dk, int dv,
                                 const int32_t* cu_seqlens, int n_seqs, int64_t max_seqlen,
                                 kda_dtype in_dtype, kda_dtype out_dtype, float scale,
                                 const void* gate, const float* norm_weight, float eps,
                                 void* stream);

/*
 * kda_chunk_fwd_noalloc_query_status -- synchronises `stream` and returns the
 * device status word of the last kda_chunk_fwd_noalloc call on the current
 * device (then clears it): KDA_OK, KDA_ERR_TIMEOUT or KDA_ERR_DEVICE_ARG, as
 * kda_query_status does for a workspace.  Allocates nothing.  Returns
 * KDA_ERR_CUDA if the array's address cannot be looked up.
 */
KDA_API kda_status kda_chunk_fwd_noalloc_query_status(void* stream);

/*
 * Per-kernel device timing (a measurement aid, off by default).
 * kda_profile_enable(1) makes every later launch of this library bracket each
 * of its kernels with CUDA events on the launch stream.  kda_profile_read
 * synchronises on those events, writes one entry per kernel kind that ran
 * (name, number of launches, summed device milliseconds) into out[0 ..
 * max_entries), stores the count in *n_entries and resets the counters.
 * Host-side only; not thread-safe.
 */
typedef struct {
    char name[16];
    int launches;
    double ms;
} kda_kernel_time;

KDA_API kda_status kda_profile_enable(int on);
KDA_API kda_status kda_profile_read(kda_kernel_time* out, int max_entries, int* n_entries);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H_ */
