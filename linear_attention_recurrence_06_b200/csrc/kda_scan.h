// kda_scan.h -- launch arguments of the element-wise gated scan (internal to libkda).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace kda {

constexpr int SCAN_CHUNK = 8;   // tokens between two rows of chunk_states
constexpr int64_t SCAN_MAX_TOKENS = (int64_t(1) << 31) - 65536;  // B * T: tokens are counted in 32 bits
constexpr int SCAN_MAX_D = 1 << 28;

struct ScanArgs {
    const void *x, *log_alpha, *gate;
    int64_t ld_x, ld_l, ld_g;  // token strides in elements
    const float* init;
    const int32_t* cu;
    int B, n_seqs, D;
    int64_t T;  // tokens per sequence, or packed tokens
    bool in_bf16, out_bf16, normalize;
    uint32_t* status;  // or null
    // forward
    void* h;
    float* final_state;
    float* chunk_states;  // written by the forward, read by the backward
    // backward (out_bf16: the gradients' type)
    const void* d_h;
    int64_t ld_dh;
    const float* d_final;
    void *dx, *dl, *dg;
    float* d_init;
};

struct ScanMaps {
    CUtensorMap m[4];    // log_alpha, x, then gate (forward) or d_h, gate (backward)
    CUtensorMap states;  // backward: chunk_states
};

cudaError_t launch_scan_fwd(const ScanArgs& a, cudaStream_t stream);
cudaError_t launch_scan_bwd(const ScanArgs& a, bool own_states, cudaStream_t stream);  // own_states: computes chunk_states first
// sets the status word: what contradicts in cu
cudaError_t launch_scan_check(const ScanArgs& a, cudaStream_t stream);
cudaError_t launch_scan_decode(float* state, const void* x, const void* log_alpha, const void* gate, void* h,
                               const int32_t* slots, int n_slots, int n_steps, int Bd, int D, bool in_bf16,
                               bool out_bf16, bool normalize, float* step_states, cudaStream_t stream);

}  // namespace kda
