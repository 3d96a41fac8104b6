// kda_scan.cu -- element-wise gated scan (include/kda.h, kda_scan_fwd), forward
// and single tokens.
#include <type_traits>

#include "kda_row_slot.cuh"
#include "kda_scan.h"
#include "kda_scan_launch.h"

namespace kda {

namespace {

// The forward: kda_scan_tile.cuh says how the work is split.  Two tiles of a CTA are in
// flight while it computes on a third's registers; a warp loads and reads only its own
// rows, so that one barrier per tile remains, between the warps' pieces and their fold.
template <bool BF16, bool GATE, bool NORM>
struct ScanFwd {
    static constexpr int NT = BF16 ? 16 : 8;
    using Geo = ScanGeo<BF16, NT>;
    static constexpr int N_IN = GATE ? 3 : 2;
    static constexpr int STAGE = N_IN * Geo::TENS;
    static constexpr int OFF_AB = 2 * STAGE;                              // [2][warps][32] float4
    static constexpr int OFF_EX = OFF_AB + 2 * SC_WARPS * 32 * 16;        // [2][cluster][32] float4
    static constexpr int OFF_TAB = OFF_EX + 2 * SC_MAX_CLUSTER * 32 * 16; // [warps][2][NT] int
    static constexpr int SMEM = OFF_TAB + SC_WARPS * 2 * NT * 4;
    static_assert(2 * (SMEM + 1024) <= 228 * 1024, "two CTAs per SM");
};

template <bool BF16, bool GATE, bool NORM>
__global__ void __launch_bounds__(SC_THREADS, 2) scan_fwd_kernel(const ScanArgs a, int cluster, int width) {
    using K = ScanFwd<BF16, GATE, NORM>;
    using Geo = typename K::Geo;
    constexpr int NT = K::NT, TILE = Geo::TILE;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = blockIdx.x % cluster, ch0 = blockIdx.x / cluster * SC_CH, ch = ch0 + 2 * lane, D = a.D;
    const ScanSpan sp = scan_span(a, blockIdx.y, gridDim.y, lane);
    const int64_t tile0 = sp.t0 / TILE, n_tiles = sp.t1 > sp.t0 ? (sp.t1 + TILE - 1) / TILE - tile0 : 0;
    const int64_t n_steps = (n_tiles + cluster - 1) / cluster;
    float4* const s_ab = reinterpret_cast<float4*>(smem + K::OFF_AB);
    float4* const s_ex = reinterpret_cast<float4*>(smem + K::OFF_EX);
    int* const tab = reinterpret_cast<int*>(smem + K::OFF_TAB) + warp * 2 * NT;
    int ptr = sp.n0;
    const bool even = (D & 1) == 0;

    auto first_token = [&](int64_t s) { return (tile0 + s * cluster + rank) * TILE + warp * NT; };
    auto load = [&](int64_t s) {
        if (s < n_steps) {
            uint8_t* st = smem + (s & 1) * K::STAGE;
            const int64_t tw = first_token(s);
            load_rows<BF16, NT>(st, a.log_alpha, a.ld_l, tw, sp.t0, sp.t1, ch0, D, width, warp, lane);
            load_rows<BF16, NT>(st + Geo::TENS, a.x, a.ld_x, tw, sp.t0, sp.t1, ch0, D, width, warp, lane);
            if (GATE)
                load_rows<BF16, NT>(st + 2 * Geo::TENS, a.gate, a.ld_g, tw, sp.t0, sp.t1, ch0, D, width, warp, lane);
        }
        cp_commit();
    };
    load(0);
    load(1);
    if (cluster > 1) {  // every CTA of the cluster runs before another writes into its shared memory
        cluster_arrive();
        cluster_wait();
    }

    float2 carry = f2(0.f);  // the state before the cluster's tiles of this step
    for (int64_t s = 0; s < n_steps; ++s) {
        const int64_t tw = first_token(s);
        const ScanBounds<NT> bd = scan_bounds<NT>(a, sp, tw, &ptr, tab, lane);
        cp_wait<1>();
        __syncwarp();
        const uint8_t* st = smem + (s & 1) * K::STAGE;

        // the warp's piece, from zero
        float2 e[NT], u[NT], sum = f2(0.f), h = f2(0.f);
        uint32_t lo[NT];
        auto piece = [&](auto has_starts) {
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const float2 la = tile_at<BF16>(st, warp * NT + i, lane);
                const float2 x = tile_at<BF16>(st + Geo::TENS, warp * NT + i, lane);
                const float2 g = GATE ? tile_at<BF16>(st + 2 * Geo::TENS, warp * NT + i, lane) : f2(0.f);
                const float2 l = f2(scan_clamp(la.x), scan_clamp(la.y));
                const ScanDecay2 d = scan_decay2(l);
                float2 sg;
                u[i] = GATE || NORM ? __fmul2_rn(scan_weight2<GATE, NORM>(d.em, g, &sg), x) : x;
                e[i] = d.e;
                lo[i] = pack_bf16x2(d.lo.x, d.lo.y);
                sum = __fadd2_rn(sum, l);
                if (decltype(has_starts)::value && (bd.starts >> i & 1)) {  // the first token's state takes u's place
                    const float2 h0 = a.init ? load2(a.init, (size_t)bd.seq_start(i), D, ch) : f2(0.f);
                    u[i] = h = scan_step2(d.e, d.lo, h0, u[i]);
                } else {
                    h = scan_step2(d.e, d.lo, h, u[i]);
                }
            }
        };
        if (bd.starts) piece(std::true_type{});
        else piece(std::false_type{});
        __syncwarp();
        load(s + 2);  // into the stage that this warp has just read
        float4* const ab = s_ab + (s & 1) * (SC_WARPS * 32);
        const bool cut = bd.starts != 0;
        ab[warp * 32 + lane] = make_float4(cut ? SCAN_CUT : scan_decay(sum.x), cut ? SCAN_CUT : scan_decay(sum.y), h.x, h.y);
        __syncthreads();

        // the state before this warp's tokens, and the carry of the next step
        float2 mine = carry;
        if (cluster > 1) {
            float4* const ex = s_ex + (s & 1) * (SC_MAX_CLUSTER * 32);
            if (warp == 0) {
                float4 all = ab[lane];
#pragma unroll
                for (int w = 1; w < SC_WARPS; ++w) all = scan_join(all, ab[w * 32 + lane]);
                const uint32_t at = smem_u32(ex + rank * 32 + lane);
                for (int c = 0; c < cluster; ++c) st_cluster(map_to_cta(at, c), all);
            }
            cluster_arrive();
            cluster_wait();
            for (int c = 0; c < cluster; ++c) {
                if (c == rank) mine = carry;
                carry = scan_fold2(ex[c * 32 + lane], carry);
            }
            for (int w = 0; w < warp; ++w) mine = scan_fold2(ab[w * 32 + lane], mine);
        } else {
#pragma unroll
            for (int w = 0; w < SC_WARPS; ++w) {
                if (w == warp) mine = carry;
                carry = scan_fold2(ab[w * 32 + lane], carry);
            }
        }

        if (a.chunk_states && tw % SCAN_CHUNK == 0 && tw >= sp.t0 && tw < sp.t1) {
            const size_t i = (size_t)(tw / SCAN_CHUNK) * D + ch;
            if (ch < D) a.chunk_states[i] = mine.x;
            if (ch + 1 < D) a.chunk_states[i + 1] = mine.y;
        }
        if (!a.h && !(a.final_state && bd.ends)) continue;
        // the same tokens from that state
        if (a.h && even && !(bd.starts | bd.ends) && tw >= sp.t0 && tw + NT <= sp.t1) {
            uint8_t* to = static_cast<uint8_t*>(a.h) + ((size_t)tw * D + ch) * (a.out_bf16 ? 2 : 4);
            const size_t row = (size_t)D * (a.out_bf16 ? 2 : 4);
            if (a.out_bf16) {
#pragma unroll
                for (int i = 0; i < NT; ++i, to += row) {
                    mine = scan_step2(e[i], unpack2(lo[i]), mine, u[i]);
                    if (ch < D) *reinterpret_cast<uint32_t*>(to) = pack_bf16x2(mine.x, mine.y);
                }
            } else {
#pragma unroll
                for (int i = 0; i < NT; ++i, to += row) {
                    mine = scan_step2(e[i], unpack2(lo[i]), mine, u[i]);
                    if (ch < D) *reinterpret_cast<float2*>(to) = mine;
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                mine = bd.starts >> i & 1 ? u[i] : scan_step2(e[i], unpack2(lo[i]), mine, u[i]);
                if (a.h && tw + i >= sp.t0 && tw + i < sp.t1) store2(a.h, a.out_bf16, (size_t)(tw + i), D, ch, mine);
                if (a.final_state && bd.ends >> i & 1) {
                    const int64_t n = bd.seq_end(i);
                    if (n >= 0) store2(a.final_state, false, (size_t)n, D, ch, mine);
                }
            }
        }
    }
    cp_wait<0>();
    if (cluster > 1) {  // no CTA leaves while another may write to it
        cluster_arrive();
        cluster_wait();
    }
    // sequences without tokens
    if (a.final_state && rank == 0) {
        for (int n = sp.n0 + warp; n < sp.n1; n += SC_WARPS) {
            int64_t first, end;
            scan_range(a.cu, n, a.T, &first, &end);
            if (first == end)
                store2(a.final_state, false, n, D, ch, a.init ? load2(a.init, n, D, ch) : f2(0.f));
        }
    }
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
    const void* in[] = {a.x, a.log_alpha, a.gate};
    const int64_t ld[] = {a.ld_x, a.ld_l, a.ld_g};
    const int width = scan_width(in, ld, a.gate ? 3 : 2, a.in_bf16);
    cudaError_t e = cudaSuccess;
    KDA_SCAN_GN(a.gate != nullptr, a.normalize, {
        if (a.in_bf16)
            e = scan_launch<scan_fwd_kernel<true, G, W>>(ScanFwd<true, G, W>::SMEM, ScanFwd<true, G, W>::Geo::TILE, a,
                                                         width, stream);
        else
            e = scan_launch<scan_fwd_kernel<false, G, W>>(ScanFwd<false, G, W>::SMEM, ScanFwd<false, G, W>::Geo::TILE, a,
                                                          width, stream);
    });
    return e;
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
