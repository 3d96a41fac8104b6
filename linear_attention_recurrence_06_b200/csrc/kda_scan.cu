// kda_scan.cu -- element-wise gated scan (include/kda.h, kda_scan_fwd), forward
// and single tokens.
#include <cudaTypedefs.h>

#include <type_traits>

#include "kda_row_slot.cuh"
#include "kda_scan.h"
#include "kda_scan_launch.h"

namespace kda {

bool make_scan_map(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t ld, int box_rows, bool bf16) {
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> encoder{nullptr};
    PFN_cuTensorMapEncodeTiled_v12000 enc = encoder.load(std::memory_order_relaxed);
    if (!enc) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return false;
        enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
        encoder.store(enc, std::memory_order_relaxed);
    }
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld * (bf16 ? 2 : 4)};
    const cuuint32_t box[2] = {SC_CH, (cuuint32_t)box_rows}, one[2] = {1, 1};
    return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void*>(base),
               dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
               CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

// The forward: kda_scan_tile.cuh says how the work is split.  A warp's first run keeps each token's
// state from zero and the product of the decays up to it; with the state before the warp's
// tokens known, the second is one fused product per value.  (Those products' rounding stays
// inside a token's output; what is carried on, final states too, goes by the sum of the log-decays.)
// 16 tokens per warp in bf16: two stages of two CTAs still fit an SM's shared memory, and the hand-overs, which
// cost as much for 8 tokens, are half as many; the 64 registers of a warp's states and decays are what
// limits it.  Gated bf16, 4 x 2048 x 4096: 54 us, 5.0 TB/s (without either factor 35 us, 5.7 TB/s; fp32 90 us, 6.0 TB/s; rows
// of 4094, without TMA, 134 us: copies of 4 bytes, and those kernels spill 140 to 152 bytes); one sequence of 8192: 70 us,
// 3.8 TB/s, of 32,768: 246 us, 4.4 TB/s (clusters of 4: an exchange per step, schedulers issue in 46 % of cycles);
// 110,842 tokens in 16 packed sequences: 685 us, 5.3 TB/s.  What bounds it: schedulers that share two CTAs issue in three of four cycles, and 256 such CTAs
// leave 40 of 148 SMs with one.
template <bool BF16, bool GATE>
struct ScanFwd {
    static constexpr int NT = BF16 ? 16 : 8;                                 // tokens of a warp
    static constexpr int N_IN = GATE ? 3 : 2;
    static constexpr int ROWS = NT * ScanGeo<BF16>::ROWB;                         // a warp's rows of one tensor
    static constexpr int STAGE = N_IN * ROWS;                                // [warps][2] stages
    static constexpr int OFF_AB = SC_WARPS * 2 * STAGE;                      // [2][warps][32] pieces up to a warp
    static constexpr int OFF_BASE = OFF_AB + 2 * SC_WARPS * 512;             // [2][32] what a tile starts from
    static constexpr int OFF_BAR = OFF_BASE + 2 * 256;                       // full[warps][2], given[warps][2], based[2]
    static constexpr int OFF_EX = OFF_BAR + (4 * SC_WARPS + 2) * 8;          // [4][cluster][32] the CTAs' pieces, sent[4][cluster]
    static constexpr int smem(int cluster) { return OFF_EX + 4 * cluster * (512 + 8); }
    static_assert(2 * (OFF_EX + 4 * 4 * 520 + 1024) <= 228 * 1024, "two CTAs per SM with clusters up to 4");
};

// TMA: rows that it can load, of even D.
template <bool BF16, bool GATE, bool NORM, bool TMA>
__global__ void __launch_bounds__(SC_THREADS, 2)
scan_fwd_kernel(const ScanArgs a, const __grid_constant__ ScanMaps maps, int cluster, int width) {
    using K = ScanFwd<BF16, GATE>;
    constexpr int NT = K::NT, TILE = SC_WARPS * NT;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_trigger();
    const int ch0 = blockIdx.x / cluster * SC_CH, ch = ch0 + 2 * lane, D = a.D;
    int rank = blockIdx.x % cluster;
    const ScanSpan sp = scan_span(a, blockIdx.y, gridDim.y, TILE, &cluster, &rank, lane);  // changes cluster and rank, too
    const int tile0 = sp.t0 / TILE, n_tiles = sp.t1 > sp.t0 ? (sp.t1 + TILE - 1) / TILE - tile0 : 0;
    const int n_steps = (n_tiles + cluster - 1) / cluster;
    uint64_t* const bars = reinterpret_cast<uint64_t*>(smem + K::OFF_BAR);
    uint64_t* const full = bars + 2 * warp;                    // this warp's loads
    uint64_t* const given = bars + 2 * SC_WARPS + 2 * warp;    // this warp's piece
    uint64_t* const based = bars + 4 * SC_WARPS;               // the state before the CTA's tile
    float2* const base = reinterpret_cast<float2*>(smem + K::OFF_BASE);
    float4* const ex = reinterpret_cast<float4*>(smem + K::OFF_EX);  // the cluster's pieces, [4][cluster][32]
    uint64_t* const sent = reinterpret_cast<uint64_t*>(smem + K::OFF_EX + 4 * cluster * 512);
    uint8_t* const stages = smem + warp * 2 * K::STAGE;
    const bool even = TMA || (D & 1) == 0;
    bool failed = false;

    if (TMA && n_steps > 0 && threadIdx.x >= 32 && threadIdx.x < 32 + K::N_IN) prefetch_tmap(&maps.m[threadIdx.x - 32]);
    if (threadIdx.x == 0) {
        for (int i = 0; i < 4 * SC_WARPS + 2; ++i) mbar_init(&bars[i], 1);
        for (int i = 0; i < 4 * cluster; ++i) mbar_init(&sent[i], 1);
        fence_mbar_init();
        if (cluster > 1)
            for (int i = 0; i < 4 * cluster; ++i) mbar_arrive_expect_tx(&sent[i], 512);
    }
    __syncthreads();
    int tw = (tile0 + rank) * TILE + warp * NT;
    const int by = cluster * TILE;
    auto load = [&](int s, int t) {  // step s, whose tokens begin at t
        uint8_t* const st = stages + (s & 1) * K::STAGE;
        if constexpr (TMA) {
            if (lane == 0 && s < n_steps) {
                uint64_t* const b = full + (s & 1);
                mbar_arrive_expect_tx(b, K::STAGE);
                tma_load_2d(st, &maps.m[0], ch0, t, b);
                tma_load_2d(st + K::ROWS, &maps.m[1], ch0, t, b);
                if (GATE) tma_load_2d(st + 2 * K::ROWS, &maps.m[2], ch0, t, b);
            }
        } else {
            if (s < n_steps) {
                load_rows<BF16, NT>(st, a.log_alpha, a.ld_l, t, sp.t0, sp.t1, ch0, D, width, lane);
                load_rows<BF16, NT>(st + K::ROWS, a.x, a.ld_x, t, sp.t0, sp.t1, ch0, D, width, lane);
                if (GATE) load_rows<BF16, NT>(st + 2 * K::ROWS, a.gate, a.ld_g, t, sp.t0, sp.t1, ch0, D, width, lane);
            }
            cp_commit();
        }
    };
    load(0, tw);
    load(1, tw + by);
    pdl_wait();  // the status word is written behind it
    if (cluster > 1) cluster_sync_all();  // every CTA's barriers are set up before another writes to them

    ScanSeen at;
    at.calm = 0;
    bool plain = false;
    float2 h0 = f2(0.f);     // where a sequence starts with this warp's first token: its initial state
    float2 carry = f2(0.f);  // the state before this CTA's tile
    for (int s = 0; s < n_steps; ++s, tw += by) {
        float4* const ab = reinterpret_cast<float4*>(smem + K::OFF_AB) + (s & 1) * (SC_WARPS * 32);
        if (s >= at.calm) {
            at = scan_see<NT>(a, sp, s, tw, by, reinterpret_cast<int*>(ab + warp * 32));
            // whole rows, and sequences meet at most before the first token and behind the last
            plain = at.own == (1u << NT) - 1u && !(at.starts & ~1u) && !(at.ends & ~(1u << (NT - 1)));
            if (at.starts & 1) {
                const int n = at.seq_start(0);
                h0 = a.init ? load2(a.init, n, D, ch) : f2(0.f);
            }
        }
        const uint32_t phase = (s >> 1) & 1;
        if constexpr (TMA) {
            failed = failed || !scan_wait<false>(full + (s & 1), phase, a.status);
        } else {
            cp_wait<1>();
            __syncwarp();
        }
        const uint8_t* const st = stages + (s & 1) * K::STAGE;

        // the warp's tokens from zero: states h, products of the decays A
        float2 hs[NT], as[NT], sum = f2(0.f);
        auto first_run = [&](auto edge) {
            constexpr bool EDGE = decltype(edge)::value;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                float2 d = depth_at<BF16>(st, i, lane), u = tile_at<BF16>(st + K::ROWS, i, lane);
                const float2 g = GATE ? tile_at<BF16>(st + 2 * K::ROWS, i, lane) : f2(0.f);
                const bool own = !EDGE || (at.own >> i & 1);
                if (!own) d = f2(0.f);
                const ScanDecay2 a2 = scan_decay2<!BF16>(d);
                if (GATE || NORM) u = __fmul2_rn(scan_weight2<GATE, NORM>(a2.m, g), u);
                if (!own) u = f2(0.f);
                // up to a sequence's last token, for its final state
                if (!EDGE || !(at.ends & ((1u << i) - 1u))) sum = __fadd2_rn(sum, d);
                if (i == 0) {
                    hs[0] = u;
                    as[0] = a2.a;
                } else {
                    if (!EDGE) {
                        hs[i] = __ffma2_rn(a2.a, hs[i - 1], u);
                    } else {  // the whole of a short sequence, perhaps, which the caller may go on with
                        float2 h = hs[i - 1];
                        if (at.starts >> i & 1) {
                            const int n = at.seq_start(i);
                            h = a.init ? load2(a.init, n, D, ch) : f2(0.f);
                        }
                        hs[i] = scan_step2(scan_p2(d, a2), h, u);
                    }
                    as[i] = __fmul2_rn(a2.a, as[i - 1]);
                }
            }
        };
        if (plain) first_run(std::false_type{});
        else first_run(std::true_type{});
        float4 piece = scan_piece(false, sum, hs[NT - 1]);
        if (at.starts) {  // nothing of what came before gets through
            const float2 b = at.starts == 1 ? scan_fold2(piece, h0) : hs[NT - 1];
            piece = make_float4(SC_CUT, SC_CUT, b.x, b.y);
        }
        __syncwarp();
        if (!failed) load(s + 2, tw + 2 * by);  // into the stage that this warp has just read

        // the pieces of the warps before it; its own joined to them goes on
        float4 before = make_float4(-0.f, -0.f, 0.f, 0.f);
        if (warp > 0) {
            failed = failed || !scan_wait<false>(given - 2 + (s & 1), phase, a.status);
            before = ab[(warp - 1) * 32 + lane];
            piece = scan_join2(before, piece);
        }
        if (warp < SC_WARPS - 1) {
            ab[warp * 32 + lane] = piece;
            __syncwarp();
            if (lane == 0) mbar_arrive(given + (s & 1));
        } else {
            // Four buffers: a CTA that sends for step s + 4 has seen all pieces of step s + 2, whose
            // warps are done with step s + 1, in which the pieces of step s are read last.  (The
            // warps' pieces and base have two: step s + 2 follows all pieces of step s + 1, whose warps
            // are done with step s.)
            const int slot = (s & 3) * cluster + rank;
            if (cluster > 1) {
                const uint32_t to = smem_u32(ex + slot * 32 + lane), on = smem_u32(sent + slot);
                for (int c = 0; c < cluster; ++c) st_async16(map_to_cta(to, c), piece, map_to_cta(on, c));
            } else {
                ex[slot * 32 + lane] = piece;
                __syncwarp();
                if (lane == 0) mbar_arrive(sent + slot);
            }
        }

        // the state before this CTA's tile: its own and the later CTAs' pieces of the last step,
        // the earlier ones' of this step; then the state before this warp's tokens
        if (warp == 0) {
            for (int k = 0; k < cluster; ++k) {
                const bool last = rank + k < cluster;
                const int c = last ? rank + k : rank + k - cluster, q = last ? s - 1 : s, slot = (q & 3) * cluster + c;
                if (q < 0) continue;
                const uint32_t ph = (q >> 2) & 1;
                if (cluster > 1) {
                    failed = failed || !scan_wait<true>(sent + slot, ph, a.status);
                    if (lane == 0) mbar_arrive_expect_tx(sent + slot, 512);  // for step q + 4
                } else {
                    failed = failed || !scan_wait<false>(sent + slot, ph, a.status);
                }
                const float4 v = ex[slot * 32 + lane];
                carry = scan_fold2(v, carry, scan_is_cut(v));
            }
            base[(s & 1) * 32 + lane] = carry;
            __syncwarp();
            if (lane == 0) mbar_arrive(based + (s & 1));
        } else {
            failed = failed || !scan_wait<false>(based + (s & 1), phase, a.status);
            carry = base[(s & 1) * 32 + lane];
        }
        float2 mine = warp > 0 ? scan_fold2(before, carry, scan_is_cut(before)) : carry;
        if (at.starts & 1) mine = h0;

        if (a.chunk_states) {
#pragma unroll
            for (int i = 0; i < NT; i += SCAN_CHUNK) {  // the state before token i
                const bool own = at.own >> i & 1, from_start = at.starts & ((1u << i) - 2u) & ((1u << i) - 1u);
                float2 h = mine;
                if (i > 0) h = from_start ? hs[i - 1] : __ffma2_rn(as[i - 1], mine, hs[i - 1]);
                if (own && even) {
                    if (ch < D)
                        *reinterpret_cast<float2*>(a.chunk_states + (size_t)((tw + i) / SCAN_CHUNK) * D + ch) = h;
                } else if (own) {
                    store2(a.chunk_states, false, (tw + i) / SCAN_CHUNK, D, ch, h);
                }
            }
        }
        // the same tokens from that state
        if (plain) {
            if (a.h && !even) {
#pragma unroll
                for (int i = 0; i < NT; ++i)
                    store2_odd(a.h, a.out_bf16, (size_t)(tw + i), D, ch, __ffma2_rn(as[i], mine, hs[i]));
            } else if (a.h && ch < D) {
                const uint32_t row = (uint32_t)D * (a.out_bf16 ? 2 : 4);
                uint8_t* const to = static_cast<uint8_t*>(a.h) + (size_t)tw * row + (size_t)ch * (a.out_bf16 ? 2 : 4);
                if (a.out_bf16) {
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        const float2 h = __ffma2_rn(as[i], mine, hs[i]);
                        *reinterpret_cast<uint32_t*>(to + (size_t)row * i) = pack_bf16x2(h.x, h.y);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < NT; ++i)
                        *reinterpret_cast<float2*>(to + (size_t)row * i) = __ffma2_rn(as[i], mine, hs[i]);
                }
            }
            if (at.ends && a.final_state) {
                const int n = at.seq_end(NT - 1);
                if (n >= 0) store2(a.final_state, false, n, D, ch, scan_fold2(scan_piece(false, sum, hs[NT - 1]), mine));
            }
        } else {
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const bool from_start = at.starts & ((2u << i) - 2u);
                const float2 h = from_start ? hs[i] : __ffma2_rn(as[i], mine, hs[i]);
                if (a.h && at.own >> i & 1) {
                    if (TMA) store2_even(a.h, a.out_bf16, (size_t)(tw + i), D, ch, h);
                    else store2(a.h, a.out_bf16, (size_t)(tw + i), D, ch, h);
                }
                if (a.final_state && at.ends >> i & 1) {
                    const int n = at.seq_end(i);
                    if (n >= 0)
                        store2(a.final_state, false, n, D, ch,
                               from_start ? hs[i] : scan_fold2(scan_piece(false, sum, hs[i]), mine));
                }
            }
        }
    }
    cp_wait<0>();
    if (failed && TMA && lane == 0) scan_drain(full);
    if (cluster > 1) {
        // The last step's pieces of this and the later CTAs have not been looked at: they have to
        // arrive before this CTA's memory goes, and no CTA leaves while another may write to it.
        if (warp == 0 && n_steps > 0 && !failed)
            for (int k = rank; k < cluster; ++k)
                scan_wait<true>(sent + ((n_steps - 1) & 3) * cluster + k, ((n_steps - 1) >> 2) & 1, a.status);
        cluster_sync_all();
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
    pdl_trigger();
    bool bad = cu && threadIdx.x == 0 && cu[0] != 0;
    if (cu)
        for (int i = threadIdx.x; i < n_seqs; i += blockDim.x) bad |= cu[i + 1] < cu[i] || cu[i + 1] > T;
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *status = bad ? 2u : 0u;
}

// Single tokens: V channels of one row per thread (4 where D allows 16-byte states), the state read
// and written once for all steps of a call.  HBM-bound for many rows, else latency: the row's
// slot, its state and the first tokens are on their way before the slot is checked against the
// rows before it, and every step's tokens are loaded a step ahead.  256 rows x 4096 through slots: 5.0 us
// (16.6 MB: 2.5 us at a copy's rate); 3 rows x 1000, five tokens: 3.0 us.
template <bool BF16, int V>
KDA_DEV void load_v(const void* base, size_t i, float* v) {
    if constexpr (V == 1) {
        v[0] = ld_in<BF16>(base, i);
    } else if constexpr (BF16) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + i));
        v[0] = __uint_as_float(w.x << 16), v[1] = __uint_as_float(w.x & 0xFFFF0000u);
        v[2] = __uint_as_float(w.y << 16), v[3] = __uint_as_float(w.y & 0xFFFF0000u);
    } else {
        const float4 w = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(base) + i));
        v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
    }
}
template <int V>
KDA_DEV void store_v(void* base, bool bf16, size_t i, const float* v) {
    if (bf16) {
        uint16_t* const p = static_cast<uint16_t*>(base) + i;
        if constexpr (V == 4) *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        else p[0] = f32_to_bf16(v[0]);
    } else {
        float* const p = static_cast<float*>(base) + i;
        if constexpr (V == 4) *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
        else p[0] = v[0];
    }
}

template <bool BF16, bool GATE, bool NORM, int V>
__global__ void __launch_bounds__(128)
scan_decode_kernel(float* state, const void* __restrict__ x, const void* __restrict__ log_alpha,
                   const void* __restrict__ gate, void* hout, const int32_t* __restrict__ slots, int n_slots,
                   int n_steps, int Bd, int D, bool out_bf16, float* step_states) {
    const int ch = (blockIdx.x * 128 + threadIdx.x) * V, b = blockIdx.y;
    const bool mine = ch < D;
    const int slot = slots ? slots[b] : b;
    const bool there = !slots || slot_in_range(slot, n_slots);
    const size_t row = (size_t)Bd * D, at = (size_t)b * D + ch;
    float h[V], xv[V], lv[V], gv[V];
#pragma unroll
    for (int k = 0; k < V; ++k) h[k] = xv[k] = lv[k] = gv[k] = 0.f;
    auto tokens = [&](int t) {
        const size_t i = t * row + at;
        load_v<BF16, V>(log_alpha, i, lv);
        load_v<BF16, V>(x, i, xv);
        if (GATE) load_v<BF16, V>(gate, i, gv);
    };
    float* const S = state + (size_t)(there ? slot : 0) * D + ch;
    if (there && mine) {
        if constexpr (V == 4) {
            const float4 w = *reinterpret_cast<const float4*>(S);
            h[0] = w.x, h[1] = w.y, h[2] = w.z, h[3] = w.w;
        } else {
            h[0] = S[0];
        }
        tokens(0);
    }
    const bool live = slots ? !slot_taken(slots, slot, b) && there : true;
    if (!mine) return;
    for (int t = 0; t < n_steps; ++t) {
        const size_t i = t * row + at;
        if (live) {
            float p[V], u[V];
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const ScanTerm r = scan_term<GATE, NORM>(xv[k], lv[k], gv[k]);
                p[k] = r.p, u[k] = r.u;
            }
            if (t + 1 < n_steps) tokens(t + 1);
#pragma unroll
            for (int k = 0; k < V; ++k) h[k] = scan_step(p[k], h[k], u[k]);
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k) h[k] = 0.f;
        }
        store_v<V>(hout, out_bf16, i, h);
        if (step_states) store_v<V>(step_states, false, i, h);
    }
    if (live) store_v<V>(state, false, (size_t)slot * D + ch, h);
}

}  // namespace

cudaError_t launch_scan_check(const ScanArgs& a, cudaStream_t stream) {
    scan_check_cu_kernel<<<1, 256, 0, stream>>>(a.cu, a.n_seqs, a.T, a.status);
    return cudaGetLastError();
}

cudaError_t launch_scan_fwd(const ScanArgs& a, cudaStream_t stream) {
    if (a.status) {
        const cudaError_t e = launch_scan_check(a, stream);
        if (e != cudaSuccess) return e;
    }
    const void* in[] = {a.log_alpha, a.x, a.gate};
    const int64_t ld[] = {a.ld_l, a.ld_x, a.ld_g};
    ScanMaps maps;
    int width = 0;
    cudaError_t e = scan_maps(a, in, ld, a.gate ? 3 : 2, a.in_bf16 ? ScanFwd<true, true>::NT : ScanFwd<false, true>::NT, &maps, &width);
    if (e != cudaSuccess) return e;
#define KDA_SCAN_FWD(BF, TMA)                                                                                      \
    e = scan_launch<scan_fwd_kernel<BF, G, W, TMA>>(ScanFwd<BF, G>::smem, SC_WARPS * ScanFwd<BF, G>::NT, a, maps, width, \
                                                    a.status != nullptr, stream)
    KDA_SCAN_GN(a.gate != nullptr, a.normalize, {
        if (a.in_bf16) { if (width == 16) KDA_SCAN_FWD(true, true); else KDA_SCAN_FWD(true, false); }
        else           { if (width == 16) KDA_SCAN_FWD(false, true); else KDA_SCAN_FWD(false, false); }
    });
#undef KDA_SCAN_FWD
    return e;
}

cudaError_t launch_scan_decode(float* state, const void* x, const void* log_alpha, const void* gate, void* h,
                               const int32_t* slots, int n_slots, int n_steps, int Bd, int D, bool in_bf16,
                               bool out_bf16, bool normalize, float* step_states, cudaStream_t stream) {
    const bool four = D % 4 == 0;  // the tensors are 16-byte aligned
    const dim3 grid((D + (four ? 511 : 127)) / (four ? 512 : 128), Bd);
#define KDA_SCAN_DEC(BF, V)                                                                                       \
    scan_decode_kernel<BF, G, W, V><<<grid, 128, 0, stream>>>(state, x, log_alpha, gate, h, slots, n_slots, n_steps, \
                                                              Bd, D, out_bf16, step_states)
    KDA_SCAN_GN(gate != nullptr, normalize, {
        if (in_bf16) { if (four) KDA_SCAN_DEC(true, 4); else KDA_SCAN_DEC(true, 1); }
        else         { if (four) KDA_SCAN_DEC(false, 4); else KDA_SCAN_DEC(false, 1); }
    });
#undef KDA_SCAN_DEC
    return cudaGetLastError();
}

}  // namespace kda
