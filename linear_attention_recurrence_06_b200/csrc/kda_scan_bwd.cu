// kda_scan_bwd.cu -- gradients of the element-wise gated scan (include/kda.h,
// kda_scan_bwd): G_t = dh_t + a_{t+1} G_{t+1} walks back over the tokens, c_t = a_t G_t goes on to the
// token before, and each gradient is G times a factor of its token:
//     dx = G (w s),   dgate = G (u (1 - s)),   dlog_alpha = G (a h_{t-1} - a^2 u / (1 - a^2))
// (a^2 s x / w = a^2 u / w^2).  Split as the forward (kda_scan_tile.cuh), with time reversed: warp 0 has a
// tile's last tokens, CTA 0 of a cluster the last tile.  A warp first runs its 8 tokens forwards
// from the state before them, which the forward keeps for every 8 tokens (half a byte per value;
// without it the warps' states would have to be handed on as well, before they could begin to
// walk back), for the factors; then back from zero.  14.5 bytes per value in bf16.  8 tokens per warp: the three
// factors, the gradient from zero and the products of the decays of 8 tokens already take the 128 registers.
// Gated bf16, 4 x 2048 x 4096: 94 us, 5.2 TB/s (without either factor 60 us; fp32 157 us, 6.1 TB/s; rows of 4094, without
// TMA, 160 us, gated ones spill 44 to 56 bytes); one sequence of 8192: 127 us, 3.8 TB/s, of 32,768: 476 us, 4.1 TB/s; 110,842
// tokens in 16 packed sequences: 1.30 ms, 5.1 TB/s.  The kept states came by plain loads at first: 114 us for the first case.
// Sequences that meet inside a tile cost most: 4,417 tokens in 23 sequences of 0 to 401, x 1000 fp32, take 47 us, 4,416 in 23 of
// 192 28 us (loads of initial states and of their gradients in the middle of the walk, one CTA per SM to hide them).
// Bound by issue slots where two CTAs share an SM, as the forward.
#include <float.h>

#include <type_traits>

#include "kda_scan_launch.h"

namespace kda {

namespace {

template <bool BF16, bool GATE>
struct ScanBwd {
    static constexpr int NT = SCAN_CHUNK;                                    // tokens of a warp
    static constexpr int N_IN = GATE ? 4 : 3;
    static constexpr int ROWS = NT * ScanGeo<BF16>::ROWB;                    // a warp's rows of one tensor
    static constexpr int STAGE = N_IN * ROWS + SC_CH * 4;                    // [warps][2] stages: and the state before them
    static constexpr int OFF_AB = SC_WARPS * 2 * STAGE;                      // as in the forward
    static constexpr int OFF_BASE = OFF_AB + 2 * SC_WARPS * 512;             // [2][32] what a tile starts from
    static constexpr int OFF_BAR = OFF_BASE + 2 * 256;                       // full[warps][2], given[warps][2], based[2]
    static constexpr int OFF_EX = OFF_BAR + (4 * SC_WARPS + 2) * 8;          // [4][cluster][32] the CTAs' pieces, sent[4][cluster]
    static constexpr int smem(int cluster) { return OFF_EX + 4 * cluster * (512 + 8); }
};

// TMA: rows that it can load, of even D.
template <bool BF16, bool GATE, bool NORM, bool TMA>
__global__ void __launch_bounds__(SC_THREADS, 2)
scan_bwd_kernel(const ScanArgs a, const __grid_constant__ ScanMaps maps, int cluster, int width) {
    using K = ScanBwd<BF16, GATE>;
    constexpr int NT = K::NT, TILE = SC_WARPS * NT;
    constexpr uint32_t ALL_BUT_LAST = (1u << (NT - 1)) - 1u;  // of a warp's tokens
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ch0 = blockIdx.x / cluster * SC_CH, ch = ch0 + 2 * lane, D = a.D;
    int rank = blockIdx.x % cluster;
    const ScanSpan sp = scan_span(a, blockIdx.y, gridDim.y, TILE, &cluster, &rank, lane);  // changes cluster and rank, too
    const int tile0 = sp.t0 / TILE, n_tiles = sp.t1 > sp.t0 ? (sp.t1 + TILE - 1) / TILE - tile0 : 0;
    const int n_steps = (n_tiles + cluster - 1) / cluster;
    uint64_t* const bars = reinterpret_cast<uint64_t*>(smem + K::OFF_BAR);
    uint64_t* const full = bars + 2 * warp;                    // this warp's loads
    uint64_t* const given = bars + 2 * SC_WARPS + 2 * warp;    // this warp's piece
    uint64_t* const based = bars + 4 * SC_WARPS;               // the gradient from behind the CTA's tile
    float2* const base = reinterpret_cast<float2*>(smem + K::OFF_BASE);
    float4* const ex = reinterpret_cast<float4*>(smem + K::OFF_EX);  // the cluster's pieces, [4][cluster][32]
    uint64_t* const sent = reinterpret_cast<uint64_t*>(smem + K::OFF_EX + 4 * cluster * 512);
    uint8_t* const stages = smem + warp * 2 * K::STAGE;
    const bool even = TMA || (D & 1) == 0;
    bool failed = false;

    if (TMA && n_steps > 0 && threadIdx.x >= 32 && threadIdx.x <= 32 + K::N_IN)
        prefetch_tmap(threadIdx.x < 32 + K::N_IN ? &maps.m[threadIdx.x - 32] : &maps.states);
    if (threadIdx.x == 0) {
        for (int i = 0; i < 4 * SC_WARPS + 2; ++i) mbar_init(&bars[i], 1);
        for (int i = 0; i < 4 * cluster; ++i) mbar_init(&sent[i], 1);
        fence_mbar_init();
        if (cluster > 1)
            for (int i = 0; i < 4 * cluster; ++i) mbar_arrive_expect_tx(&sent[i], 512);
    }
    __syncthreads();
    // tiles from the last one; those before the split's first (of the last step) have no tokens
    int tw = (tile0 + n_tiles - 1 - rank) * TILE + (SC_WARPS - 1 - warp) * NT;
    const int by = -cluster * TILE;
    auto load = [&](int s, int t) {  // step s, whose tokens begin at t
        uint8_t* const st = stages + (s & 1) * K::STAGE;
        if constexpr (TMA) {
            if (lane == 0 && s < n_steps) {
                const int y = t < 0 ? 0 : t;  // no tokens: any rows do
                uint64_t* const b = full + (s & 1);
                mbar_arrive_expect_tx(b, K::STAGE);
#pragma unroll
                for (int i = 0; i < K::N_IN; ++i) tma_load_2d(st + i * K::ROWS, &maps.m[i], ch0, y, b);
                if (s == 0) pdl_wait();  // the kernel that writes the states
                tma_load_2d(st + K::N_IN * K::ROWS, &maps.states, ch0, y / SCAN_CHUNK, b);
            }
        } else {
            if (s < n_steps) {
                load_rows<BF16, NT>(st, a.log_alpha, a.ld_l, t, sp.t0, sp.t1, ch0, D, width, lane);
                load_rows<BF16, NT>(st + K::ROWS, a.x, a.ld_x, t, sp.t0, sp.t1, ch0, D, width, lane);
                load_rows<BF16, NT>(st + 2 * K::ROWS, a.d_h, a.ld_dh, t, sp.t0, sp.t1, ch0, D, width, lane);
                if (GATE) load_rows<BF16, NT>(st + 3 * K::ROWS, a.gate, a.ld_g, t, sp.t0, sp.t1, ch0, D, width, lane);
                const int c = t < sp.t0 || t >= sp.t1 ? -1 : t / SCAN_CHUNK;
                load_rows<false, 1>(st + K::N_IN * K::ROWS, a.chunk_states, D, c, 0, INT32_MAX, ch0, D, 4, lane);
            }
            cp_commit();
        }
    };
    if (!TMA) pdl_wait();
    load(0, tw);
    load(1, tw + by);
    pdl_wait();
    if (cluster > 1) cluster_sync_all();  // every CTA's barriers are set up before another writes to them

    ScanSeen at;
    at.calm = 0;
    float2 carry = f2(0.f);  // a G of the token behind this CTA's tile
    for (int s = 0; s < n_steps; ++s, tw += by) {
        float4* const ab = reinterpret_cast<float4*>(smem + K::OFF_AB) + (s & 1) * (SC_WARPS * 32);
        if (s >= at.calm) at = scan_see<NT>(a, sp, s, tw, by, reinterpret_cast<int*>(ab + warp * 32));
        const uint32_t phase = (s >> 1) & 1;
        // whole rows, and sequences meet at most before the first token and behind the last
        const bool plain = at.own == (1u << NT) - 1u && !(at.starts & ~1u) && !(at.ends & ~(1u << (NT - 1)));
        float2 c_end = f2(0.f);
        const bool ends_here = at.ends >> (NT - 1) & 1;
        if (ends_here) {
            const int n = at.seq_end(NT - 1);
            if (a.d_final && n >= 0) c_end = load2(a.d_final, n, D, ch);
        }
        if constexpr (TMA) {
            failed = failed || !scan_wait<false>(full + (s & 1), phase, a.status);
        } else {
            cp_wait<1>();
            __syncwarp();
        }
        const uint8_t* const st = stages + (s & 1) * K::STAGE;
        float2 h = tile_at<false>(st + K::N_IN * K::ROWS, 0, lane);
        if (at.starts & 1) {
            const int n = at.seq_start(0);
            h = a.init ? load2(a.init, n, D, ch) : f2(0.f);
        }

        // forwards: the factors of each token; then back from zero: G, and the products of the decays
        // behind each token
        float2 kx[NT], kl[NT], kg[NT], gs[NT], as[NT], sum = f2(0.f), c = f2(0.f);
        auto runs = [&](auto edge) {
            constexpr bool EDGE = decltype(edge)::value;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const bool own = !EDGE || (at.own >> i & 1);
                const float2 la = tile_at<BF16>(st, i, lane);
                float2 x = tile_at<BF16>(st + K::ROWS, i, lane), d = scan_depth2(la);
                if (!own) d = x = f2(0.f);
                const ScanDecay2 a2 = scan_decay2<!BF16>(d);
                const float2 A = a2.a;
                float2 sg = f2(1.f), sn = f2(0.f), w = f2(1.f), r = f2(0.f);  // s, 1 - s
                if (GATE) {
                    const float2 g = tile_at<BF16>(st + 3 * K::ROWS, i, lane), y = __fmul2_rn(g, f2(-LOG2E));
                    const float2 e = f2(ex2_ftz(y.x), ex2_ftz(y.y)), q = __fadd2_rn(e, f2(1.f));
                    sg = f2(rcp_ftz(q.x), rcp_ftz(q.y));
                    if (!own) sg = f2(0.f);
                    // e^-gate s keeps its digits where s is next to 1 (s = 0: times 0)
                    sn = __fmul2_rn(f2(fminf(e.x, FLT_MAX), fminf(e.y, FLT_MAX)), sg);
                }
                if (NORM) {
                    const float2 n = __fmul2_rn(a2.m, __ffma2_rn(a2.m, f2(-1.f), f2(2.f)));
                    const float2 n1 = __fadd2_rn(n, f2(SCAN_TINY));
                    r = f2(rsqrt_ftz(n1.x), rsqrt_ftz(n1.y));
                    w = __fmul2_rn(n, r);
                }
                kx[i] = GATE && NORM ? __fmul2_rn(sg, w) : (GATE ? sg : w);
                const float2 u = GATE || NORM ? __fmul2_rn(kx[i], x) : x;
                if (GATE) kg[i] = __fmul2_rn(u, sn);
                if (EDGE && i > 0 && (at.starts >> i & 1)) {
                    const int n = at.seq_start(i);
                    h = a.init ? load2(a.init, n, D, ch) : f2(0.f);
                }
                const float2 ah = __fmul2_rn(A, h);
                kl[i] = ah;
                if (NORM) kl[i] = __ffma2_rn(__fmul2_rn(__fmul2_rn(A, f2(-1.f)), A), __fmul2_rn(u, __fmul2_rn(r, r)), ah);
                if (la.x > 0.f) kl[i].x = 0.f;  // the clamp passes no gradient there
                if (la.y > 0.f) kl[i].y = 0.f;
                h = __fadd2_rn(ah, u);
                as[i] = A;
                sum = __fadd2_rn(sum, d);
            }
            float2 P = f2(1.f);
#pragma unroll
            for (int i = NT - 1; i >= 0; --i) {
                float2 dh = tile_at<BF16>(st + 2 * K::ROWS, i, lane);
                if (EDGE && !(at.own >> i & 1)) dh = f2(0.f);
                if (EDGE && i < NT - 1 && (at.ends >> i & 1)) {
                    const int n = at.seq_end(i);
                    c = a.d_final && n >= 0 ? load2(a.d_final, n, D, ch) : f2(0.f);
                }
                gs[i] = __fadd2_rn(dh, c);
                c = __fmul2_rn(as[i], gs[i]);
                const float2 A = as[i];
                as[i] = P;
                P = __fmul2_rn(P, A);
            }
        };
        if (plain) {
            runs(std::false_type{});
        } else {
            runs(std::true_type{});
            // What goes beyond this call, or may, is stepped without the roundings of decays, which would add up where the
            // caller hands d_init on to an earlier call: what the tokens up to the first end hand on to an earlier warp,
            // and the d_init of sequences that are all here.
            for (uint32_t m = at.ends & ALL_BUT_LAST; m; m &= m - 1) {
                const int e = __ffs(m) - 1, n = at.seq_end(e), i0 = 31 - __clz(at.starts & ((2u << e) - 1u));  // or -1
                if (i0 < 0 ? !a.d_final : !a.d_init) continue;
                float2 v = a.d_final && n >= 0 ? load2(a.d_final, n, D, ch) : f2(0.f);
#pragma unroll 1
                for (int i = e; i >= (i0 < 0 ? 0 : i0); --i)
                    v = scan_back(scan_depth2(tile_at<BF16>(st, i, lane)), tile_at<BF16>(st + 2 * K::ROWS, i, lane), v);
                if (i0 < 0) c = v;
                else if (a.d_init && n >= 0) store2_odd(a.d_init, false, n, D, ch, v);
            }
        }
        float4 piece = scan_piece(false, sum, c);
        if (at.ends) {  // nothing of what lies behind gets through
            const float2 b = at.ends == 1u << (NT - 1) ? scan_fold2(piece, c_end) : c;
            piece = make_float4(SC_CUT, SC_CUT, b.x, b.y);
        }
        __syncwarp();
        if (!failed) load(s + 2, tw + 2 * by);  // into the stage that this warp has just read

        // the pieces of the warps with later tokens; its own joined to them goes on
        float4 before = make_float4(-0.f, -0.f, 0.f, 0.f);
        if (warp > 0) {
            failed = failed || !scan_wait<false>(given - 2 + (s & 1), phase, a.status);
            before = ab[(warp - 1) * 32 + lane];
            piece = scan_join2(before, piece);
        }
        ab[warp * 32 + lane] = piece;
        if (warp < SC_WARPS - 1) {
            __syncwarp();
            if (lane == 0) mbar_arrive(given + (s & 1));
        } else {
            const int slot = (s & 3) * cluster + rank;
            if (cluster > 1) {
                const uint32_t to = smem_u32(ex + slot * 32 + lane), on = smem_u32(sent + slot);
                for (int k = 0; k < cluster; ++k) st_async16(map_to_cta(to, k), piece, map_to_cta(on, k));
            } else {
                ex[slot * 32 + lane] = piece;
                __syncwarp();
                if (lane == 0) mbar_arrive(sent + slot);
            }
        }
        if (warp == 0) {
            for (int k = 0; k < cluster; ++k) {
                const bool last = rank + k < cluster;
                const int r = last ? rank + k : rank + k - cluster, q = last ? s - 1 : s, slot = (q & 3) * cluster + r;
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
        if (ends_here) mine = c_end;

        if (plain) {
            if (!even) {
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const float2 G = __ffma2_rn(as[i], mine, gs[i]);
                    store2_odd(a.dx, a.out_bf16, (size_t)(tw + i), D, ch, __fmul2_rn(G, kx[i]));
                    store2_odd(a.dl, a.out_bf16, (size_t)(tw + i), D, ch, __fmul2_rn(G, kl[i]));
                    if (GATE) store2_odd(a.dg, a.out_bf16, (size_t)(tw + i), D, ch, __fmul2_rn(G, kg[i]));
                }
            } else if (ch < D) {
                const uint32_t es = a.out_bf16 ? 2 : 4, row = (uint32_t)D * es;
                const size_t off = (size_t)tw * row + (size_t)ch * es;
                uint8_t* const px = static_cast<uint8_t*>(a.dx) + off;
                uint8_t* const pl = static_cast<uint8_t*>(a.dl) + off;
                uint8_t* const pg = static_cast<uint8_t*>(a.dg) + off;
                if (a.out_bf16) {
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        const float2 G = __ffma2_rn(as[i], mine, gs[i]);
                        const float2 x = __fmul2_rn(G, kx[i]), l = __fmul2_rn(G, kl[i]);
                        *reinterpret_cast<uint32_t*>(px + (size_t)row * i) = pack_bf16x2(x.x, x.y);
                        *reinterpret_cast<uint32_t*>(pl + (size_t)row * i) = pack_bf16x2(l.x, l.y);
                        if (GATE) {
                            const float2 g = __fmul2_rn(G, kg[i]);
                            *reinterpret_cast<uint32_t*>(pg + (size_t)row * i) = pack_bf16x2(g.x, g.y);
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        const float2 G = __ffma2_rn(as[i], mine, gs[i]);
                        *reinterpret_cast<float2*>(px + (size_t)row * i) = __fmul2_rn(G, kx[i]);
                        *reinterpret_cast<float2*>(pl + (size_t)row * i) = __fmul2_rn(G, kl[i]);
                        if (GATE) *reinterpret_cast<float2*>(pg + (size_t)row * i) = __fmul2_rn(G, kg[i]);
                    }
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const bool from_end = at.ends & ALL_BUT_LAST & ~((1u << i) - 1u);
                const float2 G = from_end ? gs[i] : __ffma2_rn(as[i], mine, gs[i]);
                if (!(at.own >> i & 1)) continue;
                if (TMA || (!BF16 && even)) {  // in line where the registers allow it: 101 -> 97 us, 4 x 2048 x 4096
                    store2_even(a.dx, a.out_bf16, (size_t)(tw + i), D, ch, __fmul2_rn(G, kx[i]));
                    store2_even(a.dl, a.out_bf16, (size_t)(tw + i), D, ch, __fmul2_rn(G, kl[i]));
                    if (GATE) store2_even(a.dg, a.out_bf16, (size_t)(tw + i), D, ch, __fmul2_rn(G, kg[i]));
                } else {
                    store2(a.dx, a.out_bf16, (size_t)(tw + i), D, ch, __fmul2_rn(G, kx[i]));
                    store2(a.dl, a.out_bf16, (size_t)(tw + i), D, ch, __fmul2_rn(G, kl[i]));
                    if (GATE) store2(a.dg, a.out_bf16, (size_t)(tw + i), D, ch, __fmul2_rn(G, kg[i]));
                }
            }
        }
        if (a.d_init && at.starts) {
            const int i = 31 - __clz(at.starts);  // the start whose sequence goes on behind the warp's tokens
            if (!(at.ends & ALL_BUT_LAST & ~((1u << i) - 1u))) {
                float2 v;
                if (i == 0) {  // all pieces up to the sequence's first token over what lies behind the tile
                    const float4 all = ab[warp * 32 + lane];
                    v = scan_fold2(all, base[(s & 1) * 32 + lane], scan_is_cut(all));
                } else {
                    v = scan_d_init<BF16>(a.log_alpha, a.ld_l, a.d_h, a.ld_dh, tw + i, __popc(at.own >> i), D, ch, mine);
                }
                store2(a.d_init, false, at.seq_start(i), D, ch, v);
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
    if (a.d_init && rank == 0) {
        for (int n = sp.n0 + warp; n < sp.n1; n += SC_WARPS) {
            int64_t first, end;
            scan_range(a.cu, n, a.T, &first, &end);
            if (first == end)
                store2(a.d_init, false, n, D, ch, a.d_final ? load2(a.d_final, n, D, ch) : f2(0.f));
        }
    }
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
    const void* in[] = {a.log_alpha, a.x, a.d_h, a.gate};
    const int64_t ld[] = {a.ld_l, a.ld_x, a.ld_dh, a.ld_g};
    ScanMaps maps;
    int width = 0;
    if ((e = scan_maps(a, in, ld, a.gate ? 4 : 3, SCAN_CHUNK, &maps, &width)) != cudaSuccess) return e;
    const int64_t chunks = ((a.cu ? a.T : (int64_t)a.B * a.T) + SCAN_CHUNK - 1) / SCAN_CHUNK;
    if (width == 16 && a.D % 4 != 0) width = 4;
    if (width == 16 && chunks > 0 && !make_scan_map(&maps.states, a.chunk_states, chunks, a.D, a.D, 1, false))
        return cudaErrorInvalidValue;
#define KDA_SCAN_BWD(BF, TMA) \
    e = scan_launch<scan_bwd_kernel<BF, G, W, TMA>>(ScanBwd<BF, G>::smem, SC_WARPS * SCAN_CHUNK, a, maps, width, \
                                                    own_states || a.status, stream)
    KDA_SCAN_GN(a.gate != nullptr, a.normalize, {
        if (a.in_bf16) { if (width == 16) KDA_SCAN_BWD(true, true); else KDA_SCAN_BWD(true, false); }
        else           { if (width == 16) KDA_SCAN_BWD(false, true); else KDA_SCAN_BWD(false, false); }
    });
#undef KDA_SCAN_BWD
    return e;
}

}  // namespace kda
