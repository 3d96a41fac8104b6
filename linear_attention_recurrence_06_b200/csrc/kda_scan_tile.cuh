// kda_scan_tile.cuh -- what the tiled kernels of the element-wise scan share:
// their geometry, the asynchronous loads, where sequences begin and end inside a
// tile, and the exchange between the CTAs of a cluster.
//
// A CTA of 8 warps owns 64 channels (lane l: channels 2l and 2l + 1) and walks
// tiles of 8 x NT tokens; warp w takes tokens NT w .. NT w + NT - 1 of a tile.  A
// piece of the recurrence is affine in the state before it, h -> A h + B with
// A = e^{sum l}: a warp runs its tokens from zero, joins its piece (A, B) to those of
// the warps before it and hands the result to the next warp; the last warp sends
// the tile's piece to all CTAs of the cluster, which take neighbouring tiles.  The
// first warp folds the pieces of all earlier tiles over the carried state and gives
// the others the state before the tile; each finishes its tokens in registers.
// Pieces are always joined from left to right: the result does not depend on
// timing.  Warps meet only at those hand-overs (mbarriers); loads, too, are a
// warp's own, so that warps of earlier tokens can be most of a step ahead of those
// that wait for them.
// Why this split: the channels of one sequence alone (32 x 64 lanes for 4096) cannot
// keep enough loads in flight, time has to be split; a cluster does that in one
// pass over the data, without flags in global memory and without a second launch.  (A warp's
// piece handed to all others by itself instead of along the chain took 84 us for the case that
// kda_scan.cu names first, then at 59 us.)
#pragma once
#include "kda_scan.cuh"
#include "kda_scan.h"

namespace kda {

constexpr int SC_WARPS = 8, SC_THREADS = 256;
constexpr int SC_CH = 64;           // channels of a CTA
constexpr int SC_MAX_CLUSTER = 8;   // the portable limit

template <bool BF16>
struct ScanGeo {
    static constexpr int ES = BF16 ? 2 : 4;
    static constexpr int ROWB = SC_CH * ES;       // bytes of a tile's row
};

// ---- two channels at a time
KDA_DEV float2 f2(float x, float y) { return make_float2(x, y); }
KDA_DEV float2 f2(float x) { return make_float2(x, x); }

// Decays of two channels, `d` = -l >= 0:  a = e^-d and m = 1 - a.  m is its Taylor polynomial to d^5 below
// 1/8 (the next term is below 2^-24 of m there), above it what a leaves of 1.  FINE (fp32 tokens): a = 1 - m
// below 1/8, above it the hardware's e^-d; else the latter everywhere.  A warp's tokens are stepped with a
// as it is: its rounding does not add up beyond them, for what is handed on, to the next warp or to the caller
// and a next call, goes by the sum of the d (scan_piece) or by steps of scan_p2.  The hardware's errors, below 2 steps, lean one way: h is off by 1.8e-7 of it (root mean square)
// instead of 1.2e-7, by 0.9e-7 on average instead of 1e-8.  With fp32 tokens that would reach the caller, and 1 - m costs nothing (90 us,
// 4 x 2048 x 4096 forward: those kernels wait for memory); with bf16 tokens it is a thousandth of what their own
// rounding leaves open, and 1 - m would take 55 us for 54, without either factor 40 for 35.
constexpr float SCAN_NEAR = 0.125f;
struct ScanDecay2 {
    float2 a, m;
};
template <bool FINE>
KDA_DEV ScanDecay2 scan_decay2(float2 d) {
    ScanDecay2 r;
    float2 t = __ffma2_rn(d, f2(1.f / 120.f), f2(-1.f / 24.f));
    t = __ffma2_rn(t, d, f2(1.f / 6.f));
    t = __ffma2_rn(t, d, f2(-0.5f));
    const float2 near = __ffma2_rn(__fmul2_rn(t, d), d, d);
    const float2 x = __fmul2_rn(d, f2(-LOG2E));
    const float2 e = f2(ex2_ftz(x.x), ex2_ftz(x.y));
    const float2 m1 = __ffma2_rn(e, f2(-1.f), f2(1.f)), a1 = __ffma2_rn(near, f2(-1.f), f2(1.f));
    const bool nx = d.x < SCAN_NEAR, ny = d.y < SCAN_NEAR;
    r.m = f2(nx ? near.x : m1.x, ny ? near.y : m1.y);
    r.a = FINE ? f2(nx ? a1.x : e.x, ny ? a1.y : e.y) : e;
    return r;
}
// -l of two channels: max(-log_alpha, 0), NaN kept
KDA_DEV float2 scan_depth2(float2 log_alpha) {
    float2 r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r.x) : "f"(-log_alpha.x), "f"(0.f));
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r.y) : "f"(-log_alpha.y), "f"(0.f));
    return r;
}
KDA_DEV float2 unpack2(uint32_t w) { return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }
// The same from a tile's row: two bf16 are clamped at once.
template <bool BF16>
KDA_DEV float2 depth_at(const uint8_t* tile, int row, int lane) {
    if constexpr (BF16) {
        uint32_t w = *reinterpret_cast<const uint32_t*>(tile + row * (SC_CH * 2) + lane * 4) ^ 0x80008000u;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(w) : "r"(w), "r"(0u));
        return unpack2(w);
    } else {
        return scan_depth2(*reinterpret_cast<const float2*>(tile + row * (SC_CH * 4) + lane * 8));
    }
}

// w s of two channels.  With both factors w s = sqrt(n) / q = n rsqrt(n q^2), n = 1 - a^2, q = 1 + e^-gate:
// one special function less (the forward spends three per value then; at four they alone
// take as long as the memory).  q^2 overflows for a gate below -44: s = 1e-19 counts as 0 there.
template <bool GATE, bool NORM>
KDA_DEV float2 scan_weight2(float2 m, float2 g) {
    float2 q = f2(1.f);
    if (GATE) {
        const float2 x = __fmul2_rn(g, f2(-LOG2E));
        q = __fadd2_rn(f2(ex2_ftz(x.x), ex2_ftz(x.y)), f2(1.f));
    }
    if (!NORM) return GATE ? f2(rcp_ftz(q.x), rcp_ftz(q.y)) : f2(1.f);
    const float2 n = __fmul2_rn(m, __ffma2_rn(m, f2(-1.f), f2(2.f)));
    float2 r = __fadd2_rn(n, f2(SCAN_TINY));
    if (GATE) r = __fmul2_rn(__fmul2_rn(r, q), q);
    return __fmul2_rn(n, f2(rsqrt_ftz(r.x), rsqrt_ftz(r.y)));
}

// A piece of the recurrence, h -> A h + B, of both channels in a float4 {A0, A1, B0, B1}, A in scan_decay's
// form (hundreds of slow pieces in a row would show the rounding of A itself), SC_CUT in
// both for a piece in which a sequence starts: nothing of the state before it gets through.
constexpr float SC_CUT = -2.f;
KDA_DEV float2 scan_step2(float2 p, float2 h, float2 u) {
    const float2 t = __ffma2_rn(p, h, u);
    return __fadd2_rn(t, f2(__uint_as_float(__float_as_uint(h.x) & (uint32_t)(__float_as_int(p.x) >> 31)),
                            __uint_as_float(__float_as_uint(h.y) & (uint32_t)(__float_as_int(p.y) >> 31))));
}
// e^-depth of both channels in scan_decay's form
KDA_DEV float2 scan_p2(float2 depth, const ScanDecay2& d) {
    return f2(depth.x < SCAN_NEAR ? -d.m.x : d.a.x, depth.y < SCAN_NEAR ? -d.m.y : d.a.y);
}
KDA_DEV float4 scan_piece(bool cut, float2 depth, float2 b) {
    const float2 p = scan_p2(depth, scan_decay2<true>(depth));
    return make_float4(cut ? SC_CUT : p.x, cut ? SC_CUT : p.y, b.x, b.y);
}
KDA_DEV float2 scan_fold2(float4 v, float2 h) { return scan_step2(f2(v.x, v.y), h, f2(v.z, v.w)); }
KDA_DEV float2 scan_fold2(float4 v, float2 h, bool cut) { return cut ? f2(v.z, v.w) : scan_fold2(v, h); }
// A of two pieces in a row, none of them cut
KDA_DEV float scan_join_a(float a, float b) {
    return scan_slow(a) && scan_slow(b) ? __uint_as_float(__float_as_uint(fmaf(a, b, a + b)) | 0x80000000u)
                                        : scan_a(a) * scan_a(b);
}
KDA_DEV bool scan_is_cut(float4 v) { return v.x < -1.f; }
// the piece v behind the piece all
KDA_DEV float4 scan_join2(float4 all, float4 v) {
    const bool cut = scan_is_cut(v);
    const float2 b = scan_fold2(v, f2(all.z, all.w), cut);
    if (cut || scan_is_cut(all)) return make_float4(SC_CUT, SC_CUT, b.x, b.y);
    return make_float4(scan_join_a(all.x, v.x), scan_join_a(all.y, v.y), b.x, b.y);
}

// ---- loads
// A warp's NT rows of one tensor come by TMA where its rows are 16-byte aligned (zeros behind the
// last row and channel), else by asynchronous copies of 4 bytes, or by plain loads of odd
// rows of 2-byte values; tokens outside [t0, t1) and channels from D on become zeros.  TMA has kernels
// of its own: the calls of the others take registers from it (4 x 2048 x 4096 forward: 60 us with
// them, 58 us without).
KDA_DEV void cp_async4_zfill(uint32_t dst, const void* src, int n) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
KDA_DEV void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
KDA_DEV void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <bool BF16, int NT>
__device__ __noinline__ void load_rows(uint8_t* dst, const void* base, int64_t ld, int tw, int t0, int t1, int ch0, int D,
                                       int width, int lane) {
    using Geo = ScanGeo<BF16>;
    constexpr int ES = Geo::ES;
    const uint8_t* const src = static_cast<const uint8_t*>(base);
    const bool whole = tw >= t0 && tw + NT <= t1;
    if (!BF16 || width == 4) {
#pragma unroll
        for (int k = 0; k < Geo::ROWB / 128; ++k) {
            const int ch = ch0 + (lane + 32 * k) * (4 / ES);
            const int left = (D - ch) * ES, n = left < 0 ? 0 : (left > 4 ? 4 : left);
            const uint32_t to = smem_u32(dst + (lane + 32 * k) * 4);
            if (whole) {
                const uint8_t* p = n > 0 ? src + ((size_t)tw * ld + ch) * ES : src;
                const int64_t step = n > 0 ? ld * ES : 0;
#pragma unroll
                for (int i = 0; i < NT; ++i, p += step) cp_async4_zfill(to + i * Geo::ROWB, p, n);
            } else {
                for (int i = 0; i < NT; ++i) {
                    const int t = tw + i;
                    const bool in = t >= t0 && t < t1 && n > 0;
                    cp_async4_zfill(to + i * Geo::ROWB, in ? src + ((size_t)t * ld + ch) * ES : src, in ? n : 0);
                }
            }
        }
    } else {
        // rows at odd multiples of 2 bytes: no copy fits, but all loads are on their way before the first is needed
        const int ch = ch0 + 2 * lane;
        const uint16_t* const s = reinterpret_cast<const uint16_t*>(src) + ch;
        uint32_t lo[NT], hi[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int t = tw + i;
            const bool row_in = whole || (t >= t0 && t < t1);
            lo[i] = row_in && ch < D ? __ldg(s + (size_t)t * ld) : 0u;
            hi[i] = row_in && ch + 1 < D ? __ldg(s + (size_t)t * ld + 1) : 0u;
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) *reinterpret_cast<uint32_t*>(dst + i * Geo::ROWB + lane * 4) = lo[i] | hi[i] << 16;
    }
}

// channels 2 lane, 2 lane + 1 of a tile's row
template <bool BF16>
KDA_DEV float2 tile_at(const uint8_t* tile, int row, int lane) {
    if constexpr (BF16) {
        return unpack2(*reinterpret_cast<const uint32_t*>(tile + row * (SC_CH * 2) + lane * 4));
    } else {
        return *reinterpret_cast<const float2*>(tile + row * (SC_CH * 4) + lane * 8);
    }
}

// Two channels of a row of an output [tokens, D].
static __device__ __noinline__ void store2(void* base, bool bf16, size_t row, int D, int ch, float2 v) {
    const size_t i = row * D + ch;
    if (ch + 1 < D && (D & 1) == 0) {
        if (bf16) *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(base) + i) = pack_bf16x2(v.x, v.y);
        else *reinterpret_cast<float2*>(static_cast<float*>(base) + i) = v;
        return;
    }
    if (ch < D) {
        if (bf16) static_cast<uint16_t*>(base)[i] = f32_to_bf16(v.x);
        else static_cast<float*>(base)[i] = v.x;
    }
    if (ch + 1 < D) {
        if (bf16) static_cast<uint16_t*>(base)[i + 1] = f32_to_bf16(v.y);
        else static_cast<float*>(base)[i + 1] = v.y;
    }
}
// The same in line for even D.
KDA_DEV void store2_even(void* base, bool bf16, size_t row, int D, int ch, float2 v) {
    if (ch >= D) return;
    const size_t i = row * D + ch;
    if (bf16) *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(base) + i) = pack_bf16x2(v.x, v.y);
    else *reinterpret_cast<float2*>(static_cast<float*>(base) + i) = v;
}
// The same in line for odd D.
KDA_DEV void store2_odd(void* base, bool bf16, size_t row, int D, int ch, float2 v) {
    const size_t i = row * D + ch;
    if (bf16) {
        uint16_t* const p = static_cast<uint16_t*>(base) + i;
        if (ch < D) p[0] = f32_to_bf16(v.x);
        if (ch + 1 < D) p[1] = f32_to_bf16(v.y);
    } else {
        float* const p = static_cast<float*>(base) + i;
        if (ch < D) p[0] = v.x;
        if (ch + 1 < D) p[1] = v.y;
    }
}
// A token's step of the gradient, back in time, without its decay's rounding: c from behind the token, then from
// before it.
KDA_DEV float2 scan_back(float2 depth, float2 d_h, float2 c) {
    return scan_step2(scan_p2(depth, scan_decay2<true>(depth)), __fadd2_rn(d_h, c), f2(0.f));
}
// The gradient of the initial state (channels ch, ch + 1) of a sequence whose first token is t: c, what comes from behind
// token t + n - 1, taken back over n tokens without the roundings of decays.  For the few warps in which a sequence begins
// behind the first token: its decays and d_h are loaded once more, which leaves the others their registers, a token
// ahead; rolled, as code that is new to an SM takes longer to come than to run.
template <bool BF16>
__device__ __noinline__ float2 scan_d_init(const void* log_alpha, int64_t ld, const void* d_h, int64_t ld_dh, int t, int n,
                                           int D, int ch, float2 c) {
    size_t at = (size_t)(t + n - 1) * ld + ch, at_dh = (size_t)(t + n - 1) * ld_dh + ch;
    auto row = [&](const void* base, size_t i) {
        return f2(ch < D ? ld_in<BF16>(base, i) : 0.f, ch + 1 < D ? ld_in<BF16>(base, i + 1) : 0.f);
    };
    float2 l = row(log_alpha, at), g = row(d_h, at_dh);
#pragma unroll 1
    for (int i = n; i > 0; --i) {
        const float2 d = scan_depth2(l), dh = g;
        at -= ld, at_dh -= ld_dh;
        if (i > 1) l = row(log_alpha, at), g = row(d_h, at_dh);
        c = scan_back(d, dh, c);
    }
    return c;
}
KDA_DEV float2 load2(const float* base, size_t row, int D, int ch) {
    const size_t i = row * D + ch;
    return f2(ch < D ? base[i] : 0.f, ch + 1 < D ? base[i + 1] : 0.f);
}

// ---- sequences
// First m in [lo, hi) with cu[m] >= v (hi if there is none); all lanes of a warp.
KDA_DEV int warp_lower_bound(const int32_t* __restrict__ cu, int lo, int hi, int v, int lane) {
    while (lo < hi) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + lane * step;
        const int k = __popc(__ballot_sync(0xffffffffu, at < hi && cu[at] < v));
        if (k == 0) return lo;
        const int end = lo + k * step;
        lo += (k - 1) * step + 1;
        hi = end < hi ? end : hi;
    }
    return lo;
}

// The part of the tokens that a CTA walks: whole sequences n0 .. n1 - 1, tokens [t0, t1).  (Tokens
// are counted in 32 bits; offsets of elements in 64.)
struct ScanSpan {
    int n0, n1, t0, t1;
};
// That of split s of S.  Packed sequences go to the splits by their first token.  There the CTAs of a cluster
// take a part each, on their own, where their sequences can be shared out about evenly: *cluster
// and *rank then become 1 and 0.  (Sharing the tiles of all sequences instead costs an exchange per
// tile: 40 sequences of 512 tokens x 4096 take 149 us with CTAs on their own, a quarter more in clusters; but
// 16,384 tokens in one of 41 sequences two thirds more on their own than the 161 us in clusters of 2.)
KDA_DEV ScanSpan scan_span(const ScanArgs& a, int s, int S, int tile, int* cluster, int* rank, int lane) {
    ScanSpan r;
    if (!a.cu) {
        r.n0 = S == 1 ? 0 : (int)((int64_t)a.B * s / S);
        r.n1 = S == 1 ? a.B : (int)((int64_t)a.B * (s + 1) / S);
        r.t0 = r.n0 * (int)a.T;
        r.t1 = r.n1 * (int)a.T;
        return r;
    }
    int end = a.cu[a.n_seqs];
    end = end < 0 ? 0 : (end > (int)a.T ? (int)a.T : end);
    // lane k: the first sequence of part k and its first token
    const int C = *cluster, part = s * C + (lane < C ? lane : C), parts = S * C;
    int n = 0, t = 0;
    if (part == parts) {
        n = a.n_seqs;
        t = end;
    } else if (part > 0) {
        const int v = (int)((int64_t)end * part / parts);
        for (int hi = a.n_seqs; n < hi;) {
            const int mid = n + (hi - n) / 2;
            if (a.cu[mid] < v) n = mid + 1;
            else hi = mid;
        }
        t = n < a.n_seqs ? a.cu[n] : end;
        t = t < 0 ? 0 : (t > end ? end : t);
    }
    auto part_of = [&](int from, int to) {
        ScanSpan v;
        v.n0 = __shfl_sync(0xffffffffu, n, from);
        v.n1 = __shfl_sync(0xffffffffu, n, to);
        v.t0 = __shfl_sync(0xffffffffu, t, from);
        v.t1 = __shfl_sync(0xffffffffu, t, to);
        if (v.t1 < v.t0) v.t1 = v.t0;
        return v;
    };
    r = part_of(0, C);
    if (C > 1) {
        const int next = __shfl_down_sync(0xffffffffu, t, 1);
        const int most = __reduce_max_sync(0xffffffffu, lane < C ? next - t : 0);
        // on its own, the busiest has at most a quarter more than an equal part, and a few tiles
        if ((int64_t)most * C <= (int64_t)(r.t1 - r.t0) / 4 * 5 + 4 * C * tile) {
            r = part_of(*rank, *rank + 1);
            *cluster = 1;
            *rank = 0;
        }
    }
    return r;
}

// Where sequences meet among a warp's NT tokens: bit j of `starts` / `ends`: token tw + j is the
// first / last of its sequence, whose number is seq_start(j) / seq_end(j) (-1 can come of a
// cu_seqlens that begins behind 0); bit j of `own`: the token is one of this split's.  Until
// step `calm` there is nothing more to see, and scan_look() need not be called.
struct ScanSeen {
    uint32_t starts, ends, own;
    int calm;
    int lane_start, lane_end;  // lane j: the sequences that start at and end with token tw + j
    KDA_DEV int seq_start(int j) const { return __shfl_sync(0xffffffffu, lane_start, j); }
    KDA_DEV int seq_end(int j) const { return __shfl_sync(0xffffffffu, lane_end, j); }
};

// For step s, whose tokens begin at tw; those of the next steps at tw + by, tw + 2 by, ...  `tab`: 2 NT
// ints of shared memory of this warp, used before the return.  Returns {starts | ends << 16,
// own | steps until the next look << 16, lane_start, lane_end}, the first two the same on all lanes.
// Rarely called: kept out of the loop, and its arguments and result in registers.
template <int NT>
__device__ __noinline__ uint4 scan_look(const int32_t* __restrict__ cu, int n_seqs, int T, int t0, int t1, int tw,
                                        int by, int* tab) {
    constexpr uint32_t ALL = (1u << NT) - 1u;
    const int lane = threadIdx.x & 31;
    uint32_t own = ALL;
    if (tw < t0) own = t0 - tw >= NT ? 0u : own & ~((1u << (t0 - tw)) - 1u);
    if (tw + NT > t1) own = tw >= t1 ? 0u : own & ((1u << (t1 - tw)) - 1u);
    if (own == 0) return make_uint4(0u, 1u << 16, 0u, 0u);
    int prev, next;  // the last meeting point before tw, the first at or behind it
    int m = 0;
    const int N1 = n_seqs + 1;
    if (cu) {
        m = warp_lower_bound(cu, 0, N1, tw, lane);
        next = m < N1 ? cu[m] : INT32_MAX;
        prev = m > 0 ? cu[m - 1] : -1;
    } else {
        const int r = tw % T;
        next = r == 0 ? tw : (T > INT32_MAX - tw + r ? INT32_MAX : tw - r + T);
        prev = r == 0 ? tw - T : tw - r;
    }
    if (next > tw + NT) {
        if (own != ALL) return make_uint4(0u, own | 1u << 16, 0u, 0u);
        // nothing to look at while tw + NT < next and tw + NT <= t1 (forwards), tw > prev and
        // tw >= t0 (backwards)
        const int room = by > 0 ? (next < t1 + 1 ? next : t1 + 1) - NT - tw : tw - (prev > t0 - 1 ? prev : t0 - 1);
        const int step = by > 0 ? by : -by, steps = (room - 1) / step + 1;
        return make_uint4(0u, own | (uint32_t)(steps < 1 ? 1 : (steps > 65535 ? 65535 : steps)) << 16, 0u, 0u);
    }
    uint32_t meet = 0;  // bit j: a sequence starts at tw + j, j = 0 .. NT
    int lane_start, lane_end;
    __syncwarp();
    if (cu) {
        int before = -1;  // the value of the entry before the window
        for (int k = m; k < N1; k += 32) {
            const int v = k + lane < N1 ? cu[k + lane] : INT32_MAX;
            const int up = __shfl_up_sync(0xffffffffu, v, 1), down = __shfl_down_sync(0xffffffffu, v, 1);
            const bool in = v >= tw && v <= tw + NT;
            const int j = in ? v - tw : 0;
            if (in && j < NT && (lane == 31 || down != v)) tab[j] = k + lane;  // the last entry of a value
            if (in && j > 0 && (lane == 0 ? before != v : up != v)) tab[NT + j - 1] = k + lane - 1;  // the first
            meet |= __reduce_or_sync(0xffffffffu, in ? 1u << j : 0u);
            before = __shfl_sync(0xffffffffu, v, 31);
            if (__ballot_sync(0xffffffffu, in) != 0xffffffffu) break;
            __syncwarp();
        }
        __syncwarp();
        lane_start = lane < NT ? tab[lane] : 0;
        lane_end = lane < NT ? tab[NT + lane] : 0;
        __syncwarp();
    } else {
        const int t = tw + lane, n = t / T;
        lane_start = n;
        lane_end = (t + 1) / T - 1;
        meet = __ballot_sync(0xffffffffu, lane <= NT && n * T == t);
    }
    return make_uint4((meet & own) | ((meet >> 1) & own) << 16, own | 1u << 16, (uint32_t)lane_start, (uint32_t)lane_end);
}
// The same as ScanSeen; `calm`: the step to look again.
template <int NT>
KDA_DEV ScanSeen scan_see(const ScanArgs& a, const ScanSpan& sp, int s, int tw, int by, int* tab) {
    const uint4 r = scan_look<NT>(a.cu, a.n_seqs, (int)a.T, sp.t0, sp.t1, tw, by, tab);
    ScanSeen v;
    v.starts = r.x & 0xffffu;
    v.ends = r.x >> 16;
    v.own = r.y & 0xffffu;
    v.lane_start = (int)r.z;
    v.lane_end = (int)r.w;
    v.calm = s + (int)(r.y >> 16);  // the same on all lanes, like the masks
    return v;
}

// ---- clusters
KDA_DEV void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
KDA_DEV void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Waits like mbar_wait; PEERS: for what other CTAs of the cluster have written.  The first look is in
// line, the rest out of it.
template <bool PEERS>
KDA_DEV bool scan_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    if constexpr (PEERS)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok) : "r"(bar), "r"(parity), "r"(20000u) : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok) : "r"(bar), "r"(parity), "r"(20000u) : "memory");
    return ok != 0;
}
template <bool PEERS>
__device__ __noinline__ bool scan_wait_long(uint32_t bar, uint32_t parity, uint32_t* status) {
    const unsigned long long t0 = globaltimer_ns();
    while (!scan_try<PEERS>(bar, parity)) {
        if (globaltimer_ns() - t0 > WAIT_LIMIT_NS) {
            if (status) atomicOr(status, DEV_ERR_TIMEOUT);
            return false;
        }
    }
    return true;
}
template <bool PEERS>
KDA_DEV bool scan_wait(uint64_t* bar, uint32_t parity, uint32_t* status) {
    const uint32_t b = smem_u32(bar);
    return scan_try<PEERS>(b, parity) || scan_wait_long<PEERS>(b, parity, status);
}
// After a wait has given up: a warp's loads that may still be on their way into its two stages.  How far the
// barriers had come is not known, so both parities are waited for, each with the limit.
static __device__ __noinline__ void scan_drain(uint64_t* full) {
    for (int i = 0; i < 4; ++i) scan_wait<false>(full + (i & 1), i >> 1, nullptr);
}
// 16 bytes into a CTA's shared memory, counted on its barrier
KDA_DEV void st_async16(uint32_t addr, float4 v, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr),
                 "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(bar)
                 : "memory");
}

}  // namespace kda
