// kda_scan_tile.cuh -- what the tiled kernels of the element-wise scan share:
// their geometry, the asynchronous loads, where sequences begin and end inside a
// tile, and the exchange between the CTAs of a cluster.
//
// A CTA of 8 warps owns 64 channels (lane l: channels 2l and 2l + 1) and walks
// tiles of 8 x NT tokens; warp w takes tokens NT w .. NT w + NT - 1 of a tile.  A
// piece of the recurrence is affine in the state before it, h -> A h + B with
// A = e^{sum l}, so a warp first runs its tokens from zero (A, B), the CTA folds the
// warps' pieces over the carried state in order, and each warp then runs its
// tokens again from the state it starts at, in registers.  The CTAs of a cluster
// take neighbouring tiles and exchange their (A, B) through distributed shared
// memory once per tile; every CTA folds all of them over its own copy of the
// carried state, always from left to right: the result does not depend on timing.
// Why this split: the channels of one sequence alone (32 x 64 lanes for 4096) cannot
// keep enough loads in flight, time has to be split; a cluster does that in one
// pass over the data, without flags in global memory and without a second launch.
#pragma once
#include "kda_scan.cuh"
#include "kda_scan.h"

namespace kda {

constexpr int SC_WARPS = 8, SC_THREADS = 256;
constexpr int SC_CH = 64;           // channels of a CTA
constexpr int SC_MAX_CLUSTER = 8;   // the portable limit

template <bool BF16, int NT>
struct ScanGeo {
    static constexpr int ES = BF16 ? 2 : 4;
    static constexpr int TILE = SC_WARPS * NT;
    static constexpr int ROWB = SC_CH * ES;       // bytes of a tile's row
    static constexpr int TENS = TILE * ROWB;      // bytes of one tensor's tile
};

// ---- two channels at a time
KDA_DEV float2 f2(float x, float y) { return make_float2(x, y); }
KDA_DEV float2 f2(float x) { return make_float2(x, x); }

// The tiled kernels keep a decay as e + lo: e = e^l as the hardware approximates it, lo what is missing to
// 1 + (e^l - 1) with e^l - 1 from scan_decay's polynomial (0 where l <= -1/4, where e is good
// enough).  A step is then two fused products for two channels at once, without a choice, and
// keeps slow and fast decays as scan_step does.  lo is within a few 2^-24 and its own error
// does not matter, so two of them wait in one register as bf16 for the second run.
struct ScanDecay2 {
    float2 e, lo, em;  // em = e^l - 1
};
KDA_DEV ScanDecay2 scan_decay2(float2 l) {
    ScanDecay2 r;
    float2 t = __ffma2_rn(l, f2(1.f / 720.f), f2(1.f / 120.f));
    t = __ffma2_rn(t, l, f2(1.f / 24.f));
    t = __ffma2_rn(t, l, f2(1.f / 6.f));
    t = __ffma2_rn(t, l, f2(0.5f));
    const float2 slow = __ffma2_rn(__fmul2_rn(t, l), l, l);
    const float2 x = __fmul2_rn(l, f2(LOG2E));
    r.e = f2(ex2_ftz(x.x), ex2_ftz(x.y));
    const float2 e1 = __fadd2_rn(r.e, f2(-1.f));
    r.em = f2(l.x > SCAN_SLOW ? slow.x : e1.x, l.y > SCAN_SLOW ? slow.y : e1.y);
    r.lo = __ffma2_rn(e1, f2(-1.f), r.em);
    return r;
}
KDA_DEV float2 scan_step2(float2 e, float2 lo, float2 h, float2 u) { return __ffma2_rn(lo, h, __ffma2_rn(e, h, u)); }
KDA_DEV float2 unpack2(uint32_t w) { return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }

// w s of two channels (scan_term's), and s
template <bool GATE, bool NORM>
KDA_DEV float2 scan_weight2(float2 em, float2 g, float2* s) {
    float2 ws = f2(1.f);
    if (GATE) {
        const float2 x = __fmul2_rn(g, f2(-LOG2E));
        const float2 d = __fadd2_rn(f2(ex2_ftz(x.x), ex2_ftz(x.y)), f2(1.f));
        ws = f2(rcp_ftz(d.x), rcp_ftz(d.y));
        *s = ws;
    }
    if (NORM) {
        const float2 n = __ffma2_rn(em, __fmul2_rn(em, f2(-1.f)), __fmul2_rn(em, f2(-2.f)));  // 1 - a^2
        const float2 w = __fmul2_rn(n, f2(rsqrt_ftz(fmaxf(n.x, SCAN_TINY)), rsqrt_ftz(fmaxf(n.y, SCAN_TINY))));
        ws = GATE ? __fmul2_rn(ws, w) : w;
    }
    return ws;
}

// A piece is kept as (A, B) of both channels in a float4 {A0, A1, B0, B1}, A in scan_decay's
// form (hundreds of slow pieces in a row would show the rounding of A itself), SCAN_CUT for
// a piece in which a sequence starts: nothing of the state before it gets through.
constexpr float SCAN_CUT = -2.f;
KDA_DEV float scan_fold(float A, float B, float h) { return A < -1.f ? B : scan_step(A, h, B); }
KDA_DEV float2 scan_fold2(float4 ab, float2 h) { return f2(scan_fold(ab.x, ab.z, h.x), scan_fold(ab.y, ab.w, h.y)); }
// A of two pieces in a row
KDA_DEV float scan_join_a(float a, float b) {
    if (a < -1.f || b < -1.f) return SCAN_CUT;
    if (scan_slow(a) && scan_slow(b)) return __uint_as_float(__float_as_uint(fmaf(a, b, a + b)) | 0x80000000u);
    return scan_a(a) * scan_a(b);
}
// the piece `ab` behind the piece `acc`, as one
KDA_DEV float4 scan_join(float4 acc, float4 ab) {
    return make_float4(scan_join_a(acc.x, ab.x), scan_join_a(acc.y, ab.y), scan_fold(ab.x, ab.z, acc.z),
                       scan_fold(ab.y, ab.w, acc.w));
}

// ---- loads
// 16, 8 or 4 bytes, of which `n` are read and the rest zero
KDA_DEV void cp_async16_zfill(uint32_t dst, const void* src, int n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
KDA_DEV void cp_async4_zfill(uint32_t dst, const void* src, int n) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
KDA_DEV void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
KDA_DEV void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// This warp's NT rows of one tensor's tile, token tw the first of them, into `dst` (the
// tile's start in shared memory): tokens outside [t0, t1) and channels from D on become
// zeros, which leave a state as it is.  `width`: bytes of a copy that the tensor's address
// and stride allow (16, 4, or 2: plain loads).
template <bool BF16, int NT>
KDA_DEV void load_rows(uint8_t* dst, const void* base, int64_t ld, int64_t tw, int64_t t0, int64_t t1, int ch0, int D,
                       int width, int warp, int lane) {
    using Geo = ScanGeo<BF16, NT>;
    constexpr int ES = Geo::ES;
    uint8_t* const rows = dst + warp * NT * Geo::ROWB;
    const uint8_t* const src = static_cast<const uint8_t*>(base);
    const bool whole = tw >= t0 && tw + NT <= t1;
    if (width == 16) {
        constexpr int PR = Geo::ROWB / 16;  // pieces of a row
        constexpr int RPI = 32 / PR;        // rows of a warp-wide copy
        const int col = lane % PR, row0 = lane / PR, ch = ch0 + col * (16 / ES);
        const int left = (D - ch) * ES;
        const int n = left < 0 ? 0 : (left > 16 ? 16 : left);
        const uint32_t to = smem_u32(rows) + row0 * Geo::ROWB + col * 16;
        const int64_t step = ld * (RPI * ES);
        const uint8_t* from = src + (tw + row0) * ld * ES + (int64_t)ch * ES;
        if (whole) {
            if (n == 0) from = src;
            const int64_t st = n == 0 ? 0 : step;
#pragma unroll
            for (int i = 0; i < NT / RPI; ++i, from += st) cp_async16_zfill(to + i * RPI * Geo::ROWB, from, n);
        } else {
#pragma unroll
            for (int i = 0; i < NT / RPI; ++i, from += step) {
                const int64_t t = tw + row0 + i * RPI;
                const bool in = n > 0 && t >= t0 && t < t1;
                cp_async16_zfill(to + i * RPI * Geo::ROWB, in ? from : src, in ? n : 0);
            }
        }
    } else if (width == 4) {
        constexpr int PL = Geo::ROWB / 128;  // 4-byte pieces of a row per lane
#pragma unroll 4
        for (int i = 0; i < NT; ++i) {
            const int64_t t = tw + i;
            const bool row_in = t >= t0 && t < t1;
#pragma unroll
            for (int k = 0; k < PL; ++k) {
                const int ch = ch0 + (lane + 32 * k) * (4 / ES);
                const int left = (D - ch) * ES, n = left < 0 ? 0 : (left > 4 ? 4 : left);
                const bool in = row_in && n > 0;
                cp_async4_zfill(smem_u32(rows + i * Geo::ROWB + (lane + 32 * k) * 4),
                                in ? src + ((size_t)t * ld + ch) * ES : src, in ? n : 0);
            }
        }
    } else {
        const uint16_t* const s = reinterpret_cast<const uint16_t*>(src);
        const int ch = ch0 + 2 * lane;
#pragma unroll 8
        for (int i = 0; i < NT; ++i) {
            const int64_t t = tw + i;
            const bool in = t >= t0 && t < t1;
            const uint32_t lo = in && ch < D ? s[(size_t)t * ld + ch] : 0u;
            const uint32_t hi = in && ch + 1 < D ? s[(size_t)t * ld + ch + 1] : 0u;
            *reinterpret_cast<uint32_t*>(rows + i * Geo::ROWB + lane * 4) = lo | hi << 16;
        }
    }
}

// channels 2 lane, 2 lane + 1 of a tile's row
template <bool BF16>
KDA_DEV float2 tile_at(const uint8_t* tile, int row, int lane) {
    if constexpr (BF16) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(tile + row * (SC_CH * 2) + lane * 4);
        return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    } else {
        return *reinterpret_cast<const float2*>(tile + row * (SC_CH * 4) + lane * 8);
    }
}

// Two channels of a row of an output [tokens, D].
KDA_DEV void store2(void* base, bool bf16, size_t row, int D, int ch, float2 v) {
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
KDA_DEV float2 load2(const float* base, size_t row, int D, int ch) {
    const size_t i = row * D + ch;
    return f2(ch < D ? base[i] : 0.f, ch + 1 < D ? base[i + 1] : 0.f);
}

// ---- sequences
// First m in [lo, hi) with cu[m] >= v (hi if there is none); all lanes of a warp.
KDA_DEV int warp_lower_bound(const int32_t* __restrict__ cu, int lo, int hi, int64_t v, int lane) {
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

// The part of the packed tokens that split `s` of `S` walks: whole sequences n0 .. n1 - 1,
// tokens [t0, t1).
struct ScanSpan {
    int n0, n1;
    int64_t t0, t1;
};
KDA_DEV ScanSpan scan_span(const ScanArgs& a, int s, int S, int lane) {
    ScanSpan r;
    if (!a.cu) {
        r.n0 = (int)((int64_t)a.B * s / S);
        r.n1 = (int)((int64_t)a.B * (s + 1) / S);
        r.t0 = (int64_t)r.n0 * a.T;
        r.t1 = (int64_t)r.n1 * a.T;
        return r;
    }
    int64_t end = a.cu[a.n_seqs];
    end = end < 0 ? 0 : (end > a.T ? a.T : end);
    r.n0 = 0, r.n1 = a.n_seqs, r.t0 = 0, r.t1 = end;
    if (s > 0) {
        r.n0 = warp_lower_bound(a.cu, 0, a.n_seqs, end * s / S, lane);
        r.t0 = r.n0 < a.n_seqs ? a.cu[r.n0] : end;
    }
    if (s + 1 < S) {
        r.n1 = warp_lower_bound(a.cu, 0, a.n_seqs, end * (s + 1) / S, lane);
        r.t1 = r.n1 < a.n_seqs ? a.cu[r.n1] : end;
    }
    if (r.t0 < 0) r.t0 = 0;
    if (r.t1 > end) r.t1 = end;
    if (r.t1 < r.t0) r.t1 = r.t0;
    return r;
}

// Where sequences meet among a warp's NT tokens: bit j of `starts` / `ends`: token tw + j is the
// first / last of its sequence; whose numbers are seq_start(j) and seq_end(j) (which a
// cu_seqlens that starts behind 0 can make -1).
template <int NT>
struct ScanBounds {
    uint32_t starts, ends;
    int64_t n;      // equal lengths: sequence of token tw, and tw's place in it
    uint32_t r, T;
    int* tab;       // packed: [2][NT] of this warp: last m with cu[m] = tw + j, first with cu[m] = tw + j + 1
    KDA_DEV int64_t seq_start(int j) const { return tab ? tab[j] : n + (r + j) / T; }
    KDA_DEV int64_t seq_end(int j) const { return tab ? tab[NT + j] - 1 : n + (r + j) / T; }
};

template <int NT>
KDA_DEV ScanBounds<NT> scan_bounds(const ScanArgs& a, const ScanSpan& sp, int64_t tw, int* ptr, int* tab, int lane) {
    ScanBounds<NT> b;
    uint32_t meet = 0;  // bit j: a sequence starts at token tw + j, j = 0 .. NT
    if (!a.cu) {
        b.tab = nullptr;
        if (a.T > 0) {
            b.n = tw / a.T;
            const int64_t r = tw - b.n * a.T, left = a.T - r;
            if (a.T >> 31) {  // a length past 32 bits: at most one meeting point, `left` tokens ahead
                b.r = 0;
                b.T = left > NT ? NT + 1 : (uint32_t)left;
                meet = (r == 0 ? 1u : 0u) | (left <= NT ? 1u << (int)left : 0u);
            } else {
                b.r = (uint32_t)r;
                b.T = (uint32_t)a.T;
                meet = __ballot_sync(0xffffffffu, lane <= NT && (b.r + lane) % b.T == 0);
            }
        }
    } else {
        b.tab = tab;
        const int N1 = a.n_seqs + 1;
        int m = *ptr;
        const int v0 = m + lane < N1 ? a.cu[m + lane] : INT32_MAX;
        const int k = __popc(__ballot_sync(0xffffffffu, v0 < tw));
        m = k < 32 ? m + k : warp_lower_bound(a.cu, m + 32 < N1 ? m + 32 : N1, N1, tw, lane);
        *ptr = m;
        __syncwarp();
        int before = -1;  // the value of the entry before the window
        while (m < N1) {
            const int v = m + lane < N1 ? a.cu[m + lane] : INT32_MAX;
            const int up = __shfl_up_sync(0xffffffffu, v, 1), down = __shfl_down_sync(0xffffffffu, v, 1);
            const bool in = v >= tw && v <= tw + NT;
            const int j = in ? (int)(v - tw) : 0;
            if (in && j < NT && (lane == 31 || down != v)) tab[j] = m + lane;
            if (in && j > 0 && (lane == 0 ? before != v : up != v)) tab[NT + j - 1] = m + lane;
            meet |= __reduce_or_sync(0xffffffffu, in ? 1u << j : 0u);
            before = __shfl_sync(0xffffffffu, v, 31);
            if (__ballot_sync(0xffffffffu, in) != 0xffffffffu) break;
            m += 32;
            __syncwarp();
        }
        __syncwarp();
    }
    // only tokens of [t0, t1)
    uint32_t own = NT < 32 ? (1u << NT) - 1u : 0xffffffffu;
    if (tw < sp.t0) own = sp.t0 - tw >= NT ? 0u : own & ~((1u << (int)(sp.t0 - tw)) - 1u);
    if (tw + NT > sp.t1) own = tw >= sp.t1 ? 0u : own & ((1u << (int)(sp.t1 - tw)) - 1u);
    b.starts = meet & own;
    b.ends = (meet >> 1) & own;
    return b;
}

// ---- clusters
KDA_DEV void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
KDA_DEV void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
KDA_DEV void st_cluster(uint32_t addr, float4 v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}

}  // namespace kda
