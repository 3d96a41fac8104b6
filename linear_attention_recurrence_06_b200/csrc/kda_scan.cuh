// kda_scan.cuh -- the arithmetic of one token and channel of the element-wise
// gated scan (include/kda.h, kda_scan_fwd), shared by its kernels.
#pragma once
#include "kda_sm100.cuh"

namespace kda {

// A decay a = e^l, l <= 0, in one register: `p` holds a - 1 (sign bit set, -0 for
// l = 0) where l > -1/4, else a itself (sign bit clear).  h + (a - 1) h keeps a
// state's slow decay to the precision of a - 1, where rounding a itself would
// change the decay rate by up to 2^-24 / |l|; a h keeps what a large decay
// leaves of a state, and forgets it exactly at a = 0.
constexpr float SCAN_SLOW = -0.25f;

struct ScanTerm {
    float p;  // the decay, as above
    float u;  // w s x
};

// The hardware's approximations without their denormal handling (results below 2^-126 are 0).
KDA_DEV float ex2_ftz(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
KDA_DEV float rcp_ftz(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
KDA_DEV float rsqrt_ftz(float x) {
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
constexpr float LOG2E = 1.4426950408889634f;
KDA_DEV float exp_ftz(float x) { return ex2_ftz(x * LOG2E); }

// l = min(log_alpha, 0), NaN kept
KDA_DEV float scan_clamp(float log_alpha) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(log_alpha), "f"(0.f));
    return r;
}

KDA_DEV float scan_decay(float l) {
    // e^l - 1 for l in (-1/4, 0]: its Taylor polynomial to l^6 (the next term is
    // below 2^-24 of the sum there)
    float t = fmaf(l, 1.f / 720.f, 1.f / 120.f);
    t = fmaf(t, l, 1.f / 24.f);
    t = fmaf(t, l, 1.f / 6.f);
    t = fmaf(t, l, 0.5f);
    const float em = fmaf(t * l, l, l);
    const float e = exp_ftz(l);
    return l > SCAN_SLOW ? __uint_as_float(__float_as_uint(em) | 0x80000000u) : e;
}

KDA_DEV bool scan_slow(float p) { return __float_as_int(p) < 0; }
KDA_DEV float scan_a(float p) { return scan_slow(p) ? 1.f + p : p; }
// a h + u
KDA_DEV float scan_step(float p, float h, float u) {
    const float keep = __uint_as_float(__float_as_uint(h) & (uint32_t)(__float_as_int(p) >> 31));  // h or 0
    return fmaf(p, h, u) + keep;
}
// 1 - a^2
KDA_DEV float scan_one_minus_a2(float p) { return fmaf(-p, p, scan_slow(p) ? -2.f * p : 1.f); }

constexpr float SCAN_TINY = 1e-37f;  // keeps sqrt(n) = n rsqrt(n), n = 1 - a^2, a number at n = 0

template <bool GATE, bool NORM>
KDA_DEV ScanTerm scan_term(float x, float log_alpha, float g) {
    ScanTerm r;
    r.p = scan_decay(scan_clamp(log_alpha));
    float ws = GATE ? rcp_ftz(1.f + exp_ftz(-g)) : 1.f;
    if (NORM) {
        const float n = scan_one_minus_a2(r.p);
        ws *= n * rsqrt_ftz(fmaxf(n, SCAN_TINY));
    }
    r.u = ws * x;
    return r;
}

// Tokens [first, end) of sequence n: cu (clamped into [0, T]) or n * T.
KDA_DEV void scan_range(const int32_t* cu, int n, int64_t T, int64_t* first, int64_t* end) {
    if (cu) {
        const int64_t a = cu[n], b = cu[n + 1];
        *first = a < 0 ? 0 : (a > T ? T : a);
        *end = b > T ? T : (b < *first ? *first : b);
    } else {
        *first = (int64_t)n * T;
        *end = *first + T;
    }
}

}  // namespace kda
