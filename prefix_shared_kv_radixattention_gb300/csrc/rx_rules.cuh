// rx_rules.cuh -- rules on attention scores, shared by the kernels that apply
// them (rx_extend.cu, rx_tree.cuh): a tanh cap, a bias that falls with the
// distance, and the positions a query token sees.
//
// A score s = sm_scale q . k of the query token at position p and the key at
// position j becomes
//     x = cap tanh(s / cap) - slope[h] |p - j|
// where lo <= j < hi, and takes no part elsewhere.  In log2 units, with
// E = 2^(2 log2(e) s / cap):
//     log2(e) cap tanh(s / cap) = c2 - 2 c2 / (1 + E),   c2 = cap log2(e),
// an exponential and a reciprocal of the special-function units a score (E of 0
// or infinity gives -c2 and c2), or, where every score that a warp's rows see of a
// tile is within the cap, a polynomial of degree 13 on the multiply-add units, within
// 3/8 of the cap one of degree 7: the special-function units are what a tile waits for
// otherwise.  The first way is off by c2 times a few 2^-23 (a cap of 50: under 3e-5
// log2 units, a weight's relative error under 2^-15, where the weights are rounded
// to bf16 for the product with V), the polynomials' fits by 2^-25 and 2^-26 of c2 and
// what fp32 makes of them by no more than 2^-21 of the score, so that a large cap
// costs nothing; a fixed base (below) takes another 2^-18 log2 units, half a step of
// x - m, or 2^-24 of c2.
// (tanh.approx is off by 2^-11 of its value: 0.03 log2 units at that cap.)
//
// A cap bounds the scores, so the softmax needs no running maximum: with
// |x| <= c2 and a key near enough in every row (no bias), the weights
// 2^(x - m) with the one base m = min(c2, 100 - c2) neither overflow nor, for a
// row's largest, fall below 2^-100; the maximum of a tile, the wait on it and
// the rescaling of O all go.  That is done for c2 <= 72.2 (caps up to 50: the
// largest weight is 2^45, and V may reach 2^57 before sums overflow).  Larger
// caps and biased scores keep the running maximum.
#pragma once

#include <math.h>

#include "rx_common.cuh"

namespace rx {

struct Rules {
    float c2;               // cap log2(e); 0: scores are not capped
    float to_e;             // 2 / cap: E = 2^(s sl2 to_e)
    float base;             // the weights' base, where it is fixed
    int fixed;              // the base is fixed
    float poly[7];          // c2 tanh y = y (poly[0] + poly[1] y^2 + ...), |y| <= 1
    float to_y;             // y = s / cap from log2 units
    // in units of the products x = q . k, for |x| up to near_to, 3/8 of the cap (0:
    // out of fp32's range): c2 tanh = x (near[0] + near[1] x^2 + ... + near[3] x^6)
    float near_to;
    float near[4];
    int window;             // a token sees positions above p - window; INT_MAX: all
    const float *slope;     // [q heads] or null
    const int32_t *see_from;  // [query tokens] or null
    const int32_t *see_to;    // [query tokens] or null
};

__device__ __forceinline__ float fast_rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}

// First position that a token at p sees by the window alone.
__device__ __forceinline__ int window_from(const Rules &r, int p) { return p >= r.window ? p - r.window + 1 : 0; }

// The positions [lo, hi) that query token `tok` (its row of see_from and
// see_to) at position p sees, of a context of `ctx` positions.
__device__ __forceinline__ void seen_range(const Rules &r, int tok, int p, int ctx, int &lo, int &hi)
{
    lo = window_from(r, p);
    hi = p + 1;
    if (r.see_from) lo = max(lo, __ldg(r.see_from + tok));
    if (r.see_to) hi = max(hi, min(__ldg(r.see_to + tok), ctx));
}

// What a kernel is built for: no cap and no bias; a cap with the fixed base;
// whatever else.
enum { kNoRules = 0, kRange = 1, kFixedCap = 2, kAnyRules = 3 };
inline int rules_kind(const Rules &r) { return r.fixed ? kFixedCap : r.c2 > 0.f || r.slope ? kAnyRules : kRange; }

// Which of 32 keys are among from .. to - 1, a bit each.  The words are made where
// they are used (two comparisons a key: a windowed prompt 258 us in place of 233;
// the words kept from the cap to the hiding: 64 tokens on 8,192 with a cap of 30,
// 109 us in place of 103).
__device__ __forceinline__ uint32_t among(int from, int to)
{
    return __funnelshift_lc(0u, ~0u, max(from, 0)) & ~__funnelshift_lc(0u, ~0u, max(to, 0));
}

// The scores of a tile's other keys become X (bits).
template <uint32_t X, int N>
__device__ __forceinline__ void hide(uint32_t (&sv)[N], int from, int to)
{
#pragma unroll
    for (int i = 0; i < N / 32; ++i) {
        const uint32_t seen = among(from - 32 * i, to - 32 * i);
#pragma unroll
        for (int k = 0; k < 32; ++k)
            if (!((seen >> k) & 1u)) sv[32 * i + k] = X;
    }
}

// N scores q . k of consecutive keys, the first at position kbase, in place: to
// log2 units (times sl2) with the cap and the bias, less the fixed base where
// there is one.  dist = p - kbase; slope in log2 units a position.  Scores that
// have neither cap nor bias stay as they are; the result is what the scores are
// still to be multiplied with.  SAME: sl2 is the call's, not the row's own; valid:
// the row is one (others hold anything).  masked: some row of the warp does not
// see all of the keys; this one sees from .. to - 1 of them, and the others'
// scores, which may be anything, take no part in the choice of the cap's form.
// They are for the caller to hide.
template <int KIND, bool SAME, int N>
__device__ __forceinline__ float apply_rules(uint32_t (&sv)[N], const Rules &r, float sl2, float slope, int dist, bool valid,
                                             bool masked, int from, int to)
{
    if constexpr (KIND == kRange) return sl2;
    if (KIND == kFixedCap || r.c2 > 0.f) {
        const float ky = fminf(sl2 * r.to_y, 0x1.fffffep127f);
        float a0 = 0.f, a1 = 0.f;
        // hidden scores are written over, or the maximum is taken again over the others
        // (long chat, a cap of 50, 1,437 us and 1,476; a cap of 60, 1,870 and 1,833; 64 tokens
        // on 8,192, a cap of 30, with 128 keys a thread, 109 and 102)
        constexpr bool kOver = KIND == kFixedCap && N <= 64;
        if (kOver && masked) hide<0u>(sv, from, to);
#pragma unroll
        for (int k = 0; k < N / 4; ++k) {
            a0 = fmax3(a0, fabsf(__uint_as_float(sv[4 * k])), fabsf(__uint_as_float(sv[4 * k + 1])));
            a1 = fmax3(a1, fabsf(__uint_as_float(sv[4 * k + 2])), fabsf(__uint_as_float(sv[4 * k + 3])));
        }
        if (!kOver && masked) {
            a0 = a1 = 0.f;
#pragma unroll
            for (int i = 0; i < N / 32; ++i) {
                const uint32_t seen = among(from - 32 * i, to - 32 * i);
#pragma unroll
                for (int k = 0; k < 32; k += 2) {
                    if ((seen >> k) & 1u) a0 = fmaxf(a0, fabsf(__uint_as_float(sv[32 * i + k])));
                    if ((seen >> k) & 2u) a1 = fmaxf(a1, fabsf(__uint_as_float(sv[32 * i + k + 1])));
                }
            }
        }
        const float most = valid ? fmaxf(a0, a1) : 0.f;
        if (SAME && __all_sync(0xffffffffu, most <= r.near_to)) {
            uint64_t c[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) c[i] = f2(r.near[i], r.near[i]);
            const uint64_t base2 = f2(-r.base, -r.base);
#pragma unroll
            for (int k = 0; k < N / 2; ++k) {
                const uint64_t s = f2(__uint_as_float(sv[2 * k]), __uint_as_float(sv[2 * k + 1])), z = f2_mul(s, s);
                uint64_t x = f2_fma(c[3], z, c[2]);
                x = f2_fma(x, z, c[1]);
                x = f2_fma(x, z, c[0]);
                float a, b;
                f2_split(f2_fma(x, s, base2), a, b);
                sv[2 * k] = __float_as_uint(a);
                sv[2 * k + 1] = __float_as_uint(b);
            }
        } else if (__all_sync(0xffffffffu, most * ky <= 1.f)) {
            uint64_t c[7];
#pragma unroll
            for (int i = 0; i < 7; ++i) c[i] = f2(r.poly[i], r.poly[i]);
            const uint64_t base2 = f2(-r.base, -r.base), ky2 = f2(ky, ky);
#pragma unroll
            for (int k = 0; k < N / 2; ++k) {
                const uint64_t y = f2_mul(f2(__uint_as_float(sv[2 * k]), __uint_as_float(sv[2 * k + 1])), ky2), z = f2_mul(y, y);
                uint64_t x = f2_fma(c[6], z, c[5]);
#pragma unroll
                for (int i = 4; i >= 0; --i) x = f2_fma(x, z, c[i]);
                float a, b;
                f2_split(f2_fma(x, y, base2), a, b);
                sv[2 * k] = __float_as_uint(a);
                sv[2 * k + 1] = __float_as_uint(b);
            }
        } else {
            const float ke = fminf(sl2 * r.to_e, 0x1.fffffep127f), top = r.c2 - r.base;
            const uint64_t ke2 = f2(ke, ke), one2 = f2(1.f, 1.f), minus2 = f2(-2.f * r.c2, -2.f * r.c2), top2 = f2(top, top);
#pragma unroll
            for (int k = 0; k < N / 2; ++k) {
                float a, b;
                f2_split(f2_mul(f2(__uint_as_float(sv[2 * k]), __uint_as_float(sv[2 * k + 1])), ke2), a, b);
                f2_split(f2_add(f2(fast_exp2(a), fast_exp2(b)), one2), a, b);
                f2_split(f2_fma(f2(fast_rcp(a), fast_rcp(b)), minus2, top2), a, b);
                sv[2 * k] = __float_as_uint(a);
                sv[2 * k + 1] = __float_as_uint(b);
            }
        }
        if (KIND == kFixedCap || !r.slope) return 1.f;
    } else if (!r.slope) {
        return sl2;
    }
    const float scale = r.c2 > 0.f ? 1.f : sl2, far = (float)dist;
#pragma unroll
    for (int k = 0; k < N; ++k)
        sv[k] = __float_as_uint(fmaf(-slope, fabsf(far - (float)k), scale * __uint_as_float(sv[k])));
    return 1.f;
}

// Checks a call's rules and fills in what the kernels take; `who` names the
// entry point.  scale_log2: log2 units of a score.
inline int make_rules(const char *who, const rx_attn_rules *in, float scale_log2, Rules &r)
{
    r = Rules{};
    r.window = INT32_MAX;
    if (!in) return rx_set_error(RX_ERR_INVALID, "%s: no rules (use the call without them)", who);
    if (!(in->cap >= 0.f) || in->window < 0 || ((reinterpret_cast<uintptr_t>(in->slope) | reinterpret_cast<uintptr_t>(in->see_from) |
                                                 reinterpret_cast<uintptr_t>(in->see_to)) & 3) != 0)
        return rx_set_error(RX_ERR_INVALID, "%s: cap %g and window %d must not be negative, and the rules' arrays 4-byte aligned",
                            who, in->cap, in->window);
    // a hidden score is -infinity, and 0 times it would be NaN
    if (!(scale_log2 >= 0x1p-126f && scale_log2 < INFINITY))
        return rx_set_error(RX_ERR_INVALID, "%s: sm_scale (times K's scale) outside fp32's normal range", who);
    r.slope = in->slope;
    r.see_from = in->see_from;
    r.see_to = in->see_to;
    if (in->window > 0) r.window = in->window;
    if (in->cap > 0.f) {
        r.c2 = in->cap * kLog2e;
        r.to_e = 2.f / in->cap;
        const float ke = scale_log2 * r.to_e;
        if (!(in->cap >= 1e-3f && in->cap <= 1e6f) || !(ke >= 0x1p-126f && ke < INFINITY))
            return rx_set_error(RX_ERR_UNSUPPORTED, "%s: cap %g (from 1e-3 to 1e6)", who, in->cap);
        // tanh y = y P(y^2) for |y| <= 1, off by at most 2.6e-8 as rounded here (least maximum, found by
        // reweighted least squares, 2.0e-8 before the rounding; degree 11, off by 2.4e-7, left a log-sum-exp off by 1e-6 of itself)
        static const float P[7] = {0.999999693f, -0.333321293f, 0.133195837f, -0.0532658349f, 0.0199732818f, -0.00595127971f, 0.000963771925f};
        for (int i = 0; i < 7; ++i) r.poly[i] = P[i] * r.c2;
        r.to_y = 1.f / r.c2;
        // the same for |y| <= 3/8, off by at most 1.1e-8
        static const double Q[4] = {0.99999974, -0.333308399, 0.132683921, -0.0476184644};
        const double k1 = (double)scale_log2 / r.c2;
        double c = (double)r.c2 * k1;
        r.near_to = (float)fmin(0.375 / k1, 1e18);
        for (int i = 0; i < 4; ++i, c *= k1 * k1) {
            r.near[i] = (float)(Q[i] * c);
            if (!(fabs(Q[i] * c) > 2e-38 && fabs(Q[i] * c) < 1e18)) r.near_to = 0.f;
        }
        if (r.c2 <= 72.2f && !in->slope) {
            r.fixed = 1;
            r.base = fminf(r.c2, 100.f - r.c2);
        }
    }
    return RX_OK;
}

}  // namespace rx
