// rx_rope.cuh -- angles of the rotary position embedding, shared by the
// kernels that rotate (rx_rope.cu, rx_qk_norm.cu).
//
// Angles: the host tabulates f_c = theta_c / (2 pi) as a 64-bit binary
// fraction of a turn, F_c = f_c 2^64 (f_c < 1).  Then p F_c mod 2^64 is
// p f_c mod 1 in units of 2^-64 turn, exactly as integer arithmetic wraps,
// so the reduction modulo 2 pi is exact up to the table's rounding (about
// 2^-53 of f_c) at any int32 position; its top 32 bits, read as a signed
// number, are the angle in [-pi, pi) in units of 2^-31 pi, which sincosf
// then takes.  Two integer multiplies a pair -- this GPU runs double
// precision at a small fraction of its fp32 and integer rates.
#pragma once

#include <math.h>
#include <stdint.h>

#include "rx_common.cuh"

namespace rx {

constexpr int kMaxHalf = 64;  // head_dim 128

struct RopeTab {
    uint32_t f_hi[kMaxHalf];  // theta_c / (2 pi) as a 64-bit fraction of a turn: high word
    uint32_t f_lo[kMaxHalf];  // low word
};

struct Rot8 {
    float c[8], s[8];
};

// Sine and cosine of |pos| theta_c (the caller gives the sine the sign of pos).
__device__ __forceinline__ void sincos_at(const RopeTab &tab, uint32_t up, int c, float &sn, float &cs)
{
    constexpr float kTurn = 1.4629180792671596e-9f;  // 2 pi / 2^32
    // bits 32 .. 63 of |p| F_c: the high word of |p| f_lo plus the low
    // word of |p| f_hi (the higher words are whole turns)
    const uint32_t t = __umulhi(up, tab.f_lo[c]) + up * tab.f_hi[c];
    const float ar = (float)(int32_t)t * kTurn;  // in [-pi, pi)
    sincosf(ar, &sn, &cs);
}

// The same to about half a place of the result: reduced to an eighth of a turn
// in the integers, the angle held as the sum of two fp32 values (sincos_at's
// has up to 2^-23 of absolute error near half a turn), then by the Taylor
// series: on [-pi/4, pi/4] the first term left out is below 2^-29.
__device__ __forceinline__ void sincos_exact(const RopeTab &tab, uint32_t up, int c, float &sn, float &cs)
{
    constexpr float kTurn = 1.4629180792671596e-9f;  // 2 pi / 2^32, and what its rounding left
    constexpr float kTurnLow = (float)(1.4629180792671596e-9 - (double)1.4629180792671596e-9f);
    const uint32_t t = __umulhi(up, tab.f_lo[c]) + up * tab.f_hi[c];
    const uint32_t quarter = (t + 0x20000000u) >> 30;  // nearest quarter turn
    const int32_t rest = (int32_t)(t - (quarter << 30));
    const float top = (float)rest, low = (float)(rest - (int32_t)top);
    const float x = __fmul_rn(top, kTurn);
    const float e = fmaf(low, kTurn, fmaf(top, kTurnLow, fmaf(top, kTurn, -x)));  // the angle is x + e
    const float x2 = x * x;
    float s = fmaf(x2, 1.f / 362880.f, -1.f / 5040.f);
    s = fmaf(x2, s, 1.f / 120.f);
    s = fmaf(x2, s, -1.f / 6.f);
    s = x + fmaf(x * x2, s, fmaf(-.5f * x2, e, e));
    float k = fmaf(x2, -1.f / 3628800.f, 1.f / 40320.f);
    k = fmaf(x2, k, -1.f / 720.f);
    k = fmaf(x2, k, 1.f / 24.f);
    // 1 - x^2 / 2 and what its rounding left
    const float h = fmaf(-.5f, x2, 1.f), left = fmaf(-.5f, x2, 1.f - h);
    k = h + fmaf(x2 * x2, k, fmaf(-x, e, left));
    // a quarter turn: (cos, sin) -> (-sin, cos)
    const float a = quarter & 1u ? k : s, b = quarter & 1u ? s : k;
    sn = quarter & 2u ? -a : a;
    cs = (quarter + 1u) & 2u ? -b : b;
}

__device__ __forceinline__ Rot8 angles(const RopeTab &tab, int32_t pos, int c0)
{
    // |p|, and the sine's sign: a rotation by -a is the one by a with sin negated
    const uint32_t up = pos < 0 ? 0u - (uint32_t)pos : (uint32_t)pos;
    const float sgn = pos < 0 ? -1.f : 1.f;
    Rot8 r;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        sincos_at(tab, up, c0 + k, r.s[k], r.c[k]);
        r.s[k] *= sgn;
    }
    return r;
}

inline bool make_tab(int D, double base, RopeTab &tab)
{
    if ((D != 64 && D != 128) || !(base > 1.0)) return false;
    constexpr double kTwoPi = 6.283185307179586476925286766559;
    for (int c = 0; c < D / 2; ++c) {
        // f_c < 1 / (2 pi): f_c 2^64 < 2^62, converted exactly from the double
        const double f = pow(base, -2.0 * c / D) / kTwoPi;
        const uint64_t F = (uint64_t)ldexp(f, 64);
        tab.f_hi[c] = (uint32_t)(F >> 32);
        tab.f_lo[c] = (uint32_t)F;
    }
    return true;
}

}  // namespace rx
