// rx_qk_norm.cu -- RMS norm of each q and k head, rotary embedding and slot
// scatter in one pass over a token's projected row.
//
// For every q and k head x of token i (d values) with weight w:
//     r  = 1 / sqrt(sum_c x[c]^2 / d + eps),   y[c] = x[c] r w[c]
//     y'[c]       = y[c] cos a - y[c + d/2] sin a
//     y'[c + d/2] = y[c + d/2] cos a + y[c] sin a,    a = pos theta_c, c < d/2
// in fp32, rounded once: to bf16 for q and a bf16 pool, to E4M3 (after the
// division by the pool's scale) for an FP8 pool.  V rows pass through.
//
// The floor is one read of the projected row and one write of its results:
// the separate norm, rotation and store move q and k three times.
//
// Layout: a head is d / 16 lanes, each holding eight pairs (x[c0 .. c0 + 7]
// and x[c0 + d/2 .. + 7]): both members of a pair in one thread, the sum of
// squares three shuffles at d 128, all accesses 16 bytes and coalesced.  A
// CTA takes `tok` tokens; their angles are formed once, one sine and cosine
// a thread, into shared memory (a head's own lanes forming them would
// compute each for every head), while the first rows are in flight.
//
// Bound by memory where the batch is long: 16,384 tokens of 64 q and 8 kv
// heads of 128, 671 MB, take 105 us (6.4 TB/s), 4,099 of 32/8 into an FP8
// pool 22 us (92 MB in less than two waves of CTAs).  It was bound by
// instructions before that: 397 a row of a warp, of which the general
// division, sincosf and the unpacked arithmetic were two thirds.  Two rows a
// thread in flight at four CTAs an SM; four rows and two CTAs take 115 and
// 28 us, one row and four 117 and 23.  Rows that do not fill a CTA's passes
// (two tokens of 80 rows on passes of 128) took 156 us.
//
// With positions on several axes (rx_qk_rope_axes_store) only the angles differ: a
// pair's position comes from its axis.  16,384 tokens of 64/8 heads on three axes
// and the norm take 110 us.
#include <numeric>
#include <type_traits>

#include "rx_common.cuh"
#include "rx_rope.cuh"

namespace {

using bf16 = __nv_bfloat16;

constexpr int kThreads = 256;
constexpr int kMaxTok = 16;   // tokens of one CTA
constexpr int kUnroll = 2;    // rows a thread has in flight

struct NormParams {
    const bf16 *q;
    int64_t q_stride;
    bf16 *q_out;
    const bf16 *k_new;
    const bf16 *v_new;
    int64_t kv_stride;
    const bf16 *qw;
    const bf16 *kw;
    const int32_t *slots;
    const int32_t *pos;
    int64_t n;
    int hq, hkv, tok;
    float eps;
    void *k_pool;
    void *v_pool;
    int64_t num_slots;
    float k_scale, v_scale, k_inv, v_inv;  // the inverses correctly rounded
    int32_t *status;
    rx::RopeTab tab;
    // positions on several axes (rx_qk_rope_axes_store): pair c of token i is
    // turned by pos[axis[c] * pos_stride + i]
    int64_t pos_stride;
    int norm;  // 0: no norm
    uint8_t axis[rx::kMaxHalf];
};

// Two fp32 values in one 64-bit register: this GPU's packed multiply-adds take
// one instruction for both, each rounded as the plain one.
struct F2 {
    uint64_t v;
    __device__ __forceinline__ F2() {}
    __device__ __forceinline__ F2(float a, float b) { asm("mov.b64 %0, {%1, %2};\n" : "=l"(v) : "f"(a), "f"(b)); }
    __device__ __forceinline__ void split(float &a, float &b) const { asm("mov.b64 {%0, %1}, %2;\n" : "=f"(a), "=f"(b) : "l"(v)); }
};

__device__ __forceinline__ F2 mul(F2 a, F2 b)
{
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

__device__ __forceinline__ void widen(const uint4 &v, F2 (&x)[4])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = F2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u));
}

__device__ __forceinline__ uint4 narrow(const F2 (&x)[4])
{
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float a, b;
        x[k].split(a, b);
        w[k] = rx::pack_bf16(a, b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Out of line: hardly ever called.
__device__ __noinline__ float divide_any(float x, float y) { return __fdiv_rn(x, y); }

// Eight fp32 values as E4M3 codes of value / scale: a correctly rounded
// division, then the nearest code, magnitudes past 448 saturated.
//
// plain: 2^-60 <= scale <= 2^60 and no magnitude above 2^40.  Then with inv,
// 1 / scale correctly rounded, the first step's quotient is within one place
// and the second rounds it correctly (Markstein, IBM J. Res. Dev. 34, 1990):
// nothing overflows, and what underflows is far below the least code.
__device__ __forceinline__ uint2 codes(F2 (&x)[4], float scale, float inv, bool plain)
{
    const F2 s(scale, scale), i(inv, inv), minus(-1.f, -1.f), ni(-inv, -inv);
    uint16_t pair[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float lo, hi;
        if (plain) {
            const F2 nx = mul(x[k], minus);
            F2 y = mul(x[k], i);
            y = fma(fma(y, s, nx), ni, y);
            y = fma(fma(y, s, nx), ni, y);
            y.split(lo, hi);
        } else {
            x[k].split(lo, hi);
            lo = divide_any(lo, scale);
            hi = divide_any(hi, scale);
        }
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(pair[k]) : "f"(hi), "f"(lo));
    }
    return make_uint2((uint32_t)pair[0] | ((uint32_t)pair[1] << 16), (uint32_t)pair[2] | ((uint32_t)pair[3] << 16));
}

// 1 / sqrt(v): the hardware's approximation and a Newton step, whose v r^2 is
// held to more than 32 bits.
__device__ __forceinline__ float inverse_root(float v)
{
    const float r = rsqrtf(v);
    if (!(r > 0.f && r < INFINITY)) return r;
    const float p = __fmul_rn(v, r), low = __fmaf_rn(v, r, -p);
    return fmaf(.5f * r, fmaf(-low, r, __fmaf_rn(-p, r, 1.f)), r);
}

// AX: positions on several axes, the norm only where the call asks for it.
template <int D, bool F8, bool AX>
__global__ void __launch_bounds__(kThreads, 4) qk_norm_rope_store_kernel(const __grid_constant__ NormParams p)
{
    constexpr int LPR = D / 16;             // lanes of one head
    constexpr int RPP = kThreads / LPR;     // heads of one pass of the CTA
    constexpr int HALF = D / 2;
    using Chunk = std::conditional_t<F8, uint2, uint4>;  // 8 values of the pool
    // columns 2j, 2j + 1 of lane gi: {cos, cos, sin, sin} at [token][j][gi], and
    // the weights of q and k, of columns 4j .. 4j + 3 of a lane's two octets, so
    // that the lanes of a head read consecutive 16-byte words
    __shared__ float4 cs[kMaxTok][4][LPR];
    __shared__ float4 weight[2][2][2][LPR];
    const int gi = threadIdx.x % LPR, sub = threadIdx.x / LPR;
    const int64_t t0 = (int64_t)blockIdx.x * p.tok;
    const int ntok = (int)min((int64_t)p.tok, p.n - t0);
    const int R = p.hq + 2 * p.hkv;
    const int step_t = RPP / R, step_h = RPP - step_t * R;  // token and head of the next row of a thread
    auto advance = [&](int &tt, int &h) {
        tt += step_t;
        h += step_h;
        if (h >= R) {
            h -= R;
            ++tt;
        }
    };

    uint4 lo[kUnroll], hi[kUnroll];
    int lt = sub / R, lh = sub - lt * R;  // of the next row to load
    auto load = [&]() {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            lo[u] = hi[u] = make_uint4(0, 0, 0, 0);
            if (lt < ntok) {
                const bf16 *src = lh < p.hq            ? p.q + (t0 + lt) * p.q_stride + lh * D
                                  : lh < p.hq + p.hkv ? p.k_new + (t0 + lt) * p.kv_stride + (lh - p.hq) * D
                                                      : p.v_new + (t0 + lt) * p.kv_stride + (lh - p.hq - p.hkv) * D;
                // plain loads: q_out may be q
                lo[u] = *reinterpret_cast<const uint4 *>(src + gi * 8);
                hi[u] = *reinterpret_cast<const uint4 *>(src + HALF + gi * 8);
            }
            advance(lt, lh);
        }
    };
    int tt = lt, h = lh;  // of the next row to work off
    load();

    for (int i = threadIdx.x; i < ntok * HALF; i += kThreads) {
        const int t = i / HALF, c = i % HALF;
        const int32_t pos = __ldg(p.pos + (AX ? p.axis[c] * p.pos_stride : 0) + t0 + t);
        const uint32_t up = pos < 0 ? 0u - (uint32_t)pos : (uint32_t)pos;
        float sn, cn;
        rx::sincos_exact(p.tab, up, c, sn, cn);
        float *dst = reinterpret_cast<float *>(&cs[t][(c % 8) / 2][c / 8]) + c % 2;
        dst[0] = cn;
        dst[2] = pos < 0 ? -sn : sn;
    }
    bool small = true;
    if (threadIdx.x < 2 * D) {
        const int c = threadIdx.x % D;
        const bf16 *w = threadIdx.x < D ? p.qw : p.kw;
        const float f = w ? __bfloat162float(w[c]) : 1.f;
        small = fabsf(f) <= 0x1p30f;
        reinterpret_cast<float *>(&weight[threadIdx.x / D][c / HALF][c % 8 / 4][c % HALF / 8])[c % 4] = f;
    }
    // a normalised value is at most sqrt(D), a rotated one sqrt(2) times that:
    // below 2^40 with weights up to 2^30
    small = __syncthreads_and(small);

    for (int left = ntok * R; left > 0; left -= RPP * kUnroll) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            F2 a[4], b[4];
            widen(lo[u], a);
            widen(hi[u], b);
            F2 sq(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < 4; ++k) sq = fma(a[k], a[k], fma(b[k], b[k], sq));
            float ss, odd;
            sq.split(ss, odd);
            ss += odd;
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const int t = tt, hh = h;
            advance(tt, h);
            if (t >= ntok) continue;
            const bool is_q = hh < p.hq, is_v = hh >= p.hq + p.hkv;
            if (!is_v) {
                const float r = AX && !p.norm ? 1.f : inverse_root(ss * (1.f / D) + p.eps);
                const F2 rr(r, r), minus(-1.f, -1.f);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 q = cs[t][j][gi], wa = weight[is_q ? 0 : 1][0][j / 2][gi], wb = weight[is_q ? 0 : 1][1][j / 2][gi];
                    const F2 c(q.x, q.y), s(q.z, q.w);
                    const F2 x = mul(mul(a[j], rr), j % 2 ? F2(wa.z, wa.w) : F2(wa.x, wa.y));
                    const F2 y = mul(mul(b[j], rr), j % 2 ? F2(wb.z, wb.w) : F2(wb.x, wb.y));
                    a[j] = fma(x, c, mul(mul(y, s), minus));
                    b[j] = fma(y, c, mul(x, s));
                }
            }
            if (is_q) {
                bf16 *dst = p.q_out + ((t0 + t) * p.hq + hh) * D;
                *reinterpret_cast<uint4 *>(dst + gi * 8) = narrow(a);
                *reinterpret_cast<uint4 *>(dst + HALF + gi * 8) = narrow(b);
                continue;
            }
            const int32_t slot = __ldg(p.slots + t0 + t);
            if (slot < 0 || (int64_t)slot >= p.num_slots) {
                if (p.status && hh == p.hq && gi == 0) atomicOr(p.status, RX_DEV_BAD_SLOT);
                continue;
            }
            const int g = hh - p.hq - (is_v ? p.hkv : 0);
            Chunk *dst = static_cast<Chunk *>(is_v ? p.v_pool : p.k_pool) + ((int64_t)slot * p.hkv + g) * (D / 8);
            if constexpr (F8) {
                const float scale = is_v ? p.v_scale : p.k_scale, inv = is_v ? p.v_inv : p.k_inv;
                // without a norm a rotated value is at most sqrt(2) times the head's largest
                const bool plain = scale >= 0x1p-60f && scale <= 0x1p60f &&
                                   (is_v ? ss <= 0x1p80f : AX && !p.norm ? ss <= 0x1p78f : small);
                dst[gi] = codes(a, scale, inv, plain);
                dst[LPR + gi] = codes(b, scale, inv, plain);
            } else {
                dst[gi] = is_v ? lo[u] : narrow(a);
                dst[LPR + gi] = is_v ? hi[u] : narrow(b);
            }
        }
        if (left > RPP * kUnroll) load();
    }
}

struct Pool {
    void *k, *v;
    int64_t num_slots;
    int hkv, D;
    bool f8;
    float k_scale, v_scale;
};

// Positions on several axes, and whether there is a norm.
struct Axes {
    int64_t stride;
    int n;
    const uint8_t *pair;
    int norm;
};

int norm_call(const char *who, const Pool &pool, const void *q, int64_t q_stride, void *q_out, const void *k_new,
              const void *v_new, int64_t kv_stride, const void *qw, const void *kw, const int32_t *slots,
              const int32_t *pos, int64_t n, int32_t hq, double base, float eps, int32_t *dev_status, void *stream,
              const Axes *axes = nullptr)
{
    if (axes && !axes->norm) eps = 0.f;
    if (n < 0 || hq < 0 || !(eps >= 0.f) || eps > 3.4e38f ||
        (n > 0 && (!k_new || !v_new || !slots || !pos || (hq > 0 && (!q || !q_out)))))
        return rx_set_error(RX_ERR_INVALID, "%s: invalid argument", who);
    if (pool.D != 64 && pool.D != 128)
        return rx_set_error(RX_ERR_UNSUPPORTED, "%s: head_dim %d (supported: 64, 128)", who, pool.D);
    if (!(base > 1.0)) return rx_set_error(RX_ERR_UNSUPPORTED, "%s: base %g (need base > 1)", who, base);
    if (kv_stride % 8 != 0 || kv_stride < (int64_t)pool.hkv * pool.D ||
        (hq > 0 && (q_stride % 8 != 0 || q_stride < (int64_t)hq * pool.D)))
        return rx_set_error(RX_ERR_INVALID, "%s: row strides must be multiples of 8 and hold the row", who);
    const uintptr_t pool_align = pool.f8 ? 7 : 15;
    if ((reinterpret_cast<uintptr_t>(pool.k) & pool_align) != 0 ||
        (reinterpret_cast<uintptr_t>(pool.v) & pool_align) != 0 || rx_misaligned16(q) || rx_misaligned16(q_out) ||
        rx_misaligned16(k_new) || rx_misaligned16(v_new) || rx_misaligned16(qw) || rx_misaligned16(kw))
        return rx_set_error(RX_ERR_INVALID, "%s: pools must be %d-byte and the other tensors 16-byte aligned", who,
                            (int)pool_align + 1);
    if (hq > 0 && q_out == q && q_stride != (int64_t)hq * pool.D)
        return rx_set_error(RX_ERR_INVALID, "%s: q_out may be q only when q's rows are contiguous", who);
    if ((int64_t)hq + 2 * (int64_t)pool.hkv > 65535)
        return rx_set_error(RX_ERR_UNSUPPORTED, "%s: %d q heads and %d kv heads", who, hq, pool.hkv);
    if (axes) {
        if (axes->n < 1 || axes->n > 8)
            return rx_set_error(RX_ERR_UNSUPPORTED, "%s: %d axes (1 to 8)", who, axes->n);
        if (!axes->pair || (axes->n > 1 && axes->stride < n) || (!axes->norm && (qw || kw)))
            return rx_set_error(RX_ERR_INVALID, "%s: pair_axis missing, pos_stride below n, or weights without a norm", who);
        for (int c = 0; c < pool.D / 2; ++c)
            if (axes->pair[c] >= axes->n)
                return rx_set_error(RX_ERR_INVALID, "%s: pair %d on axis %d of %d", who, c, axes->pair[c], axes->n);
    }
    if (n == 0) return RX_OK;
    // the frequency table of the last (head_dim, base) of this thread: a
    // model calls with one base, and 64 powers cost more host time than the launch
    static thread_local rx::RopeTab tab;
    static thread_local int tab_D = 0;
    static thread_local double tab_base = 0;
    if (tab_D != pool.D || tab_base != base) {
        rx::make_tab(pool.D, base, tab);
        tab_D = pool.D;
        tab_base = base;
    }
    NormParams p{};
    p.q = (const bf16 *)q;
    p.q_stride = q_stride;
    p.q_out = (bf16 *)q_out;
    p.k_new = (const bf16 *)k_new;
    p.v_new = (const bf16 *)v_new;
    p.kv_stride = kv_stride;
    p.qw = (const bf16 *)qw;
    p.kw = (const bf16 *)kw;
    p.slots = slots;
    p.pos = pos;
    p.n = n;
    p.hq = hq;
    p.hkv = pool.hkv;
    p.eps = eps;
    p.k_pool = pool.k;
    p.v_pool = pool.v;
    p.num_slots = pool.num_slots;
    p.k_scale = pool.k_scale;
    p.v_scale = pool.v_scale;
    p.k_inv = 1.f / pool.k_scale;
    p.v_inv = 1.f / pool.v_scale;
    p.status = dev_status;
    p.tab = tab;
    if (axes) {
        p.pos_stride = axes->stride;
        p.norm = axes->norm;
        for (int c = 0; c < pool.D / 2; ++c) p.axis[c] = axes->pair[c];
    }
    // tokens of a CTA: rows that fill its passes, fewer while that would leave
    // less than four CTAs an SM
    const int R = hq + 2 * pool.hkv, pass = kUnroll * kThreads / (pool.D / 16);
    int64_t tok = pass / std::gcd(R, pass);
    if (tok > kMaxTok) tok = kMaxTok;
    if (tok > n / 608) tok = n / 608;
    if (tok < 1) tok = 1;
    p.tok = (int)tok;
    const int64_t grid = (n + tok - 1) / tok;
    if (grid > INT32_MAX) return rx_set_error(RX_ERR_UNSUPPORTED, "%s: %lld tokens", who, (long long)n);
    auto pick = [&](auto ax) {
        constexpr bool AX = decltype(ax)::value;
        return pool.D == 128 ? (pool.f8 ? qk_norm_rope_store_kernel<128, true, AX> : qk_norm_rope_store_kernel<128, false, AX>)
                             : (pool.f8 ? qk_norm_rope_store_kernel<64, true, AX> : qk_norm_rope_store_kernel<64, false, AX>);
    };
    auto kernel = axes ? pick(std::true_type{}) : pick(std::false_type{});
    kernel<<<(unsigned)grid, kThreads, 0, (cudaStream_t)stream>>>(p);
    RX_CUDA_CHECK(cudaGetLastError());
    return RX_OK;
}

}  // namespace

extern "C" int rx_qk_norm_rope_store(const rx_kv_pool *pool_in, const void *q, int64_t q_stride, void *q_out,
                                     const void *k_new, const void *v_new, int64_t kv_stride, const void *q_weight,
                                     const void *k_weight, const int32_t *slots, const int32_t *pos, int64_t n,
                                     int32_t num_q_heads, double base, float eps, int32_t *dev_status, void *stream)
{
    rx_kv_pool v;
    if (const int rc = rx_pool_layer(pool_in, &v, 0, "rx_qk_norm_rope_store")) return rc;
    if (!pool_in || !v.k || !v.v || v.num_slots <= 0 || v.num_kv_heads <= 0)
        return rx_set_error(RX_ERR_INVALID, "rx_qk_norm_rope_store: invalid pool");
    const Pool pool{v.k, v.v, v.num_slots, v.num_kv_heads, v.head_dim, false, 1.f, 1.f};
    return norm_call("rx_qk_norm_rope_store", pool, q, q_stride, q_out, k_new, v_new, kv_stride, q_weight, k_weight,
                     slots, pos, n, num_q_heads, base, eps, dev_status, stream);
}

extern "C" int rx_qk_norm_rope_store_fp8(const rx_kv_pool_fp8 *pool_in, const void *q, int64_t q_stride, void *q_out,
                                         const void *k_new, const void *v_new, int64_t kv_stride,
                                         const void *q_weight, const void *k_weight, const int32_t *slots,
                                         const int32_t *pos, int64_t n, int32_t num_q_heads, double base, float eps,
                                         int32_t *dev_status, void *stream)
{
    rx_kv_pool_fp8 v;
    if (const int rc = rx_pool_layer(pool_in, &v, 1, "rx_qk_norm_rope_store_fp8")) return rc;
    if (!pool_in || !v.k || !v.v || v.num_slots <= 0 || v.num_kv_heads <= 0 || !(v.k_scale > 0.f) ||
        !(v.v_scale > 0.f))
        return rx_set_error(RX_ERR_INVALID, "rx_qk_norm_rope_store_fp8: invalid pool");
    const Pool pool{v.k, v.v, v.num_slots, v.num_kv_heads, v.head_dim, true, v.k_scale, v.v_scale};
    return norm_call("rx_qk_norm_rope_store_fp8", pool, q, q_stride, q_out, k_new, v_new, kv_stride, q_weight,
                     k_weight, slots, pos, n, num_q_heads, base, eps, dev_status, stream);
}

extern "C" int rx_qk_rope_axes_store(const rx_kv_pool *pool_in, const void *q, int64_t q_stride, void *q_out,
                                     const void *k_new, const void *v_new, int64_t kv_stride, int32_t norm,
                                     const void *q_weight, const void *k_weight, const int32_t *slots, const int32_t *pos,
                                     int64_t pos_stride, int32_t num_axes, const uint8_t *pair_axis, int64_t n,
                                     int32_t num_q_heads, double base, float eps, int32_t *dev_status, void *stream)
{
    rx_kv_pool v;
    if (const int rc = rx_pool_layer(pool_in, &v, 0, "rx_qk_rope_axes_store")) return rc;
    if (!pool_in || !v.k || !v.v || v.num_slots <= 0 || v.num_kv_heads <= 0)
        return rx_set_error(RX_ERR_INVALID, "rx_qk_rope_axes_store: invalid pool");
    const Pool pool{v.k, v.v, v.num_slots, v.num_kv_heads, v.head_dim, false, 1.f, 1.f};
    const Axes axes{pos_stride, num_axes, pair_axis, norm};
    return norm_call("rx_qk_rope_axes_store", pool, q, q_stride, q_out, k_new, v_new, kv_stride, q_weight, k_weight,
                     slots, pos, n, num_q_heads, base, eps, dev_status, stream, &axes);
}

extern "C" int rx_qk_rope_axes_store_fp8(const rx_kv_pool_fp8 *pool_in, const void *q, int64_t q_stride, void *q_out,
                                         const void *k_new, const void *v_new, int64_t kv_stride, int32_t norm,
                                         const void *q_weight, const void *k_weight, const int32_t *slots,
                                         const int32_t *pos, int64_t pos_stride, int32_t num_axes,
                                         const uint8_t *pair_axis, int64_t n, int32_t num_q_heads, double base, float eps,
                                         int32_t *dev_status, void *stream)
{
    rx_kv_pool_fp8 v;
    if (const int rc = rx_pool_layer(pool_in, &v, 1, "rx_qk_rope_axes_store_fp8")) return rc;
    if (!pool_in || !v.k || !v.v || v.num_slots <= 0 || v.num_kv_heads <= 0 || !(v.k_scale > 0.f) ||
        !(v.v_scale > 0.f))
        return rx_set_error(RX_ERR_INVALID, "rx_qk_rope_axes_store_fp8: invalid pool");
    const Pool pool{v.k, v.v, v.num_slots, v.num_kv_heads, v.head_dim, true, v.k_scale, v.v_scale};
    const Axes axes{pos_stride, num_axes, pair_axis, norm};
    return norm_call("rx_qk_rope_axes_store_fp8", pool, q, q_stride, q_out, k_new, v_new, kv_stride, q_weight, k_weight,
                     slots, pos, n, num_q_heads, base, eps, dev_status, stream, &axes);
}
