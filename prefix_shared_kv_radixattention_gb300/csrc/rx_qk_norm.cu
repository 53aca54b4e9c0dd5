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
#include <type_traits>

#include "rx_common.cuh"
#include "rx_rope.cuh"

namespace {

using bf16 = __nv_bfloat16;

constexpr int kThreads = 256;
constexpr int kMaxTok = 16;   // tokens of one CTA
constexpr int kUnroll = 4;    // rows a thread has in flight

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
    float k_scale, v_scale;
    int32_t *status;
    rx::RopeTab tab;
};

__device__ __forceinline__ void widen(const uint4 &v, float (&x)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[k]));
        x[2 * k] = f.x;
        x[2 * k + 1] = f.y;
    }
}

__device__ __forceinline__ uint4 narrow(const float (&x)[8])
{
    return make_uint4(rx::pack_bf16(x[0], x[1]), rx::pack_bf16(x[2], x[3]), rx::pack_bf16(x[4], x[5]),
                      rx::pack_bf16(x[6], x[7]));
}

// Eight fp32 values as E4M3 codes of value / scale: a correctly rounded
// division, then the nearest code, magnitudes past 448 saturated.
__device__ __forceinline__ uint2 codes(const float (&x)[8], float scale)
{
    uint16_t pair[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float lo = __fdiv_rn(x[2 * k], scale), hi = __fdiv_rn(x[2 * k + 1], scale);
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(pair[k]) : "f"(hi), "f"(lo));
    }
    return make_uint2((uint32_t)pair[0] | ((uint32_t)pair[1] << 16), (uint32_t)pair[2] | ((uint32_t)pair[3] << 16));
}

template <int D, bool F8>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_store_kernel(const __grid_constant__ NormParams p)
{
    constexpr int LPR = D / 16;             // lanes of one head
    constexpr int RPP = kThreads / LPR;     // heads of one pass of the CTA
    constexpr int HALF = D / 2;
    using Chunk = std::conditional_t<F8, uint2, uint4>;  // 8 values of the pool
    // pair 2j, 2j + 1 of lane gi: {cos, sin, cos, sin} at [token][j][gi], so
    // that the lanes of a head read consecutive 16-byte words
    __shared__ float4 cs[kMaxTok][4][LPR];
    const int gi = threadIdx.x % LPR, sub = threadIdx.x / LPR;
    const int64_t t0 = (int64_t)blockIdx.x * p.tok;
    const int ntok = (int)min((int64_t)p.tok, p.n - t0);
    const int R = p.hq + 2 * p.hkv;
    const int total = ntok * R;

    uint4 lo[kUnroll], hi[kUnroll];
    auto load = [&](int base) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int idx = base + u * RPP + sub;
            lo[u] = hi[u] = make_uint4(0, 0, 0, 0);
            if (idx < total) {
                const int tt = idx / R, h = idx - tt * R;
                const bf16 *src = h < p.hq            ? p.q + (t0 + tt) * p.q_stride + (int64_t)h * D
                                  : h < p.hq + p.hkv ? p.k_new + (t0 + tt) * p.kv_stride + (int64_t)(h - p.hq) * D
                                                     : p.v_new + (t0 + tt) * p.kv_stride +
                                                           (int64_t)(h - p.hq - p.hkv) * D;
                // plain loads: q_out may be q
                lo[u] = *reinterpret_cast<const uint4 *>(src + gi * 8);
                hi[u] = *reinterpret_cast<const uint4 *>(src + HALF + gi * 8);
            }
        }
    };
    load(0);

    for (int i = threadIdx.x; i < ntok * HALF; i += kThreads) {
        const int tt = i / HALF, c = i % HALF;
        const int32_t pos = __ldg(p.pos + t0 + tt);
        const uint32_t up = pos < 0 ? 0u - (uint32_t)pos : (uint32_t)pos;
        float sn, cn;
        rx::sincos_at(p.tab, up, c, sn, cn);
        float *dst = reinterpret_cast<float *>(&cs[tt][(c % 8) / 2][c / 8]) + 2 * (c % 2);
        dst[0] = cn;
        dst[1] = pos < 0 ? -sn : sn;
    }
    __syncthreads();

    for (int base = 0; base < total; base += RPP * kUnroll) {
        if (base > 0) load(base);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int idx = base + u * RPP + sub;
            const bool in = idx < total;
            const int tt = in ? idx / R : 0, h = in ? idx - tt * R : 0;
            float a[8], b[8];
            widen(lo[u], a);
            widen(hi[u], b);
            float ss = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) ss = fmaf(a[k], a[k], fmaf(b[k], b[k], ss));
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (!in) continue;
            const bool is_q = h < p.hq, is_v = h >= p.hq + p.hkv;
            if (!is_v) {
                const float r = 1.f / sqrtf(ss * (1.f / D) + p.eps);
                const bf16 *w = is_q ? p.qw : p.kw;
                float wa[8], wb[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) wa[k] = wb[k] = 1.f;
                if (w) {
                    widen(__ldg(reinterpret_cast<const uint4 *>(w + gi * 8)), wa);
                    widen(__ldg(reinterpret_cast<const uint4 *>(w + HALF + gi * 8)), wb);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 q = cs[tt][j][gi];
                    const float a0 = a[2 * j] * r * wa[2 * j], b0 = b[2 * j] * r * wb[2 * j];
                    const float a1 = a[2 * j + 1] * r * wa[2 * j + 1], b1 = b[2 * j + 1] * r * wb[2 * j + 1];
                    a[2 * j] = a0 * q.x - b0 * q.y;
                    b[2 * j] = b0 * q.x + a0 * q.y;
                    a[2 * j + 1] = a1 * q.z - b1 * q.w;
                    b[2 * j + 1] = b1 * q.z + a1 * q.w;
                }
            }
            if (is_q) {
                bf16 *dst = p.q_out + ((t0 + tt) * p.hq + h) * D;
                *reinterpret_cast<uint4 *>(dst + gi * 8) = narrow(a);
                *reinterpret_cast<uint4 *>(dst + HALF + gi * 8) = narrow(b);
                continue;
            }
            const int32_t s = __ldg(p.slots + t0 + tt);
            if (s < 0 || (int64_t)s >= p.num_slots) {
                if (p.status && h == p.hq && gi == 0) atomicOr(p.status, RX_DEV_BAD_SLOT);
                continue;
            }
            const int g = h - p.hq - (is_v ? p.hkv : 0);
            Chunk *dst = static_cast<Chunk *>(is_v ? p.v_pool : p.k_pool) + ((int64_t)s * p.hkv + g) * (D / 8);
            if constexpr (F8) {
                dst[gi] = codes(a, is_v ? p.v_scale : p.k_scale);
                dst[LPR + gi] = codes(b, is_v ? p.v_scale : p.k_scale);
            } else {
                dst[gi] = is_v ? lo[u] : narrow(a);
                dst[LPR + gi] = is_v ? hi[u] : narrow(b);
            }
        }
    }
}

struct Pool {
    void *k, *v;
    int64_t num_slots;
    int hkv, D;
    bool f8;
    float k_scale, v_scale;
};

int norm_call(const char *who, const Pool &pool, const void *q, int64_t q_stride, void *q_out, const void *k_new,
              const void *v_new, int64_t kv_stride, const void *qw, const void *kw, const int32_t *slots,
              const int32_t *pos, int64_t n, int32_t hq, double base, float eps, int32_t *dev_status, void *stream)
{
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
    p.status = dev_status;
    p.tab = tab;
    // tokens of a CTA: enough for kUnroll rows a thread, fewer while that
    // would leave less than two CTAs an SM
    const int R = hq + 2 * pool.hkv, rpp = kThreads / (pool.D / 16);
    int64_t tok = (kUnroll * rpp + R - 1) / R;
    if (tok > kMaxTok) tok = kMaxTok;
    if (tok > n / 304) tok = n / 304;
    if (tok < 1) tok = 1;
    p.tok = (int)tok;
    const int64_t grid = (n + tok - 1) / tok;
    if (grid > INT32_MAX) return rx_set_error(RX_ERR_UNSUPPORTED, "%s: %lld tokens", who, (long long)n);
    auto kernel = pool.D == 128 ? (pool.f8 ? qk_norm_rope_store_kernel<128, true> : qk_norm_rope_store_kernel<128, false>)
                                : (pool.f8 ? qk_norm_rope_store_kernel<64, true> : qk_norm_rope_store_kernel<64, false>);
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
