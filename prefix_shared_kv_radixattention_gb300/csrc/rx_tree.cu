// rx_tree.cu -- attention of drafted token trees over the slot pool.
//
// Drafted token i of request b sees the request's whole prefix (positions
// 0 .. P_b - 1) and, of the drafted tokens (positions P_b + j), those whose
// bit j is set in its mask row:
//     s_j = sm_scale q . K[slot_j],  o = sum_seen softmax(s)_j V[slot_j],
//     lse = log sum_seen exp(s_j);   nothing seen: o = 0, lse = -inf.
//
// One warp per (drafted token, q head) walks the positions with a running
// maximum and sum; each lane holds d / 32 of the head's values.
#include <math.h>

#include "rx_common.cuh"

namespace {

using bf16 = __nv_bfloat16;

constexpr int kMaxTree = 1024;

struct TParams {
    const bf16 *q;
    bf16 *o;
    float *lse;
    const void *k;
    const void *v;
    int64_t num_slots;
    int hq, hkv, G;
    const int32_t *qo_indptr;
    const int32_t *req_idx;
    const int32_t *prefix_len;
    const uint32_t *mask;
    int words;
    const int32_t *rtt;
    int64_t rtt_stride;
    int batch, max_tree;
    float scale_log2;   // sm_scale log2(e), times K's scale for an FP8 pool
    float v_scale;      // V's scale for an FP8 pool; 1 otherwise
    int32_t *status;
};

template <bool F8>
__device__ __forceinline__ float value(const void *pool, int64_t at)
{
    if constexpr (F8) {
        const uint32_t h = rx::e4m3x2_to_f16x2(__ldg(static_cast<const unsigned char *>(pool) + at));
        return __half2float(__ushort_as_half((unsigned short)(h & 0xFFFFu)));
    } else {
        return __bfloat162float(static_cast<const bf16 *>(pool)[at]);
    }
}

template <int D, bool F8>
__global__ void __launch_bounds__(128) tree_warp_kernel(const TParams p)
{
    constexpr int PER = D / 32;
    const int lane = threadIdx.x & 31;
    const int b = blockIdx.y;
    const int t0 = __ldg(p.qo_indptr + b), T = __ldg(p.qo_indptr + b + 1) - t0;
    const int64_t P = __ldg(p.prefix_len + b);
    if (T == 0) return;
    if (T < 0 || T > p.max_tree || P < 0 || P + T > p.rtt_stride) {
        if (p.status && threadIdx.x == 0) atomicOr(p.status, RX_DEV_BAD_LEN);
        return;
    }
    const int w = (int)((blockIdx.x * blockDim.x + threadIdx.x) >> 5);
    const int i = w / p.hq, h = w - i * p.hq;
    if (i >= T) return;
    const int g = h / p.G;
    const int32_t *slots = p.rtt + (int64_t)__ldg(p.req_idx + b) * p.rtt_stride;
    const int64_t row = ((int64_t)(t0 + i) * p.hq + h) * D;
    float q[PER], o[PER];
#pragma unroll
    for (int c = 0; c < PER; ++c) {
        q[c] = __bfloat162float(p.q[row + c * 32 + lane]);
        o[c] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int64_t j = 0; j < P + T; ++j) {
        if (j >= P) {
            const int e = (int)(j - P);
            const bool see = p.mask ? (__ldg(p.mask + (int64_t)(t0 + i) * p.words + (e >> 5)) >> (e & 31)) & 1u : e <= i;
            if (!see) continue;
        }
        const int32_t s = __ldg(slots + j);
        const bool ok = s >= 0 && (int64_t)s < p.num_slots;
        if (!ok && p.status && lane == 0) atomicOr(p.status, RX_DEV_BAD_SLOT);
        const int64_t at = ((int64_t)(ok ? s : 0) * p.hkv + g) * D + lane;
        float x = 0.f;
#pragma unroll
        for (int c = 0; c < PER; ++c) x = fmaf(q[c], ok ? value<F8>(p.k, at + c * 32) : 0.f, x);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
        x *= p.scale_log2;
        const float mn = fmaxf(m, x), a = m == -INFINITY ? 0.f : exp2f(m - mn), e = exp2f(x - mn);
        l = l * a + e;
#pragma unroll
        for (int c = 0; c < PER; ++c) o[c] = o[c] * a + e * (ok ? value<F8>(p.v, at + c * 32) : 0.f);
        m = mn;
    }
    const float inv = l == 0.f ? 0.f : p.v_scale / l;
#pragma unroll
    for (int c = 0; c < PER; ++c) p.o[row + c * 32 + lane] = __float2bfloat16_rn(o[c] * inv);
    if (p.lse && lane == 0) p.lse[row / D] = l == 0.f ? -INFINITY : (m + log2f(l)) * rx::kLn2;
}

struct TreePool {
    const void *k, *v;
    int64_t num_slots;
    int hkv, D;
    bool f8;
    float k_scale, v_scale;
};

bool tree_shape_ok(int32_t batch, int32_t hq, int32_t hkv, int32_t D, int32_t max_tree)
{
    return batch >= 0 && batch <= 65535 && hq > 0 && hkv > 0 && hq % hkv == 0 && hq / hkv <= 128 &&
           (D == 64 || D == 128) && max_tree >= 1 && max_tree <= kMaxTree;
}

int tree_call(const char *who, const TreePool &pool, const void *q, void *o, float *lse, int32_t hq,
              const int32_t *qo_indptr, const int32_t *req_idx, const int32_t *prefix_len, const uint32_t *mask,
              int32_t words, const int32_t *rtt, int64_t rtt_stride, int32_t batch, int32_t max_tree,
              void *workspace, size_t ws_bytes, float sm_scale, int32_t *dev_status, void *stream)
{
    if (!q || !o || !qo_indptr || !req_idx || !prefix_len || !rtt || rtt_stride <= 0 || rtt_stride > INT32_MAX ||
        batch < 0 || hq <= 0 || !(sm_scale > 0.f) || max_tree < 1)
        return rx_set_error(RX_ERR_INVALID, "%s: invalid argument", who);
    if (pool.D != 64 && pool.D != 128)
        return rx_set_error(RX_ERR_UNSUPPORTED, "%s: head_dim %d (supported: 64, 128)", who, pool.D);
    if (!tree_shape_ok(batch, hq, pool.hkv, pool.D, max_tree))
        return rx_set_error(RX_ERR_UNSUPPORTED,
                            "%s: batch %d (up to 65535), %d q heads over %d kv heads (up to 128 each), trees of %d (up to %d)",
                            who, batch, hq, pool.hkv, max_tree, kMaxTree);
    if (mask && (int64_t)words * 32 < max_tree)
        return rx_set_error(RX_ERR_INVALID, "%s: mask rows of %d words for trees of %d", who, words, max_tree);
    const uintptr_t pool_align = pool.f8 ? 7 : 15;
    if (rx_misaligned16(q) || rx_misaligned16(o) || (reinterpret_cast<uintptr_t>(pool.k) & pool_align) != 0 ||
        (reinterpret_cast<uintptr_t>(pool.v) & pool_align) != 0 || (reinterpret_cast<uintptr_t>(lse) & 3) != 0 ||
        (reinterpret_cast<uintptr_t>(mask) & 3) != 0)
        return rx_set_error(RX_ERR_INVALID, "%s: q and o must be 16-byte aligned, the pools %d-byte aligned", who,
                            (int)pool_align + 1);
    const size_t need = rx_attn_tree_workspace(batch, hq, pool.hkv, pool.D, max_tree);
    if (!workspace || ws_bytes < need)
        return rx_set_error(RX_ERR_CAPACITY, "%s: workspace of %zu bytes, %zu needed", who, workspace ? ws_bytes : (size_t)0,
                            need);
    if ((reinterpret_cast<uintptr_t>(workspace) & 255) != 0)
        return rx_set_error(RX_ERR_INVALID, "%s: workspace must be 256-byte aligned", who);
    if (batch == 0) return RX_OK;
    TParams p{};
    p.q = (const bf16 *)q;
    p.o = (bf16 *)o;
    p.lse = lse;
    p.k = pool.k;
    p.v = pool.v;
    p.num_slots = pool.num_slots;
    p.hq = hq;
    p.hkv = pool.hkv;
    p.G = hq / pool.hkv;
    p.qo_indptr = qo_indptr;
    p.req_idx = req_idx;
    p.prefix_len = prefix_len;
    p.mask = mask;
    p.words = words;
    p.rtt = rtt;
    p.rtt_stride = rtt_stride;
    p.batch = batch;
    p.max_tree = max_tree;
    p.scale_log2 = sm_scale * pool.k_scale * rx::kLog2e;
    p.v_scale = pool.v_scale;
    p.status = dev_status;
    const dim3 grid((unsigned)(((int64_t)max_tree * hq + 3) / 4), (unsigned)batch);
    auto kernel = pool.D == 128 ? (pool.f8 ? tree_warp_kernel<128, true> : tree_warp_kernel<128, false>)
                                : (pool.f8 ? tree_warp_kernel<64, true> : tree_warp_kernel<64, false>);
    kernel<<<grid, 128, 0, (cudaStream_t)stream>>>(p);
    RX_CUDA_CHECK(cudaGetLastError());
    return RX_OK;
}

}  // namespace

extern "C" size_t rx_attn_tree_workspace(int32_t batch, int32_t hq, int32_t hkv, int32_t head_dim, int32_t max_tree)
{
    if (!tree_shape_ok(batch, hq, hkv, head_dim, max_tree)) {
        rx_set_error(RX_ERR_INVALID, "rx_attn_tree_workspace: invalid argument");
        return 0;
    }
    return 256;
}

extern "C" int rx_attn_tree(const rx_kv_pool *pool_in, const void *q, void *o, float *lse, int32_t hq,
                            const int32_t *qo_indptr, const int32_t *req_idx, const int32_t *prefix_len,
                            const uint32_t *mask, int32_t words, const int32_t *rtt, int64_t rtt_stride, int32_t batch,
                            int32_t max_tree, void *workspace, size_t ws_bytes, float sm_scale, int32_t *dev_status,
                            void *stream)
{
    rx_kv_pool v;
    if (const int rc = rx_pool_layer(pool_in, &v, 0, "rx_attn_tree")) return rc;
    if (!pool_in || !v.k || !v.v || v.num_slots <= 0 || v.num_kv_heads <= 0)
        return rx_set_error(RX_ERR_INVALID, "rx_attn_tree: invalid pool");
    const TreePool pool{v.k, v.v, v.num_slots, v.num_kv_heads, v.head_dim, false, 1.f, 1.f};
    return tree_call("rx_attn_tree", pool, q, o, lse, hq, qo_indptr, req_idx, prefix_len, mask, words, rtt, rtt_stride,
                     batch, max_tree, workspace, ws_bytes, sm_scale, dev_status, stream);
}

extern "C" int rx_attn_tree_fp8(const rx_kv_pool_fp8 *pool_in, const void *q, void *o, float *lse, int32_t hq,
                                const int32_t *qo_indptr, const int32_t *req_idx, const int32_t *prefix_len,
                                const uint32_t *mask, int32_t words, const int32_t *rtt, int64_t rtt_stride,
                                int32_t batch, int32_t max_tree, void *workspace, size_t ws_bytes, float sm_scale,
                                int32_t *dev_status, void *stream)
{
    rx_kv_pool_fp8 v;
    if (const int rc = rx_pool_layer(pool_in, &v, 1, "rx_attn_tree_fp8")) return rc;
    if (!pool_in || !v.k || !v.v || v.num_slots <= 0 || v.num_kv_heads <= 0 || !(v.k_scale > 0.f) ||
        !(v.v_scale > 0.f))
        return rx_set_error(RX_ERR_INVALID, "rx_attn_tree_fp8: invalid pool");
    const TreePool pool{v.k, v.v, v.num_slots, v.num_kv_heads, v.head_dim, true, v.k_scale, v.v_scale};
    return tree_call("rx_attn_tree_fp8", pool, q, o, lse, hq, qo_indptr, req_idx, prefix_len, mask, words, rtt,
                     rtt_stride, batch, max_tree, workspace, ws_bytes, sm_scale, dev_status, stream);
}
