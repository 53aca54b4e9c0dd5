// rx_rules.cu -- attention with rules on the scores by the kernels of rx_tree.cuh,
// which share each context among CTAs: one token a request (rx_attn_decode_rules)
// and the rx_attn_extend_rules calls with few query rows.
#include "rx_tree.cuh"

namespace {

template <int RU>
int go_kind(const TParams &p, const TreePool &pool, cudaStream_t st)
{
    return pool.D == 128 ? launch_of<RU, 128>(p, pool, st) : launch_of<RU, 64>(p, pool, st);
}

template <int GN>
int go_keys(const TParams &p, const TreePool &pool, cudaStream_t st)
{
    return pool.f8 ? launch<kRows, true, rx::kAnyRules, 1, true, GN>(p, st) : launch<kRows, false, rx::kAnyRules, 1, true, GN>(p, st);
}

int go(const TParams &p, const TreePool &pool, cudaStream_t st)
{
    // one token a request: the products with the positions as their wide side.
    // It takes 16 rows, and a head_dim that fills the tensor core's 128 lanes.
    // (Long chat, a cap of 50: 254 us, with the rows as the wide side 403; few-shot
    // with slopes 163, 406.)
    // It takes the cap from the exponential and the reciprocal alone (the
    // polynomials beside them: windowed E4M3 208 us, without 170 then), whose error grows
    // with the cap: up to 150 a log-sum-exp is off by less than 1e-6 of itself.
    if (!p.qo_indptr && p.G <= kKeyRows && pool.D == kRows && p.rules.c2 <= 150.f * rx::kLog2e)
        return p.G <= 8 ? go_keys<8>(p, pool, st) : go_keys<kKeyRows>(p, pool, st);
    switch (rx::rules_kind(p.rules)) {
    case rx::kFixedCap: return go_kind<rx::kFixedCap>(p, pool, st);
    case rx::kRange: return go_kind<rx::kRange>(p, pool, st);
    default: return go_kind<rx::kAnyRules>(p, pool, st);
    }
}

}  // namespace

int rx_split_rules(const char *who, const RxAttnPool &pool, const void *q, void *o, float *lse, int32_t hq,
                   const int32_t *qo_indptr, const int32_t *req_idx, const int32_t *prefix_len, const int32_t *extend_len,
                   const int32_t *rtt, int64_t rtt_stride, int32_t batch, int32_t max_len, void *workspace, size_t ws_bytes,
                   float sm_scale, const rx_attn_rules *rules, int32_t *dev_status, void *stream)
{
    return tree_call(who, pool, q, o, lse, hq, qo_indptr, req_idx, prefix_len, nullptr, 0, rtt, rtt_stride, batch, max_len,
                     workspace, ws_bytes, sm_scale, dev_status, stream, go, rules, extend_len);
}

size_t rx_split_workspace(int32_t batch, int32_t hq, int32_t hkv, int32_t head_dim, int32_t max_len)
{
    return rx_attn_tree_workspace(batch, hq, hkv, head_dim, max_len);
}

namespace {

// One token a request, after the pool's checks.
int decode_rules(const char *who, const RxAttnPool &pool, const void *q, void *o, float *lse, int32_t hq,
                 const int32_t *req_idx, const int32_t *seq_len, const int32_t *rtt, int64_t rtt_stride, int32_t batch,
                 void *workspace, size_t ws_bytes, float sm_scale, const rx_attn_rules *rules, int32_t *dev_status, void *stream)
{
    if (!rules) return rx_set_error(RX_ERR_INVALID, "%s: no rules (rx_attn_decode is the call without them)", who);
    if (rules->see_to) return rx_set_error(RX_ERR_INVALID, "%s: a last token sees nothing behind itself (see_to)", who);
    return rx_split_rules(who, pool, q, o, lse, hq, nullptr, req_idx, seq_len, nullptr, rtt, rtt_stride, batch, 1, workspace,
                          ws_bytes, sm_scale, rules, dev_status, stream);
}

}  // namespace

extern "C" int rx_attn_decode_rules(const rx_kv_pool *pool_in, const void *q, void *o, float *lse, int32_t hq,
                                    const int32_t *req_idx, const int32_t *seq_len, const int32_t *rtt, int64_t rtt_stride,
                                    int32_t batch, const rx_attn_rules *rules, void *workspace, size_t ws_bytes,
                                    float sm_scale, int32_t *dev_status, void *stream)
{
    rx_kv_pool v;
    if (const int rc = rx_pool_layer(pool_in, &v, 0, "rx_attn_decode_rules")) return rc;
    if (!pool_in || !v.k || !v.v || v.num_slots <= 0 || v.num_kv_heads <= 0)
        return rx_set_error(RX_ERR_INVALID, "rx_attn_decode_rules: invalid pool");
    const RxAttnPool pool{v.k, v.v, v.num_slots, v.num_kv_heads, v.head_dim, false, 1.f, 1.f};
    return decode_rules("rx_attn_decode_rules", pool, q, o, lse, hq, req_idx, seq_len, rtt, rtt_stride, batch, workspace,
                        ws_bytes, sm_scale, rules, dev_status, stream);
}

extern "C" int rx_attn_decode_rules_fp8(const rx_kv_pool_fp8 *pool_in, const void *q, void *o, float *lse, int32_t hq,
                                        const int32_t *req_idx, const int32_t *seq_len, const int32_t *rtt,
                                        int64_t rtt_stride, int32_t batch, const rx_attn_rules *rules, void *workspace,
                                        size_t ws_bytes, float sm_scale, int32_t *dev_status, void *stream)
{
    rx_kv_pool_fp8 v;
    if (const int rc = rx_pool_layer(pool_in, &v, 1, "rx_attn_decode_rules_fp8")) return rc;
    if (!pool_in || !v.k || !v.v || v.num_slots <= 0 || v.num_kv_heads <= 0 || !(v.k_scale > 0.f) || !(v.v_scale > 0.f))
        return rx_set_error(RX_ERR_INVALID, "rx_attn_decode_rules_fp8: invalid pool");
    const RxAttnPool pool{v.k, v.v, v.num_slots, v.num_kv_heads, v.head_dim, true, v.k_scale, v.v_scale};
    return decode_rules("rx_attn_decode_rules_fp8", pool, q, o, lse, hq, req_idx, seq_len, rtt, rtt_stride, batch, workspace,
                        ws_bytes, sm_scale, rules, dev_status, stream);
}
