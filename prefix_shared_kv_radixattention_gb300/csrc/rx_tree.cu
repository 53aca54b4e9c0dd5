// rx_tree.cu -- the entry points of tree attention; the kernels are in rx_tree.cuh.
#include "rx_tree.cuh"

namespace {

int go(const TParams &p, const TreePool &pool, cudaStream_t st)
{
    return pool.D == 128 ? launch_of<rx::kNoRules, 128>(p, pool, st) : launch_of<rx::kNoRules, 64>(p, pool, st);
}

}  // namespace

extern "C" size_t rx_attn_tree_workspace(int32_t batch, int32_t hq, int32_t hkv, int32_t head_dim, int32_t max_tree)
{
    if (!tree_shape_ok(batch, hq, hkv, head_dim, max_tree)) {
        rx_set_error(RX_ERR_INVALID, "rx_attn_tree_workspace: invalid argument");
        return 0;
    }
    const int nt = row_tiles(hq, hkv, max_tree);
    return part_bytes(nt, head_dim) + (size_t)2 * kCtas * nt * kRows * sizeof(float) +
           kCtas * sizeof(Cut);
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
                     batch, max_tree, workspace, ws_bytes, sm_scale, dev_status, stream, go);
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
                     rtt_stride, batch, max_tree, workspace, ws_bytes, sm_scale, dev_status, stream, go);
}
