// rx_split.h -- attention with rules on the scores by the kernels that share a
// context among CTAs (rx_rules.cu), for rx_attn_decode_rules and, where a call
// has few query rows, rx_attn_extend_rules.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "rx.h"

// One layer of a pool: bf16 rows, or E4M3 codes with a scale per pool.
struct RxAttnPool {
    const void *k, *v;
    int64_t num_slots;
    int hkv, D;
    bool f8;
    float k_scale, v_scale;
};

#define RX_SPLIT_MAX_LEN 1024  // new tokens of a request

// qo_indptr null: one token a request, and prefix_len holds its context's
// length.  extend_len: the requests' new tokens, with qo_indptr.
int rx_split_rules(const char *who, const RxAttnPool &pool, const void *q, void *o, float *lse, int32_t hq,
                   const int32_t *qo_indptr, const int32_t *req_idx, const int32_t *prefix_len, const int32_t *extend_len,
                   const int32_t *rtt, int64_t rtt_stride, int32_t batch, int32_t max_len, void *workspace, size_t ws_bytes,
                   float sm_scale, const rx_attn_rules *rules, int32_t *dev_status, void *stream);
size_t rx_split_workspace(int32_t batch, int32_t hq, int32_t hkv, int32_t head_dim, int32_t max_len);
