// rx_maps.cu -- the lists that the calls of a step take for a ragged batch,
// from the requests' lengths: where each request's new tokens start, the
// contexts' lengths, and the position and slot of every new token.
//
//     qo_indptr[b] = sum_{a < b} new_len[a]
//     token t of request b (qo_indptr[b] + i = t): pos = prefix_len[b] + i,
//     slot = req_to_token[req_idx[b]][pos], or from the request's pages.
//
// A few bytes a token: what costs is the way from the launch to the last
// dependent load.  So it is one kernel, in which every CTA scans the lengths
// for itself (they are read from L2 once a CTA, and no CTA waits for another)
// and takes a share of the tokens; a token finds its request in the sums by
// binary search in shared memory.  64 requests of one token 3.1 us in a graph, 256
// prompts of up to 1,024 tokens over pages 5.8 us.
#include "rx_common.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 4;  // tokens of a thread

struct MapParams {
    const int32_t *req_idx, *prefix_len, *new_len;
    int batch;
    int32_t *rtt;
    int64_t rtt_stride;
    const int32_t *pages;
    int64_t pages_stride;
    int page_size;
    int64_t num_slots;
    int64_t positions;   // that a request can have
    int32_t *qo_indptr, *seq_len, *pos, *slots;
    int64_t max_tokens;
    int32_t *status;
};

// New tokens of request b (0: none, or its lengths are out of range).
__device__ __forceinline__ int new_tokens(const MapParams &p, int b, bool &bad)
{
    const int64_t P = __ldg(p.prefix_len + b), E = __ldg(p.new_len + b);
    bad = P < 0 || E < 0 || P + E > p.positions;
    return bad ? 0 : (int)E;
}

__global__ void __launch_bounds__(kThreads) step_maps_kernel(const __grid_constant__ MapParams p)
{
    // pre[i]: new tokens of the requests before those of thread i
    __shared__ int64_t pre[kThreads + 1];
    __shared__ int64_t warp_tot[kThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (p.batch + kThreads - 1) / kThreads;
    const int b0 = min((int64_t)threadIdx.x * per, (int64_t)p.batch), b1 = min((int64_t)b0 + per, (int64_t)p.batch);
    int64_t sum = 0;
    for (int b = b0; b < b1; ++b) {
        bool bad;
        sum += new_tokens(p, b, bad);
        if (blockIdx.x == 0) {
            if (bad && p.status) atomicOr(p.status, RX_DEV_BAD_LEN);
            if (p.seq_len) p.seq_len[b] = bad ? 0 : __ldg(p.prefix_len + b) + __ldg(p.new_len + b);
        }
    }
    int64_t x = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) warp_tot[warp] = x;
    __syncthreads();
    int64_t base = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) base += warp_tot[w];
        total += warp_tot[w];
    }
    base += x - sum;
    pre[threadIdx.x] = base;
    if (threadIdx.x == 0) pre[kThreads] = total;
    if (blockIdx.x == 0) {
        int64_t at = base;
        for (int b = b0; b < b1; ++b) {
            bool bad;
            p.qo_indptr[b] = (int32_t)min(at, p.max_tokens);
            at += new_tokens(p, b, bad);
        }
        if (threadIdx.x == 0) {
            p.qo_indptr[p.batch] = (int32_t)min(total, p.max_tokens);
            if (total > p.max_tokens && p.status) atomicOr(p.status, RX_DEV_BAD_LEN);
        }
    }
    __syncthreads();

    const int64_t end = min(total, p.max_tokens);
#pragma unroll
    for (int u = 0; u < kTokens; ++u) {
        const int64_t t = ((int64_t)blockIdx.x * kTokens + u) * kThreads + threadIdx.x;
        if (t >= end) break;
        int lo = 0, hi = kThreads - 1;  // the last thread whose requests start at or before token t
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (pre[mid] <= t) lo = mid; else hi = mid - 1;
        }
        int64_t i = t - pre[lo];
        int b = lo * per;
        for (;;) {
            bool bad;
            const int e = new_tokens(p, b, bad);
            if (i < e) break;
            i -= e;
            ++b;
        }
        const int at = __ldg(p.prefix_len + b) + (int)i;
        const int64_t row = __ldg(p.req_idx + b);
        int32_t slot;
        if (p.pages) {
            const int pg = at / p.page_size;
            const int64_t page = __ldg(p.pages + row * p.pages_stride + pg);
            const int64_t s = page * p.page_size + (at - pg * p.page_size);
            slot = page < 0 || s >= p.num_slots ? -1 : (int32_t)s;
            p.rtt[row * p.rtt_stride + at] = slot;
        } else {
            slot = __ldg(p.rtt + row * p.rtt_stride + at);
            if (slot < 0 || slot >= p.num_slots) slot = -1;
        }
        if (slot < 0 && p.status) atomicOr(p.status, RX_DEV_BAD_SLOT);
        p.pos[t] = at;
        p.slots[t] = slot;
    }
}

}  // namespace

extern "C" int rx_step_maps(const int32_t *req_idx, const int32_t *prefix_len, const int32_t *new_len, int32_t batch,
                            int32_t *req_to_token, int64_t rtt_stride, const int32_t *pages, int64_t pages_stride,
                            int32_t page_size, int64_t num_slots, int32_t *qo_indptr, int32_t *seq_len, int32_t *pos,
                            int32_t *slots, int64_t max_tokens, int32_t *dev_status, void *stream)
{
    if (batch < 0 || max_tokens < 0 || max_tokens > INT32_MAX || !qo_indptr || rtt_stride <= 0 || rtt_stride > INT32_MAX ||
        num_slots <= 0 || num_slots > INT32_MAX || (batch > 0 && (!req_idx || !prefix_len || !new_len || !req_to_token)) ||
        (max_tokens > 0 && (!pos || !slots)))
        return rx_set_error(RX_ERR_INVALID, "rx_step_maps: invalid argument");
    if (seq_len && (seq_len == prefix_len || seq_len == new_len))
        return rx_set_error(RX_ERR_INVALID, "rx_step_maps: seq_len must not be one of the inputs");
    if (pages && (page_size <= 0 || pages_stride <= 0 || pages_stride > INT32_MAX))
        return rx_set_error(RX_ERR_INVALID, "rx_step_maps: pages of %d tokens, %lld a request", page_size, (long long)pages_stride);
    MapParams p{req_idx, prefix_len, new_len, batch, req_to_token, rtt_stride, pages, pages_stride, page_size, num_slots,
                rtt_stride, qo_indptr, seq_len, pos, slots, max_tokens, dev_status};
    if (pages && pages_stride * page_size < rtt_stride) p.positions = pages_stride * page_size;
    const int64_t share = (int64_t)kThreads * kTokens;
    const int64_t grid = max_tokens > share ? (max_tokens + share - 1) / share : 1;
    step_maps_kernel<<<(unsigned)grid, kThreads, 0, (cudaStream_t)stream>>>(p);
    RX_CUDA_CHECK(cudaGetLastError());
    return RX_OK;
}
