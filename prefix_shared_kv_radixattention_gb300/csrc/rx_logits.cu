// rx_logits.cu -- penalties for repeated tokens, biases and grammar masks on
// logits.
//
// For every id t of a logits row of request b, x = logits[t]:
//     y = seen ? (x > 0 ? x / repetition : x repetition) : x
//     y = y - frequency count;  y = count > 0 ? y - presence : y
//     y = y + sum of the request's biases of t;  out = allowed ? y : -inf
// with seen / count over the request's token list and, for a drafted tree,
// the drafted tokens on the row's path.
//
// The floor is one write of the fp32 row and one read of the logits that the
// mask allows: an element needs a handful of operations, so the work is a
// stream.  Few ids are touched by a penalty or a bias; the rest are copied
// (or become -inf).  A CTA takes a tile of consecutive ids for some rows of
// one request: it first counts the request's tokens that fall into its tile
// in shared memory (32-bit words: the count, a bit "in the prompt", a bit
// "has a bias"), with a bit map of the touched groups of four ids, then
// streams the rows through that table.  A group of four ids without an
// allowed one is not read at all.  A row's path is added to the table before
// the row and taken out after it.
#include <algorithm>
#include <math.h>

#include "rx_common.cuh"

namespace {

using bf16 = __nv_bfloat16;

constexpr int kThreads = 512;
constexpr int kUnroll = 4;                  // groups of four ids a thread has in flight
constexpr uint32_t kPrompt = 0x80000000u;   // the id is in the prompt
constexpr uint32_t kBias = 0x40000000u;     // the id has a bias
constexpr uint32_t kCount = 0x3FFFFFFFu;
constexpr int kMaxPath = 1024;              // drafted tokens of one request

struct LParams {
    rx_logits_rules r;
    const void *logits;
    int64_t stride;
    float *out;
    int64_t out_stride;
    int32_t rows, tile, words;
    int32_t *status;
};

// y of one touched id: c is its table word.
struct Penalty {
    float rep, freq, pres;
    const int32_t *btok;   // the request's biases, nb of them
    const float *bval;
    int64_t nb;

    __device__ float apply(float x, uint32_t c, int id) const
    {
        const uint32_t n = c & kCount;
        if (n || (c & kPrompt)) x = x > 0.f ? __fdiv_rn(x, rep) : __fmul_rn(x, rep);
        // the product is rounded before the difference, as the formula's steps are
        x = __fsub_rn(x, __fmul_rn(freq, (float)n));
        if (n) x = __fsub_rn(x, pres);
        if (c & kBias) {
            int64_t lo = 0, hi = nb;  // first entry at or above id
            while (lo < hi) {
                const int64_t mid = (lo + hi) >> 1;
                if (__ldg(btok + mid) < id) lo = mid + 1; else hi = mid;
            }
            if (lo < nb && __ldg(btok + lo) == id) {
                float s = __ldg(bval + lo);
                for (++lo; lo < nb && __ldg(btok + lo) == id; ++lo) s = __fadd_rn(s, __ldg(bval + lo));
                x = __fadd_rn(x, s);
            }
        }
        return x;
    }
};

template <bool BF16>
__device__ __forceinline__ float logit(const void *row, int id)
{
    if constexpr (BF16) return __bfloat162float(static_cast<const bf16 *>(row)[id]);
    else return static_cast<const float *>(row)[id];
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) logits_kernel(const __grid_constant__ LParams p)
{
    extern __shared__ uint32_t sm[];
    uint32_t *table = sm;                       // [tile]
    uint32_t *touched = sm + p.tile;            // a bit for each group of four ids
    const rx_logits_rules &r = p.r;
    const int b = blockIdx.y;
    const int lo = (int)blockIdx.x * p.tile, hi = min(r.vocab, lo + p.tile), n = hi - lo;
    int row0 = b, row1 = b + 1;
    if (r.qo_indptr) {
        row0 = __ldg(r.qo_indptr + b);
        row1 = __ldg(r.qo_indptr + b + 1);
    }
    const int tree = row1 - row0;
    if (tree == 0) return;
    if (row0 < 0 || tree < 0 || row1 > p.rows || (r.draft_tok && tree > kMaxPath) ||
        (r.draft_tok && r.tree_mask && (int64_t)tree > 32ll * r.tree_words)) {
        if (p.status && threadIdx.x == 0) atomicOr(p.status, RX_DEV_BAD_LEN);
        return;
    }
    if (row0 + (int)blockIdx.z >= row1) return;

    Penalty pen;
    pen.rep = r.repetition ? __ldg(r.repetition + b) : 1.f;
    pen.freq = r.frequency ? __ldg(r.frequency + b) : 0.f;
    pen.pres = r.presence ? __ldg(r.presence + b) : 0.f;
    const bool penal = pen.rep != 1.f || pen.freq != 0.f || pen.pres != 0.f;
    const int64_t b0 = r.bias_ptr ? __ldg(r.bias_ptr + b) : 0;
    pen.nb = r.bias_ptr ? __ldg(r.bias_ptr + b + 1) - b0 : 0;
    pen.btok = r.bias_tok + b0;
    pen.bval = r.bias_val + b0;

    for (int i = threadIdx.x; i < p.tile + p.tile / 128; i += kThreads) sm[i] = 0;
    __syncthreads();
    auto touch = [&](int t) { atomicOr(touched + (t >> 7), 1u << ((t >> 2) & 31)); };
    bool bad = false;
    // an id outside the vocabulary is reported by the CTAs of the first tile
    auto outside = [&](int t) {
        if (t >= 0 && t < r.vocab) return false;
        bad = true;
        return true;
    };
    if (r.hist) {
        const int64_t h0 = __ldg(r.hist_ptr + b), h1 = __ldg(r.hist_ptr + b + 1);
        const int64_t hp = h0 + (r.prompt_len ? __ldg(r.prompt_len + b) : 0);
        if (penal || lo == 0)  // neutral penalties: only the check of the ids
            for (int64_t i = h0 + threadIdx.x; i < h1; i += kThreads) {
                const int t = __ldg(r.hist + i);
                if (outside(t) || !penal || t < lo || t >= hi) continue;
                if (i < hp) atomicOr(table + (t - lo), kPrompt);
                else atomicAdd(table + (t - lo), 1u);
                touch(t - lo);
            }
    }
    for (int64_t i = threadIdx.x; i < pen.nb; i += kThreads) {
        const int t = __ldg(pen.btok + i);
        if (i > 0 && __ldg(pen.btok + i - 1) > t) bad = true;
        if (outside(t) || t < lo || t >= hi) continue;
        atomicOr(table + (t - lo), kBias);
        touch(t - lo);
    }

    for (int row = row0 + (int)blockIdx.z; row < row1; row += (int)gridDim.z) {
        // the drafted tokens on the row's path (sign +1: in, -1: out again)
        auto path = [&](uint32_t add) {
            if (!r.draft_tok || (!penal && lo != 0)) return;  // neutral penalties: only the check of the ids
            for (int j = threadIdx.x; j < tree; j += kThreads) {
                const bool on = r.tree_mask
                                    ? (__ldg(r.tree_mask + (int64_t)row * r.tree_words + (j >> 5)) >> (j & 31)) & 1u
                                    : j <= row - row0;
                if (!on) continue;
                const int t = __ldg(r.draft_tok + row0 + j);
                if (outside(t) || !penal || t < lo || t >= hi) continue;
                atomicAdd(table + (t - lo), add);
                touch(t - lo);
            }
        };
        path(1u);
        __syncthreads();
        const unsigned char *in = static_cast<const unsigned char *>(p.logits) + (int64_t)row * p.stride * (BF16 ? 2 : 4);
        float *out = p.out + (int64_t)row * p.out_stride;
        // the row's mask: null allows all; a row that is not there, nothing
        const uint32_t *allow = nullptr;
        bool none = false;
        if (r.allow) {
            const int a = __ldg(r.allow_row + row);
            if (a >= 0 && a < r.n_allow) {
                allow = r.allow + (int64_t)a * p.words;
            } else if (a != -1) {
                none = true;
                if (p.status && threadIdx.x == 0) atomicOr(p.status, RX_DEV_BAD_STATE);
            }
        }
        // groups of four ids; a row that does not start on 16 bytes (8 for
        // bf16) goes element by element
        const bool vec = (reinterpret_cast<uintptr_t>(in) & (BF16 ? 7 : 15)) == 0 &&
                         (reinterpret_cast<uintptr_t>(out) & 15) == 0;
        const int groups = vec ? n / 4 : 0;
        for (int g0 = threadIdx.x; g0 < groups; g0 += kThreads * kUnroll) {
            float4 x[kUnroll];
            uint32_t ok[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int g = g0 + u * kThreads;
                ok[u] = 0u;
                if (g >= groups) continue;
                const int id = lo + 4 * g;
                ok[u] = none ? 0u : allow ? (__ldg(allow + (id >> 5)) >> (id & 31)) & 15u : 15u;
                if (!ok[u]) continue;
                if constexpr (BF16) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(in + 2 * (int64_t)id);
                    x[u] = make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                                       __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
                } else {
                    x[u] = *reinterpret_cast<const float4 *>(in + 4 * (int64_t)id);
                }
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int g = g0 + u * kThreads;
                if (g >= groups) continue;
                const int id = lo + 4 * g;
                float y[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
                if (ok[u] && (touched[g >> 5] >> (g & 31)) & 1u) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t c = table[4 * g + k];
                        if (c) y[k] = pen.apply(y[k], c, id + k);
                    }
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (!((ok[u] >> k) & 1u)) y[k] = -INFINITY;
                *reinterpret_cast<float4 *>(out + id) = make_float4(y[0], y[1], y[2], y[3]);
            }
        }
        for (int i = groups * 4 + (int)threadIdx.x; i < n; i += kThreads) {
            const int id = lo + i;
            const bool ok = !none && (!allow || ((__ldg(allow + (id >> 5)) >> (id & 31)) & 1u));
            float y = -INFINITY;
            if (ok) {
                y = logit<BF16>(in, id);
                const uint32_t c = table[i];
                if (c) y = pen.apply(y, c, id);
            }
            out[id] = y;
        }
        __syncthreads();
        path(0xFFFFFFFFu);
    }
    if (bad && lo == 0 && p.status) atomicOr(p.status, RX_DEV_BAD_TOKEN);
}

int logits_num_sms()
{
    static int sms = 0;
    if (sms == 0) {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            sms = 152;
    }
    return sms;
}

}  // namespace

extern "C" int rx_logits_process(const rx_logits_rules *rules, const void *logits, int32_t logits_bf16,
                                 int64_t logits_stride, float *out, int64_t out_stride, int32_t rows,
                                 int32_t *dev_status, void *stream)
{
    if (!rules || rules->n_req < 0 || rules->vocab < 1 || rows < 0 || (logits_bf16 != 0 && logits_bf16 != 1))
        return rx_set_error(RX_ERR_INVALID, "rx_logits_process: invalid argument");
    const rx_logits_rules &r = *rules;
    if (!r.qo_indptr && rows != r.n_req)
        return rx_set_error(RX_ERR_INVALID, "rx_logits_process: %d rows for %d requests", rows, r.n_req);
    if (rows == 0 || r.n_req == 0) return RX_OK;
    if (!logits || !out) return rx_set_error(RX_ERR_INVALID, "rx_logits_process: null pointer");
    if (logits_stride < r.vocab || out_stride < r.vocab)
        return rx_set_error(RX_ERR_INVALID, "rx_logits_process: row strides %lld and %lld for %d ids",
                            (long long)logits_stride, (long long)out_stride, r.vocab);
    if ((reinterpret_cast<uintptr_t>(logits) & (logits_bf16 ? 1 : 3)) != 0 || (reinterpret_cast<uintptr_t>(out) & 3) != 0)
        return rx_set_error(RX_ERR_INVALID, "rx_logits_process: rows must start on an element");
    if (out == logits && (logits_bf16 || logits_stride != out_stride))
        return rx_set_error(RX_ERR_INVALID, "rx_logits_process: out may be logits only as fp32 of the same stride");
    if ((r.hist && !r.hist_ptr) || (r.bias_ptr && (!r.bias_tok || !r.bias_val)) ||
        (r.allow && (!r.allow_row || r.n_allow < 1)) || (r.draft_tok && !r.qo_indptr) ||
        (r.draft_tok && r.tree_mask && r.tree_words < 1))
        return rx_set_error(RX_ERR_INVALID, "rx_logits_process: a part of the rules is missing");
    if (r.n_req > 65535) return rx_set_error(RX_ERR_UNSUPPORTED, "rx_logits_process: %d requests (up to 65535)", r.n_req);
    LParams p{};
    p.r = r;
    p.logits = logits;
    p.stride = logits_stride;
    p.out = out;
    p.out_stride = out_stride;
    p.rows = rows;
    p.words = (r.vocab + 127) / 128 * 4;
    p.status = dev_status;
    // the largest tile (its list of tokens is read once a tile) that still
    // gives two CTAs an SM over all requests
    const int64_t want = 2 * (int64_t)logits_num_sms();
    int tile = 16384;
    while (tile > 2048 && (int64_t)((r.vocab + tile - 1) / tile) * r.n_req < want) tile /= 2;
    p.tile = tile;
    const int tiles = (r.vocab + tile - 1) / tile;
    // few requests with several rows each: the rows of one are shared out
    int64_t slices = 1;
    if (r.qo_indptr) {
        const int64_t per = (rows + r.n_req - 1) / r.n_req;
        slices = std::min<int64_t>(per, (want + (int64_t)tiles * r.n_req - 1) / ((int64_t)tiles * r.n_req));
        slices = std::max<int64_t>(1, std::min<int64_t>(slices, 65535));
    }
    const size_t smem = (size_t)(tile + tile / 128) * sizeof(uint32_t);
    auto kernel = logits_bf16 ? logits_kernel<true> : logits_kernel<false>;
    // per device and function; cheap, and right whichever device is current
    RX_CUDA_CHECK(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)((16384 + 128) * sizeof(uint32_t))));
    kernel<<<dim3((unsigned)tiles, (unsigned)r.n_req, (unsigned)slices), kThreads, smem, (cudaStream_t)stream>>>(p);
    RX_CUDA_CHECK(cudaGetLastError());
    return RX_OK;
}
