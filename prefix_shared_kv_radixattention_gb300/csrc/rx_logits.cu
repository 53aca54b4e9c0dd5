// rx_logits.cu -- penalties for repeated tokens, biases and grammar masks on
// logits.
//
// For every id t of a logits row of request b, x = logits[t]:
//     y = seen ? (x > 0 ? x / repetition : x repetition) : x
//     y = count > 0 ? (y - frequency count) - presence : y
//     y = y + sum of the request's biases of t;  out = allowed ? y : -inf
// with seen / count over the request's token list and, for a drafted tree,
// the drafted tokens on the row's path.
//
// The floor is one write of the fp32 row and one read of the logits that the
// mask allows.  A CTA takes a tile of the ids of one request and all of its rows
// (with few requests, some of them):
//
//   - the request's words for the tile's ids (the count, a bit "in the prompt",
//     "has a bias", "is drafted") are made in shared memory: each CTA reads all
//     of the request's tokens and counts those of its tile, the others cost a few
//     instructions;
//   - row by row, a thread takes groups of four ids: the logits (not read where
//     the mask allows none of the four), their words, the values.  The next
//     row's logits are on their way meanwhile.
//
// So the rows move once, in whole sectors (rows that start off 16 bytes, 8 for
// bf16 logits, go id by id and none is fetched ahead: 64 fp32 rows of 50,257 ids
// take 29 us, of 50,256 15).  What bounds it is the instructions:
// 192 drafted rows of 128,256 bf16 logits over 32,768 tokens a request take 55
// us (2.8 times the 20 us of their bytes) and 34 million warp instructions at
// 2.4 a cycle, a quarter of them the counting, which every tile's CTA does for
// all of the tokens, the rest some 130 for a warp's 128 ids (the touched ones of
// a group one after the other: 69 us).  64 rows of fp32 logits take 31 us, where
// the chain of loads and barriers before the first row (two thirds of a CTA's
// time) counts, one row of 32,000 ids 5.8 us.
//
// A copy of the rows followed by a kernel for the listed touched ids alone took
// 92, 37 and 5.6 us: partial sectors, and the common tokens in a few CTAs.  The
// list spread over a cluster through its shared memory, 82, 38 and 6.8 us;
// through global memory, a third kernel, 61, 45 and 14 us.
//
// In place, only groups with a forbidden or a touched id are read and written.
#include <algorithm>
#include <climits>
#include <math.h>

#include <type_traits>

#include "rx_common.cuh"

namespace {

using bf16 = __nv_bfloat16;

constexpr int kThreads = 512;
constexpr int kVecs = 4;                    // groups of four ids of a thread
constexpr int kTile = kThreads * kVecs * 4; // ids of a CTA, at most
constexpr uint32_t kPrompt = 0x80000000u;   // the id is in the prompt
constexpr uint32_t kBias = 0x40000000u;     // the id has a bias
constexpr uint32_t kDraft = 0x20000000u;    // the id is a drafted token
constexpr uint32_t kCount = 0x1FFFFFFFu;
constexpr int kMaxPath = 1024;              // drafted tokens of one request

struct LParams {
    rx_logits_rules r;
    const void *logits;
    int64_t stride;
    float *out;
    int64_t out_stride;
    int32_t rows, words;
    int32_t *status;
};

// One request's rules; false where it is flagged (those of its rows that there
// are then get their mask only).
struct Request {
    int row0, tree;          // its rows
    float rep, freq, pres, inv;   // inv: 1 / rep
    bool plain_rep;               // rep is in divide's range
    bool penal;              // any of them does anything
    int64_t bias0, nbias;
    int64_t hist0, nhist;
    int prompt;              // of them the prompt's

    __device__ __forceinline__ bool load(const LParams &p, int b)
    {
        const rx_logits_rules &r = p.r;
        int row1 = b + 1;
        row0 = b;
        if (r.qo_indptr) {
            row0 = __ldg(r.qo_indptr + b);
            row1 = __ldg(r.qo_indptr + b + 1);
        }
        rep = r.repetition ? __ldg(r.repetition + b) : 1.f;
        freq = r.frequency ? __ldg(r.frequency + b) : 0.f;
        pres = r.presence ? __ldg(r.presence + b) : 0.f;
        inv = __frcp_rn(rep);
        plain_rep = rep >= 0x1p-60f && rep <= 0x1p60f;
        bias0 = r.bias_ptr ? __ldg(r.bias_ptr + b) : 0;
        nbias = r.bias_ptr ? __ldg(r.bias_ptr + b + 1) - bias0 : 0;
        hist0 = r.hist ? __ldg(r.hist_ptr + b) : 0;
        nhist = r.hist ? __ldg(r.hist_ptr + b + 1) - hist0 : 0;
        prompt = r.prompt_len ? __ldg(r.prompt_len + b) : 0;
        penal = rep != 1.f || freq != 0.f || pres != 0.f;
        tree = row1 - row0;
        if (row0 >= 0 && tree >= 0 && row1 <= p.rows && nhist >= 0 && nhist <= (int64_t)kCount - kMaxPath && nbias >= 0 &&
            !(r.draft_tok && (tree > kMaxPath || (r.tree_mask && (int64_t)tree > 32ll * r.tree_words))))
            return true;
        if (p.status && threadIdx.x == 0) atomicOr(p.status, RX_DEV_BAD_LEN);
        row0 = max(row0, 0);
        tree = max(min(row1, p.rows) - row0, 0);
        return false;
    }
    // x / rep of two values, correctly rounded, for 2^-60 <= rep <= 2^60 and x
    // <= 0 (any value: unused) or 2^-40 <= x <= 2^40: with 1 / rep correctly
    // rounded, the first step is within one place of the quotient and the
    // second rounds it correctly (Markstein, IBM J. Res. Dev. 34, 1990).  Five
    // packed operations for two quotients, where the general division takes
    // some ten for one.
    __device__ __forceinline__ uint64_t divide(uint64_t x) const
    {
        const uint64_t i = rx::f2(inv, inv), m = rx::f2(-rep, -rep);
        uint64_t y = rx::f2_mul(x, i);
        y = rx::f2_fma(rx::f2_fma(m, y, x), i, y);
        return rx::f2_fma(rx::f2_fma(m, y, x), i, y);
    }
    // the values of two ids with words c0 and c1, biases apart, from their
    // logits x and quotients d
    __device__ __forceinline__ void penalise(float &x0, float &x1, float d0, float d1, uint32_t c0, uint32_t c1) const
    {
        float y0, y1, z0, z1;
        rx::f2_split(rx::f2_mul(rx::f2(x0, x1), rx::f2(rep, rep)), y0, y1);
        y0 = x0 > 0.f ? d0 : y0;
        y1 = x1 > 0.f ? d1 : y1;
        y0 = (c0 & (kPrompt | kCount)) ? y0 : x0;
        y1 = (c1 & (kPrompt | kCount)) ? y1 : x1;
        const uint32_t n0 = c0 & kCount, n1 = c1 & kCount;
        // the product is rounded before the difference, as the formula's steps
        // are (a packed product would be joined with the packed difference)
        const uint64_t fn = rx::f2(__fmul_rn(-freq, (float)n0), __fmul_rn(-freq, (float)n1));
        rx::f2_split(rx::f2_add(rx::f2_add(rx::f2(y0, y1), fn), rx::f2(-pres, -pres)), z0, z1);
        x0 = n0 ? z0 : y0;
        x1 = n1 ? z1 : y1;
    }
};

// Out of line: hardly ever called.
__device__ __noinline__ float4 divide_any(float4 x, float rep)
{
    return make_float4(__fdiv_rn(x.x, rep), __fdiv_rn(x.y, rep), __fdiv_rn(x.z, rep), __fdiv_rn(x.w, rep));
}

// Grid: x = tiles, y = requests, z = shares of a request's rows.  IN_PLACE: out
// is logits.
template <bool BF16, bool IN_PLACE>
__global__ void __launch_bounds__(kThreads, 2) logits_kernel(const __grid_constant__ LParams p, int tile, bool touched)
{
    extern __shared__ __align__(16) uint32_t table[];                // [tile] words
    uint8_t *prompt = reinterpret_cast<uint8_t *>(table + tile);    // [tile] the id is in the prompt
    float *bias = reinterpret_cast<float *>(prompt + tile);         // [tile] the sum of its biases, where it has some
    const rx_logits_rules &r = p.r;
    const int b = blockIdx.y, lo = (int)blockIdx.x * tile, n = min(r.vocab - lo, tile);
    Request q;
    const bool listed = q.load(p, b) && touched;

    // a thread's groups of four are 4 (threadIdx.x + u kThreads) of the tile
    const int i0 = 4 * threadIdx.x, step = (int)gridDim.z;
    using Raw = std::conditional_t<BF16, uint2, float4>;
    Raw x[kVecs];
    uint32_t hot = 0;    // bit u: group u has an id whose word is not 0
    // the tile of the request's row k
    auto in = [&](int k) {
        return static_cast<const unsigned char *>(p.logits) + ((int64_t)(q.row0 + k) * p.stride + lo) * (BF16 ? 2 : 4);
    };
    auto out = [&](int k) { return p.out + (int64_t)(q.row0 + k) * p.out_stride + lo; };
    // its groups of four start on 16 bytes (8 of bf16)
    auto aligned = [&](int k) {
        return (reinterpret_cast<uintptr_t>(in(k)) & (BF16 ? 7 : 15)) == 0 && (reinterpret_cast<uintptr_t>(out(k)) & 15) == 0;
    };
    auto one = [&](int k, int i) {  // a plain load: out may be logits
        return BF16 ? __bfloat162float(reinterpret_cast<const bf16 *>(in(k))[i]) : reinterpret_cast<const float *>(in(k))[i];
    };
    // row k's mask: its entry of allow_row (-1: all ids; a row that is not there
    // allows none), from which the words of this thread's groups, from which
    // bits 4 u ..: the allowed ids of group u
    auto mask_row = [&](int k) { return r.allow && k < q.tree ? __ldg(r.allow_row + q.row0 + k) : -1; };
    auto mask_word = [&](int a, int i) {
        if (a >= 0 && a < r.n_allow) return __ldg(r.allow + (int64_t)a * p.words + ((lo + i) >> 5));
        return a == -1 ? ~0u : 0u;
    };
    auto mask_words = [&](int a, uint32_t (&w)[kVecs]) {
#pragma unroll
        for (int u = 0; u < kVecs; ++u) {
            const int i = i0 + 4 * kThreads * u;
            w[u] = i + 4 <= n ? mask_word(a, i) : 0u;
        }
    };
    auto pack = [&](const uint32_t (&w)[kVecs]) {
        uint32_t m = 0;
#pragma unroll
        for (int u = 0; u < kVecs; ++u) m |= (w[u] >> (i0 & 31) & 15u) << (4 * u);
        return m;
    };
    auto fetch = [&](int k, bool vec, uint32_t m, int u) {
        m = m >> (4 * u) & 15u;
        x[u] = {};
        if (vec && m != 0u && (!IN_PLACE || m != 15u || ((hot >> u) & 1u)))
            x[u] = *reinterpret_cast<const Raw *>(in(k) + (BF16 ? 2 : 4) * (i0 + 4 * kThreads * u));
    };
    int k = blockIdx.z;
    if (k >= q.tree) return;
    // rows ahead: entries of allow_row three, mask words two, logits one
    int a0 = mask_row(k), a1 = mask_row(k + step), a2 = mask_row(k + 2 * step);
    uint32_t word[kVecs];
    const bool vec0 = aligned(k);

    // this thread's drafted tokens (threadIdx.x and the one kThreads behind): their places in the tile
    static_assert(kMaxPath <= 2 * kThreads, "drafted tokens of a thread");
    int drafted[2] = {-1, -1};
    bool paths = false;
    // the biases' ids: this thread's first and its neighbours' (-1: there is none)
    auto id_at = [&](int64_t i) { return i >= 0 && i < q.nbias ? __ldg(r.bias_tok + q.bias0 + i) : -1; };
    int t = -1, before = -1, next = -1;
    if (listed) {
        for (int i = threadIdx.x; i < tile / 4; i += kThreads) reinterpret_cast<uint4 *>(table)[i] = make_uint4(0, 0, 0, 0);
        for (int i = threadIdx.x; i < tile / 16; i += kThreads) reinterpret_cast<uint4 *>(prompt)[i] = make_uint4(0, 0, 0, 0);
        t = id_at(threadIdx.x);
        before = id_at((int64_t)threadIdx.x - 1);
        next = id_at((int64_t)threadIdx.x + 1);
    }
    mask_words(a0, word);
    // ids outside the vocabulary are reported by the first tile
    const bool first = lo == 0 && blockIdx.z == 0;
    bool bad = false;
    if (listed) {
        __syncthreads();
        const int32_t *h = r.hist + q.hist0;
        const uint32_t ids = q.penal ? (uint32_t)n : 0u;
        const int len = q.penal || first ? (int)q.nhist : 0;  // neutral penalties: only the check of the ids
        // a prompt's token needs no more than a mark
        auto mark = [&](int t) {
            const uint32_t d = (uint32_t)t - (uint32_t)lo;
            if (d < ids) prompt[d] = 1;
        };
        auto count = [&](int t) {
            const uint32_t d = (uint32_t)t - (uint32_t)lo;
            if (d < ids) atomicAdd(table + d, 1u);
        };
        auto token = [&](int t, int i) {
            if (first) bad |= (uint32_t)t >= (uint32_t)r.vocab;
            if (i < q.prompt) mark(t);
            else count(t);
        };
        // single tokens up to a 16-byte boundary, four at a time, the rest
        const int head = min(len, (int)((16 - (reinterpret_cast<uintptr_t>(h) & 15)) >> 2 & 3)), n4 = (len - head) / 4;
        const int4 *h4 = reinterpret_cast<const int4 *>(h + head);
        constexpr int U = 4;
        for (int i = threadIdx.x; i < n4; i += U * kThreads) {
            int4 x[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i + u * kThreads < n4) x[u] = __ldg(h4 + i + u * kThreads);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (i + u * kThreads >= n4) break;
                const int at = head + 4 * (i + u * kThreads);
                if (!first && at + 3 < q.prompt) {
                    mark(x[u].x);
                    mark(x[u].y);
                    mark(x[u].z);
                    mark(x[u].w);
                } else if (!first && at >= q.prompt) {
                    count(x[u].x);
                    count(x[u].y);
                    count(x[u].z);
                    count(x[u].w);
                } else {
                    token(x[u].x, at);
                    token(x[u].y, at + 1);
                    token(x[u].z, at + 2);
                    token(x[u].w, at + 3);
                }
            }
        }
        // at most three before the first four and three behind the last
        const int at = (int)threadIdx.x < head ? threadIdx.x : 4 * n4 + (int)threadIdx.x;
        if (threadIdx.x < 8 && at < len) token(__ldg(h + at), at);
    }
    uint32_t m = pack(word);
    bool vec = vec0;
    if (!IN_PLACE) {
#pragma unroll
        for (int u = 0; u < kVecs; ++u) fetch(k, vec, m, u);
    }
    mask_words(a1, word);
    if (listed) {
        for (int64_t i = threadIdx.x; i < q.nbias; i += kThreads) {
            if (i >= kThreads) {
                t = id_at(i);
                before = id_at(i - 1);
                next = id_at(i + 1);
            }
            bad |= (i > 0 && before > t) || (uint32_t)t >= (uint32_t)r.vocab;
            const uint32_t d = (uint32_t)t - (uint32_t)lo;
            if (d >= (uint32_t)n || (i > 0 && before == t)) continue;
            float sum = __ldg(r.bias_val + q.bias0 + i);
            for (int64_t j = i + 1; next == t; ++j) {  // the same id again
                sum = __fadd_rn(sum, __ldg(r.bias_val + q.bias0 + j));
                next = id_at(j + 1);
            }
            bias[d] = sum;
            atomicOr(table + d, kBias);
        }
        if (r.draft_tok) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int node = (int)threadIdx.x + j * kThreads;
                if (node >= q.tree) break;
                const int t = __ldg(r.draft_tok + q.row0 + node);
                bad |= (uint32_t)t >= (uint32_t)r.vocab;
                if (q.penal && (uint32_t)t - (uint32_t)lo < (uint32_t)n) {
                    drafted[j] = t - lo;
                    atomicOr(table + drafted[j], kDraft);
                }
            }
        }
        if (bad && first && p.status) atomicOr(p.status, RX_DEV_BAD_TOKEN);
        // drafted tokens in this tile: the rows' paths count
        paths = __syncthreads_or(drafted[0] >= 0 || drafted[1] >= 0);
        uint4 *words = reinterpret_cast<uint4 *>(table);
#pragma unroll
        for (int u = 0; u < kVecs; ++u) {
            const int g = threadIdx.x + kThreads * u;
            if (4 * g >= tile) break;
            uint4 v = words[g];
            const uint32_t seen = reinterpret_cast<const uint32_t *>(prompt)[g];
            if (seen) {
                v.x |= seen << 31;
                v.y |= (seen & 0x100u) << 23;
                v.z |= (seen & 0x10000u) << 15;
                v.w |= (seen & 0x1000000u) << 7;
                words[g] = v;
            }
            if (v.x | v.y | v.z | v.w) hot |= 1u << u;
        }
        __syncthreads();  // single ids' words are read by other threads
    }
    if (IN_PLACE) {
#pragma unroll
        for (int u = 0; u < kVecs; ++u) fetch(k, vec, m, u);
    }
    uint32_t ahead = pack(word);
    // the values of ids i .. i + 3 of the tile with words c
    auto process = [&](float4 v, uint4 c, int i) {
        // the quotients' range: the largest value, and the least bits (the
        // positive values'; a zero takes the general division)
        const float top = fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w));
        const uint32_t low = min(min(__float_as_uint(v.x), __float_as_uint(v.y)), min(__float_as_uint(v.z), __float_as_uint(v.w)));
        float4 d;
        rx::f2_split(q.divide(rx::f2(v.x, v.y)), d.x, d.y);
        rx::f2_split(q.divide(rx::f2(v.z, v.w)), d.z, d.w);
        if (!(q.plain_rep && top <= 0x1p40f && low >= 0x2B800000u)) d = divide_any(v, q.rep);  // 2^-40
        q.penalise(v.x, v.y, d.x, d.y, c.x, c.y);
        q.penalise(v.z, v.w, d.z, d.w, c.z, c.w);
        if ((c.x | c.y | c.z | c.w) & kBias) {
            if (c.x & kBias) v.x = __fadd_rn(v.x, bias[i]);
            if (c.y & kBias) v.y = __fadd_rn(v.y, bias[i + 1]);
            if (c.z & kBias) v.z = __fadd_rn(v.z, bias[i + 2]);
            if (c.w & kBias) v.w = __fadd_rn(v.w, bias[i + 3]);
        }
        return v;
    };
    // which of this thread's drafted tokens are on row k's path: its mask words
    // (of the row after the one at hand, so that nobody waits for them)
    uint32_t path[2];
    auto path_words = [&](int k) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int at = (int)threadIdx.x + j * kThreads;
            path[j] = 0;
            if (drafted[j] < 0 || k >= q.tree) continue;
            if (r.tree_mask) path[j] = __ldg(r.tree_mask + (int64_t)(q.row0 + k) * r.tree_words + (at >> 5));
            else path[j] = at <= k ? ~0u : 0u;
        }
    };
    bool counted[2] = {false, false};  // the token is counted in its word
    if (paths) path_words(k);
    for (;;) {
        if (a0 != -1 && (a0 < 0 || a0 >= r.n_allow) && threadIdx.x == 0 && p.status) atomicOr(p.status, RX_DEV_BAD_STATE);
        if (paths) {  // the words of the path's tokens
            __syncthreads();  // the row before has been worked off
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const bool on = (path[j] >> (threadIdx.x & 31)) & 1u;
                if (on != counted[j]) atomicAdd(table + drafted[j], on ? 1u : ~0u);
                counted[j] = on;
            }
            __syncthreads();
            path_words(k + step);
        }
        const bool more = k + step < q.tree, vec1 = more && aligned(k + step);
        mask_words(a2, word);
        const int a3 = mask_row(k + 3 * step);
#pragma unroll
        for (int u = 0; u < kVecs; ++u) {
            const int i = i0 + 4 * kThreads * u;
            float4 v;
            if constexpr (BF16)
                v = make_float4(__uint_as_float(x[u].x << 16), __uint_as_float(x[u].x & 0xFFFF0000u),
                                __uint_as_float(x[u].y << 16), __uint_as_float(x[u].y & 0xFFFF0000u));
            else
                v = x[u];
            const uint32_t mu = m >> (4 * u) & 15u;
            const bool touches = (hot >> u) & 1u;
            if (mu != 0u && touches) v = process(v, reinterpret_cast<const uint4 *>(table)[threadIdx.x + kThreads * u], i);
            if (vec && i + 4 <= n && (!IN_PLACE || mu != 15u || touches))
                *reinterpret_cast<float4 *>(out(k) + i) =
                    make_float4(mu & 1u ? v.x : -INFINITY, mu & 2u ? v.y : -INFINITY, mu & 4u ? v.z : -INFINITY,
                                mu & 8u ? v.w : -INFINITY);
            fetch(k + step, vec1, ahead, u);
        }
        // single ids: the rest behind the last four, or the whole of a row that is not aligned
        for (int i = (vec ? n / 4 * 4 : 0) + (int)threadIdx.x; i < n; i += kThreads) {
            const bool ok = mask_word(a0, i) >> (i & 31) & 1u;
            const uint32_t c = listed ? table[i] : 0u;
            float y = -INFINITY;
            if (ok && (!IN_PLACE || c)) {
                y = one(k, i);
                if (c) y = process(make_float4(y, 1.f, 1.f, 1.f), make_uint4(c, 0u, 0u, 0u), i).x;
            }
            if (!IN_PLACE || c || !ok) out(k)[i] = y;
        }
        if (!more) return;
        k += step;
        vec = vec1;
        m = ahead;
        ahead = pack(word);
        a0 = a1;
        a1 = a2;
        a2 = a3;
    }
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
    if (r.vocab > (1 << 30)) return rx_set_error(RX_ERR_UNSUPPORTED, "rx_logits_process: vocabulary of %d ids", r.vocab);
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
    cudaStream_t st = (cudaStream_t)stream;
    const bool in_place = out == logits, touched = r.hist || r.bias_ptr || r.draft_tok;
    if (in_place && !touched && !r.allow) return RX_OK;
    const int tile = kTile;
    const int64_t tiles = (r.vocab + (int64_t)tile - 1) / tile;
    // four CTAs an SM (two at a time): with fewer, a request's rows are dealt out
    // to several, which all count.  16 requests of 8 to 16 rows of 128,256 ids:
    // 60 us with 1 share, 57 with 2, 59 with 3, 61 with 4 (55 with 2 since)
    const int64_t shares = std::max<int64_t>(1, std::min<int64_t>(4 * rx_num_sms() / (tiles * r.n_req), rows));
    const size_t smem = (size_t)tile * (r.bias_ptr ? 9 : touched ? 5 : 0);
    auto kernel = in_place ? logits_kernel<false, true> : logits_bf16 ? logits_kernel<true, false> : logits_kernel<false, false>;
    // per device and function; cheap, and right whichever device is current
    if (smem > 48 * 1024) RX_CUDA_CHECK(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
    kernel<<<dim3((unsigned)tiles, (unsigned)r.n_req, (unsigned)shares), kThreads, smem, st>>>(p, tile, touched);
    RX_CUDA_CHECK(cudaGetLastError());
    return RX_OK;
}
