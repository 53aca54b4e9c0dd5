// rx_tree.cu -- attention of drafted token trees over the slot pool, on the
// 5th-generation tensor cores (tcgen05.mma, accumulators in TMEM).
//
// Drafted token i of request b sees the request's whole prefix (positions
// 0 .. P_b - 1) and, of the drafted tokens (positions P_b + j), those whose
// bit j is set in its mask row:
//     s_j = sm_scale q . K[slot_j],  o = sum_seen softmax(s)_j V[slot_j],
//     lse = log sum_seen exp(s_j);   nothing seen: o = 0, lse = -inf.
//
// What bounds it: T drafted tokens times the G q heads of a kv head are a few
// dozen to a few hundred query rows, fewer than the 280 or so flops a byte
// that this GPU needs to be compute bound: the K and V rows' bytes are the
// floor.  So:
//
//   - the rows of one kv head are one tensor-core tile of 128 rows (M), padded
//     (an unused row costs nothing but its share of the MMA, which has time to
//     spare), and every K/V tile of 128 positions is read once for all of them;
//   - K/V rows are gathered through the slot list by producer warps in 16-byte
//     asynchronous copies that land in the swizzled tile that the tensor core
//     reads (see producer()).  Rows of 256 bytes at random slots stream at 6.7
//     TB/s this way with 64 KB in flight an SM (2.9 TB/s as bulk copies, 2.8
//     TB/s through three warps), so no copy of the context is needed first;
//   - the work is cut evenly: the (kv head, request, row tile, position tile)
//     units are one long list of which every CTA takes a contiguous share; a
//     (kv head, request, row tile) cut by a CTA's end leaves fp32 partial
//     results that a second kernel joins by the log-sum-exp identity.  The
//     heads are outermost, so with 8 heads on 152 SMs nineteen CTAs walk each
//     head in step and the rows of one slot are read at about the same time;
//   - four softmax warps a row tile (one row a thread) take the scores S = Q K^T of a tile
//     from TMEM into registers at once, which frees S for the next tile's, and
//     write P to a TMEM buffer of its own, from where O += P V reads it: the
//     tensor core works on the tiles before and after meanwhile.
//
// All lengths are read on the device, by every CTA for itself: a scan of the
// batch's lengths in shared memory finds its share.
//
// Measured, with what is left: 16 requests of up to 32,768 positions, 64/8
// heads of 128, 229 us, 6.8 TB/s of the rows read (a shared prefix is read once
// a request; read once in all it would be 164 us); 64 of 1,281, 32/32 heads,
// 211 us (149 us of bytes; four of a tile's 128 rows are used, and a softmax
// warp takes 2,300 cycles for a tile however few rows it has); E4M3 pools, 16 of
// up to 32,768, 32/8 heads, 295 us (119 us of bytes: the softmax warps' 3,300
// cycles a tile, two of the four with rows, with the producers' 2,500 for K and
// 2,900 for V close behind; a part of the exponentials on the multiply-add units, 368 us, or the
// rows put in twice and the tiles' positions, 382 us, or the tiles, 325 us,
// shared between the copies were no faster: the warps that got less to do took
// as much longer for it, so it is the SM's units that are shared); trees of
// 64 tokens, 64/8 heads, 8 requests, 121 us (42 us of tensor-core time: 4,000
// cycles for two row tiles, half of them the softmax, a quarter its waits for
// S); one request of 333 positions 13 us: 3 until the roles start, 3.5 until the
// first scores, 4 until the segment's end, 2 for the merge.
#include <math.h>

#include <algorithm>
#include <climits>
#include <type_traits>

#include "rx_common.cuh"
#include "rx_pipe.cuh"

namespace {

using bf16 = __nv_bfloat16;
using rx::sw128;
using rx::u2f;
using rx::wait_or_abort;
using rx::warp_wait;

constexpr int kMaxTree = 1024;
constexpr int kCtas = 152;           // CTAs of a call: one an SM
constexpr int kRows = 128;           // query rows of a row tile (MMA M)
constexpr int kMaxNt = 2;            // row tiles that share a K/V tile
constexpr int kBN = 128;             // positions of a K/V tile
constexpr int kStages = 2;           // K ring and V ring depth
constexpr int kSegs = 4;             // segments handed out ahead
constexpr int kMaskT = 128;          // trees up to this size have their mask words in shared memory
constexpr int kRing = 4;             // score scales kept (see query_loader)
constexpr int kCodeBufs = 3;         // FP8: half tiles of codes in flight, for K and for V
// The roles of the warps: for each row tile four softmax warps, one query row a
// thread; producers for K and as many for V; one each that loads the query rows,
// issues S = Q K^T, hands out the segments, issues the other product.
template <int NT>
struct Ro {
    static constexpr int SOFT = 4 * NT, PROD = NT == 1 ? 8 : 4;
    static constexpr int ROWS = kBN / PROD;              // rows of a tile each producer warp gathers
    static constexpr int Q = SOFT + 2 * PROD, MMA = Q + 1, SCHED = Q + 2, PV = Q + 3;
    static constexpr int THREADS = 32 * (Q + 4);
    // registers a thread, by role (a softmax thread holds a row's 128 scores):
    // 128 x 192 + 640 x 56 of the 768 x 80 launched; with two row tiles
    // 256 x 168 + 384 x 48 of 640 x 96
    static constexpr int R_SOFT = NT == 1 ? 192 : 168, R_REST = NT == 1 ? 56 : 48, R_LAUNCH = NT == 1 ? 80 : 96;
    static_assert(32 * (SOFT * R_SOFT + (2 * PROD + 4) * R_REST) <= THREADS * R_LAUNCH,
                  "a share is granted out of the launched registers only");
    static_assert(THREADS * R_LAUNCH <= 65536, "registers of an SM");
};
// TMEM: an O for each row tile, then S buffers (two; one beside two O), then
// two P of 64 columns (16-bit pairs)
constexpr uint32_t kTmemCols = 512;
template <int NT>
struct Tm {
    static __device__ __forceinline__ uint32_t o(int t) { return t * 128; }
    static __device__ __forceinline__ uint32_t s(int b) { return NT * 128 + (NT == 1 ? b * 128 : 0); }
    static __device__ __forceinline__ uint32_t p(int b) { return 384 + b * 64; }
};
// An item's S, P and product barriers and buffers: with one row tile the items
// take turns at two; with two row tiles each has its own (but one S for both).
// c: which item of its row tile it is.
template <int NT>
struct Turn {
    int b, phase;
    __device__ __forceinline__ Turn(int t, int c) : b(NT == 1 ? c & 1 : t), phase(NT == 1 ? c >> 1 : c) {}
};
constexpr float kRescale = 8.f;      // log2 units the running max may lag
constexpr int kMergeThreads = 128;
constexpr int kMergeRows = kMergeThreads / 32;  // rows of one merge CTA

// A segment: the position tiles [j0, j1) of a (kv head g, request, row tiles)
// that are this CTA's.
struct Seg {
    int g, j0, j1;
    int P, T;        // the request's prefix and drafted tokens
    int row;         // of req_to_token
    int node, ntok;  // the rows' drafted tokens: node .. node + ntok - 1 of the tree,
    int tok;         //   the first of them at this query row
    int nt;          // row tiles: 1 or 2
    int whole;       // every tile of the context: the result is final
    int last;        // the CTA's last segment
};

template <int D, bool F8>
struct TL {
    static constexpr int NB = D / 64;             // 128-byte column blocks of a row
    static constexpr int BLK = kRows * 128;       // bytes of one column block of a tile
    // query buffers: two for bf16 pools (of segments in turn, or of a segment's
    // row tiles); one for FP8 pools, whose codes need the room
    static constexpr int QB = F8 ? 1 : 2;
    static constexpr int CODE = F8 ? kBN * D / 2 : 0;  // bytes of half a tile of codes
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = OFF_Q + QB * NB * BLK;
    static constexpr int OFF_V = OFF_K + kStages * NB * BLK;
    static constexpr int OFF_CODE = OFF_V + kStages * NB * BLK;
    static constexpr int OFF_NF = OFF_CODE + 2 * kCodeBufs * CODE;    // kSegs x 32 words
    static constexpr int OFF_QS = OFF_NF + kSegs * 32 * 4;            // kRing x 128 floats
    static constexpr int OFF_MASK = OFF_QS + kRing * kRows * 4;       // kSegs x 128 tokens x 4 words;
    static constexpr int MASK = kSegs * kMaskT * (kMaskT / 32) * 4;   //   before them, the scan of the lengths
    static_assert((Ro<1>::THREADS + 1) * 8 <= MASK && (Ro<2>::THREADS + 1) * 8 <= MASK, "room for the scan");
    static constexpr int OFF_SEG = OFF_MASK + MASK;
    static constexpr int OFF_BAR = OFF_SEG + kSegs * 64;
    static constexpr int B_KFULL = 0, B_KEMPTY = B_KFULL + kStages, B_VFULL = B_KEMPTY + kStages,
                         B_VEMPTY = B_VFULL + kStages, B_QFULL = B_VEMPTY + kStages, B_QEMPTY = B_QFULL + QB,
                         B_SFULL = B_QEMPTY + QB, B_SEMPTY = B_SFULL + 2, B_PFULL = B_SEMPTY + 2, B_PVDONE = B_PFULL + 2,
                         B_OEMPTY = B_PVDONE + 2, B_SEGFULL = B_OEMPTY + 2, B_SEGEMPTY = B_SEGFULL + kSegs,
                         B_FINAL = B_SEGEMPTY + kSegs, N_BAR = B_FINAL + 2;
    static constexpr int OFF_TMEM = OFF_BAR + N_BAR * 8;
    static constexpr int OFF_ABORT = OFF_TMEM + 8;
    static constexpr int OFF_START = OFF_ABORT + 8;                   // Start
    static constexpr int BYTES = OFF_START + 32 + 1024;               // + room to align the base to 1024
};
static_assert(sizeof(Seg) <= 64, "room of a segment");
static_assert(TL<128, false>::BYTES <= 226 * 1024 && TL<128, true>::BYTES <= 226 * 1024, "shared memory budget");
static_assert(TL<128, false>::OFF_MASK % 16 == 0 && TL<128, false>::OFF_BAR % 8 == 0, "alignment");

struct TParams {
    const bf16 *q;
    bf16 *o;
    float *lse;
    const unsigned char *k;
    const unsigned char *v;
    int64_t num_slots;
    int hq, hkv, G;
    int tb;                 // drafted tokens of a row tile: 128 / G
    int nt;                 // row tiles that share a K/V tile
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
    float *part_o;      // [2 kCtas][128 nt][D] partial results, normalised
    float *part_l;      // [2 kCtas][128 nt] their log2-sum-exps
    struct Cut *cuts;   // [kCtas] what the merge has to do
    int32_t *status;
};

// ---------------------------------------------------------------------------
// the list of work
// ---------------------------------------------------------------------------

// The list is (kv head g, request b, group qt of nt row tiles, position tile
// j), j innermost; a unit is one entry.
struct Req {
    int T, P;
    int row;          // of req_to_token
    int tok;          // its first query row
    int ntiles, nqt;  // 0 where there is nothing to do (no drafted token, or lengths out of range)

    __device__ __forceinline__ int64_t units() const { return (int64_t)ntiles * nqt; }
};

__device__ __forceinline__ Req load_req(const TParams &p, int b, bool flag = false)
{
    Req r;
    r.tok = __ldg(p.qo_indptr + b);
    r.T = __ldg(p.qo_indptr + b + 1) - r.tok;
    r.P = __ldg(p.prefix_len + b);
    r.row = __ldg(p.req_idx + b);
    r.ntiles = r.nqt = 0;
    if (r.T == 0) return r;
    if (r.T < 0 || r.T > p.max_tree || r.P < 0 || (int64_t)r.P + r.T > p.rtt_stride) {
        if (flag && p.status) atomicOr(p.status, RX_DEV_BAD_LEN);
        return r;
    }
    r.ntiles = (int)(((int64_t)r.P + r.T + kBN - 1) / kBN);
    r.nqt = (r.T + p.tb * p.nt - 1) / (p.tb * p.nt);
    return r;
}

// A place in the list, and how many units of it from there on.
struct Start {
    int g, b, qt, j, left;
    int64_t total;  // units of the list
};

// The (kv head g, request, row tiles) that the end of a CTA's share cuts, when
// it also begins in that share: its parts are the CTA's last segment (slot 1)
// and the first segments (slot 0) of the CTAs after it.
struct __align__(16) Cut {
    int parts;      // 0: there is none
    int g;
    int tok, ntok;  // first query row, drafted tokens
};

// Exclusive prefix sums of the requests' units, `per` requests a thread, into
// pre[0 .. threads]; returns the total.  Whole block.
template <int THREADS>
__device__ int64_t scan_units(const TParams &p, int64_t *pre, int per, bool flag)
{
    __shared__ int64_t warp_tot[THREADS / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t sum = 0;
    for (int i = 0; i < per; ++i) {
        const int64_t b = (int64_t)threadIdx.x * per + i;
        if (b < p.batch) sum += load_req(p, (int)b, flag).units();
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
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) base += warp_tot[w];
        total += warp_tot[w];
    }
    pre[threadIdx.x] = base + x - sum;
    if (threadIdx.x == THREADS - 1) pre[THREADS] = total;
    __syncthreads();
    return total;
}

// The place of unit u (0 <= u < hkv * per_head); r: its request.
template <int THREADS>
__device__ Start locate(const TParams &p, const int64_t *pre, int per, int64_t per_head, int64_t u, Req &r)
{
    Start c;
    c.left = 0;
    c.total = per_head * p.hkv;
    c.g = (int)(u / per_head);
    int64_t x = u - c.g * per_head;
    int lo = 0, hi = THREADS - 1;  // the thread whose requests hold unit x
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (pre[mid] <= x) lo = mid; else hi = mid - 1;
    }
    x -= pre[lo];
    c.b = lo * per;
    for (r = load_req(p, c.b); x >= r.units(); r = load_req(p, c.b)) {
        x -= r.units();
        ++c.b;
    }
    c.qt = (int)(x / r.ntiles);
    c.j = (int)(x - (int64_t)c.qt * r.ntiles);
    return c;
}

// First unit of CTA c out of `ctas` (no more CTAs than units: none is empty).
__device__ __forceinline__ int64_t first_unit(int64_t total, int ctas, int c) { return total * c / ctas; }

// One warp walks the CTA's share and hands its segments to the other roles,
// up to kSegs ahead, each with its tree's mask words where positions of the
// tree are among its tiles: under load a read of global memory takes
// microseconds, which no other role then waits for.  The lanes hold the
// lengths of 32 requests at a time.
template <int D, bool F8>
__device__ void scheduler(const TParams &p, unsigned char *smem, uint32_t sbase)
{
    using L = TL<D, F8>;
    const uint32_t bar = sbase + L::OFF_BAR;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::OFF_ABORT);
    const int lane = threadIdx.x & 31;
    Start c = *reinterpret_cast<const Start *>(smem + L::OFF_START);
    int base = c.b;
    Req mine;  // of request base + lane
    auto fill = [&]() {
        mine.ntiles = 0;
        if (base + lane < p.batch) mine = load_req(p, base + lane);
    };
    fill();
    Cut cut{0, 0, 0, 0};
    for (int s = 0;; ++s) {
        const int slot = s % kSegs, l = c.b - base;
        if (s >= kSegs && !warp_wait(bar + 8 * (L::B_SEGEMPTY + slot), (s / kSegs - 1) & 1, abort_flag, p.status)) break;
        // no drafted position of the new segment noted yet (see the V producers)
        if (s >= kSegs) reinterpret_cast<uint32_t *>(smem + L::OFF_NF)[slot * 32 + lane] = 0;
        Seg g;
        const int ntiles = __shfl_sync(0xffffffffu, mine.ntiles, l), nqt = __shfl_sync(0xffffffffu, mine.nqt, l);
        g.g = c.g;
        g.P = __shfl_sync(0xffffffffu, mine.P, l);
        g.T = __shfl_sync(0xffffffffu, mine.T, l);
        g.row = __shfl_sync(0xffffffffu, mine.row, l);
        g.j0 = c.j;
        g.j1 = c.left < ntiles - c.j ? c.j + c.left : ntiles;
        g.node = c.qt * p.tb * p.nt;
        g.ntok = min(p.tb * p.nt, g.T - g.node);
        g.tok = __shfl_sync(0xffffffffu, mine.tok, l) + g.node;
        g.nt = g.ntok > p.tb ? 2 : 1;
        g.whole = g.j0 == 0 && g.j1 == ntiles;
        c.left -= g.j1 - g.j0;
        g.last = c.left <= 0;
        if (lane == 0) *reinterpret_cast<Seg *>(smem + L::OFF_SEG + slot * 64) = g;
        if (p.mask && g.T <= kMaskT && g.j1 * kBN > g.P) {
            const int W = (g.T + 31) / 32;
            const uint32_t dst = sbase + L::OFF_MASK + slot * (kMaskT * (kMaskT / 32) * 4);
            for (int i = lane; i < g.ntok * W; i += 32) {
                const int t = i / W, w = i - t * W;
                rx::cp_async_4(dst + (t * (kMaskT / 32) + w) * 4, p.mask + (int64_t)(g.tok + t) * p.words + w, 4);
            }
        }
        rx::cp_async_mbar_arrive(bar + 8 * (L::B_SEGFULL + slot));  // the words, as they land
        __syncwarp();
        if (lane == 0) rx::mbar_arrive(bar + 8 * (L::B_SEGFULL + slot));  // the segment
        if (g.last) {
            if (g.j0 == 0 && g.j1 < ntiles) {
                const int ctas = (int)min((int64_t)gridDim.x, c.total), x = (int)blockIdx.x;
                const int64_t end = first_unit(c.total, ctas, x + 1) + (ntiles - g.j1);
                cut = Cut{2, g.g, g.tok, g.ntok};
                for (int n = 32; n == 32;) {  // the CTAs behind the next whose share begins inside
                    const int y = x + cut.parts + lane;
                    n = __popc(__ballot_sync(0xffffffffu, y < ctas && first_unit(c.total, ctas, y) < end));
                    cut.parts += n;
                }
            }
            break;
        }
        c.j = 0;
        if (++c.qt < nqt) continue;
        c.qt = 0;
        unsigned next;  // the next request with anything to do: there is one
        do {
            const int from = c.b - base;
            next = __ballot_sync(0xffffffffu, mine.ntiles > 0) & (from >= 31 ? 0u : 0xFFFFFFFEu << (from < 0 ? 0 : from));
            if (from < 0) next = __ballot_sync(0xffffffffu, mine.ntiles > 0);
            if (!next) {
                base += 32;
                if (base >= p.batch) {
                    base = 0;
                    ++c.g;
                }
                c.b = base - 1;
                fill();
            }
        } while (!next);
        c.b = base + __ffs(next) - 1;
    }
    if (lane == 0) p.cuts[blockIdx.x] = cut;
    rx::cp_async_wait_all();
}

// The CTA's segment s for another role; false when a wait gave up.  The role
// arrives on the segment's empty barrier once it needs it no more.
template <typename L>
__device__ __forceinline__ bool get_seg(int s, Seg &g, unsigned char *smem, uint32_t sbase, int32_t *status)
{
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::OFF_ABORT);
    if (!wait_or_abort(sbase + L::OFF_BAR + 8 * (L::B_SEGFULL + s % kSegs), (s / kSegs) & 1, abort_flag, status)) return false;
    const int4 *w = reinterpret_cast<const int4 *>(smem + L::OFF_SEG + (s % kSegs) * 64);
    const int4 a = w[0], b = w[1], c = w[2];
    g = Seg{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, c.z, c.w};
    return true;
}
template <typename L>
__device__ __forceinline__ void free_seg(int s, uint32_t sbase)
{
    rx::mbar_arrive(sbase + L::OFF_BAR + 8 * (L::B_SEGEMPTY + s % kSegs));
}

// ---------------------------------------------------------------------------
// which drafted tokens a row sees
// ---------------------------------------------------------------------------

// Word i of drafted token `node`'s mask: prefix positions (i < 0) are seen,
// bits at and past T are not.  row: its words, or null for a chain.
__device__ __forceinline__ uint32_t mask_word(const uint32_t *row, int words, int node, int T, int i)
{
    uint32_t w = 0xFFFFFFFFu;
    int n = T - 32 * i;  // drafted tokens from bit 0 of this word on
    if (row) w = row[min(max(i, 0), words - 1)];
    else n = min(n, node + 1 - 32 * i);
    w = n >= 32 ? w : n <= 0 ? 0u : w & ((1u << (n & 31)) - 1u);
    return i < 0 ? 0xFFFFFFFFu : w;
}

// ---------------------------------------------------------------------------
// producer warps
// ---------------------------------------------------------------------------

// Which halves of a word are NaN or infinite (bf16 pairs): 0xFFFF masks.
__device__ __forceinline__ uint32_t not_finite(uint32_t w)
{
    constexpr uint32_t E = 0x7F80u;
    return ((w & E) == E ? 0xFFFFu : 0u) | ((w & (E << 16)) == (E << 16) ? 0xFFFF0000u : 0u);
}
__device__ __forceinline__ bool drop_not_finite(uint4 &x)
{
    const uint32_t a = not_finite(x.x), b = not_finite(x.y), c = not_finite(x.z), d = not_finite(x.w);
    x = make_uint4(x.x & ~a, x.y & ~b, x.z & ~c, x.w & ~d);
    return (a | b | c | d) != 0u;
}

// Eight E4M3 codes as eight f16 (exact).
__device__ __forceinline__ uint4 widen_f16(uint32_t lo, uint32_t hi)
{
    return make_uint4(rx::e4m3x2_to_f16x2((uint16_t)lo), rx::e4m3x2_to_f16x2((uint16_t)(lo >> 16)),
                      rx::e4m3x2_to_f16x2((uint16_t)hi), rx::e4m3x2_to_f16x2((uint16_t)(hi >> 16)));
}

// Eight producer warps for K and eight for V, four with two row tiles (V's wait
// for the softmax does not hold up K); each gathers the same rows of every tile
// in 16-byte async copies, slot ids two tiles ahead.  (Loads into registers go
// through L1, which this kernel's shared memory leaves 28 KB: they ran at half
// the rate.)
//
// bf16 pools: the copies land in the swizzled tile itself and report to its
// barrier.  FP8 pools: they land in a ring of three half tiles of codes; each
// thread widens the chunks that it copied and stores them to the tile: K to
// f16, V to bf16, as the weights are (both hold every E4M3 value).
//
// V at drafted positions is looked at before it is handed over: a NaN or
// infinity there would reach rows that do not see the position (0 * inf), so it
// is dropped, noted, and added back to the rows that see it at the end.
template <int D, bool F8, int NT, bool IS_V>
__device__ void producer(const TParams &p, unsigned char *smem, uint32_t sbase)
{
    using L = TL<D, F8>;
    constexpr int ROWS = Ro<NT>::ROWS;
    constexpr int EB = F8 ? 1 : 2;                    // bytes of a value
    constexpr int CPR = D * EB / 16;                  // 16-byte chunks of a row
    constexpr int RPI = 32 / CPR;                     // rows of one instruction
    constexpr int U = ROWS / RPI;                     // instructions for this warp's rows
    const uint32_t bar_full = sbase + L::OFF_BAR + 8 * (IS_V ? L::B_VFULL : L::B_KFULL);
    const uint32_t bar_empty = sbase + L::OFF_BAR + 8 * (IS_V ? L::B_VEMPTY : L::B_KEMPTY);
    const unsigned char *pool = IS_V ? p.v : p.k;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::OFF_ABORT);
    const int lane = threadIdx.x & 31, pw = ((int)(threadIdx.x >> 5) - Ro<NT>::SOFT) % Ro<NT>::PROD;
    const int r0 = pw * ROWS;
    const int sub = lane / CPR, ch = lane % CPR;
    const int row_bytes = p.hkv * D * EB;             // at most 2^21 (the heads are bounded)

    struct Tile {
        int32_t slot;  // lane l < ROWS: slot of row r0 + l, in flight until check() looks at it
        int lim;       // positions of the request from the tile's first on; 0: no tile
        int meta;      // kv head, T, segment mod kSegs: bits 0, 13 and 24 on

        __device__ __forceinline__ int g() const { return meta & 0x1FFF; }
        __device__ __forceinline__ int rel() const { return ((meta >> 13) & 0x7FF) - lim; }  // first position, from the first drafted one
        __device__ __forceinline__ int seg() const { return meta >> 24; }
    };
    static_assert(kMaxTree < 2048 && kSegs <= 64, "the fields of meta");
    // the segment being handed out: its next tile, and how many it still has
    int s = -1, left = 0, lim = 0, meta = 0;
    bool last = false;
    const int32_t *slots = nullptr;  // of this lane's row in that tile
    // the next tile, with the loads of its slot ids
    auto take = [&](Tile &t) {
        t.slot = -1;
        t.lim = t.meta = 0;
        if (left == 0) {
            if (last) return;
            Seg q;
            if (!__all_sync(0xffffffffu, get_seg<L>(s + 1, q, smem, sbase, p.status))) {
                last = true;  // gave up
                return;
            }
            __syncwarp();
            ++s;
            if (lane == 0) free_seg<L>(s, sbase);
            left = q.j1 - q.j0;
            lim = q.P + q.T - q.j0 * kBN;
            meta = q.g | (q.T << 13) | ((s % kSegs) << 24);
            last = q.last;
            slots = p.rtt + (int64_t)q.row * p.rtt_stride + (int64_t)q.j0 * kBN + r0 + lane;
        }
        t.lim = lim;
        t.meta = meta;
        if (lane < ROWS && r0 + lane < lim) t.slot = rx::ld_stream_b32(slots);
        --left;
        lim -= kBN;
        slots += kBN;
    };
    // slots past the end or outside the pool (flagged) become -1
    auto check = [&](Tile &t) {
        if (t.slot >= 0 && (int64_t)t.slot < p.num_slots) return;
        if (lane < ROWS && r0 + lane < t.lim && p.status) atomicOr(p.status, RX_DEV_BAD_SLOT);
        t.slot = -1;
    };
    auto source = [&](const Tile &t, int u, bool &ok) {
        const int32_t id = __shfl_sync(0xffffffffu, t.slot, u * RPI + sub);
        ok = id >= 0;
        return pool + (ok ? (int64_t)id * row_bytes : 0) + (t.g() * (D * EB) + ch * 16);
    };
    // this thread's chunks of V at drafted positions, once they are in the tile
    auto scrub = [&](uint32_t off, const Tile &t) {
        constexpr int CH = F8 ? 2 : 1;  // 16-byte chunks of the tile for one of the row
#pragma unroll 1
        for (int u = 0; u < U * CH; ++u) {
            const int r = r0 + u / CH * RPI + sub, e = t.rel() + r;
            uint4 *at = reinterpret_cast<uint4 *>(smem + off + sw128(r, CH * ch + u % CH, L::BLK));
            uint4 x = *at;
            if (e >= 0 && drop_not_finite(x)) {
                *at = x;
                atomicOr(reinterpret_cast<uint32_t *>(smem + L::OFF_NF) + t.seg() * 32 + (e >> 5), 1u << (e & 31));
            }
        }
    };

    if constexpr (!F8) {
        Tile cur, nxt, nx2;
        take(cur);
        take(nxt);
        for (int n = 0; cur.lim > 0; ++n) {
            const int st = n % kStages;
            take(nx2);
            check(cur);
            const uint32_t off = (IS_V ? L::OFF_V : L::OFF_K) + st * L::NB * L::BLK;
            if (n >= kStages && !warp_wait(bar_empty + 8 * st, (n / kStages - 1) & 1, abort_flag, p.status)) break;
#pragma unroll 2
            for (int u = 0; u < U; ++u) {
                bool ok;
                const unsigned char *src = source(cur, u, ok);
                rx::cp_async_16(sbase + off + sw128(r0 + u * RPI + sub, ch, L::BLK), src, ok ? 16 : 0);
            }
            if (IS_V && cur.rel() + kBN > 0) {  // the tile has drafted positions
                rx::cp_async_wait_all();
                scrub(off, cur);
                rx::fence_proxy_async_smem();
                rx::mbar_arrive(bar_full + 8 * st);
            } else {
                rx::cp_async_mbar_arrive(bar_full + 8 * st);
            }
            cur = nxt;
            nxt = nx2;
        }
        rx::cp_async_wait_all();  // nothing may still be landing when the CTA exits
    } else {
        constexpr int H = U / 2;  // instructions of half a tile
        // chunk u of half-tile buffer b: + b CODE + 512 u
        const uint32_t mine = L::OFF_CODE + (IS_V ? kCodeBufs * L::CODE : 0) + (uint32_t)(pw * H * 32 + lane) * 16;
        auto fetch = [&](const Tile &t, int h, int buf) {
#pragma unroll
            for (int u = 0; u < H; ++u) {
                bool ok;
                const unsigned char *src = source(t, h * H + u, ok);
                rx::cp_async_16(sbase + mine + buf * L::CODE + u * 512, src, ok ? 16 : 0);
            }
            rx::cp_async_commit();
        };
        // this thread's chunks of a landed half into the tile at `off`
        auto widen = [&](uint32_t off, int h, int buf) {
#pragma unroll
            for (int u = 0; u < H; ++u) {
                const uint4 x = *reinterpret_cast<const uint4 *>(smem + mine + buf * L::CODE + u * 512);
                const uint4 a = IS_V ? rx::e4m3x8_to_bf16x8(make_uint2(x.x, x.y)) : widen_f16(x.x, x.y);
                const uint4 b = IS_V ? rx::e4m3x8_to_bf16x8(make_uint2(x.z, x.w)) : widen_f16(x.z, x.w);
                const int r = r0 + (h * H + u) * RPI + sub;
                // the upper lanes of a row store their second chunk first: the
                // two column blocks of a row lie on the same banks
                const int swap = D == 128 ? (ch >> 2) & 1 : 0;
                *reinterpret_cast<uint4 *>(smem + off + sw128(r, 2 * ch + swap, L::BLK)) = swap ? b : a;
                *reinterpret_cast<uint4 *>(smem + off + sw128(r, 2 * ch + 1 - swap, L::BLK)) = swap ? a : b;
            }
        };
        Tile cur, nxt, nx2;
        take(cur);
        take(nxt);
        check(cur);
        check(nxt);
        fetch(cur, 0, 0);
        fetch(cur, 1, 1);
        fetch(nxt, 0, 2);
        int buf = 0;  // of the tile's first half; three halves are in flight
        for (int n = 0; cur.lim > 0; ++n) {
            const int st = n % kStages, buf1 = buf == 2 ? 0 : buf + 1, buf2 = buf1 == 2 ? 0 : buf1 + 1;
            const uint32_t off = (IS_V ? L::OFF_V : L::OFF_K) + st * L::NB * L::BLK;
            take(nx2);
            rx::cp_async_wait<2>();     // the first half
            if (n >= kStages && !warp_wait(bar_empty + 8 * st, (n / kStages - 1) & 1, abort_flag, p.status)) break;
            widen(off, 0, buf);
            fetch(nxt, 1, buf);
            rx::cp_async_wait<2>();     // the second
            widen(off, 1, buf1);
            if (IS_V && cur.rel() + kBN > 0) scrub(off, cur);  // the tile has drafted positions
            rx::fence_proxy_async_smem();
            rx::mbar_arrive(bar_full + 8 * st);
            check(nx2);
            fetch(nx2, 0, buf1);
            buf = buf2;
            cur = nxt;
            nxt = nx2;
        }
        rx::cp_async_wait_all();
    }
}

// ---------------------------------------------------------------------------
// query rows
// ---------------------------------------------------------------------------

// One warp copies each segment's query rows (row r of row tile t: drafted token
// t tb + r / G of the segment, q head g G + r % G).  bf16 pools: 16-byte async
// copies.  FP8 pools: S = Q K^T runs in f16, which holds every E4M3 value; a
// query row is brought to f16 times a power of two that puts its largest value
// just below 2^15 (values 2^-29 of that and above stay exact), and the power
// goes into the row's score scale.
//
// Buffers: with one row tile a segment, of the segments in turn; with two, one
// for each row tile.
template <int D, bool F8, int NT>
__device__ void query_loader(const TParams &p, unsigned char *smem, uint32_t sbase)
{
    using L = TL<D, F8>;
    constexpr int CPR = D / 8, RPI = 32 / CPR;   // chunks of a row, rows of one instruction
    constexpr int UQ = 4;                        // FP8: instructions in flight
    const uint32_t bar = sbase + L::OFF_BAR;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::OFF_ABORT);
    const int lane = threadIdx.x & 31, sub = lane / CPR, ch = lane % CPR;
    int uses[2] = {0, 0};  // of each buffer
    for (int s = 0;; ++s) {
        Seg g;
        if (!__all_sync(0xffffffffu, get_seg<L>(s, g, smem, sbase, p.status))) break;
        __syncwarp();
        if (lane == 0) free_seg<L>(s, sbase);
        bool ok = true;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (t >= g.nt || !ok) break;
            const int buf = NT == 1 ? s % L::QB : t, use = NT == 1 ? s / L::QB : uses[t]++;
            const int M = min(p.tb, g.ntok - t * p.tb) * p.G;
            if (use >= 1 && !(ok = warp_wait(bar + 8 * (L::B_QEMPTY + buf), (use - 1) & 1, abort_flag, p.status))) break;
            const uint32_t dst = L::OFF_Q + buf * L::NB * L::BLK;
            // this lane's row, its drafted token's query row and its head
            int r = sub;
            const int step_t = RPI / p.G, step_h = RPI - step_t * p.G;
            int h = r % p.G;
            int64_t src = ((int64_t)(g.tok + t * p.tb + r / p.G) * p.hq + (int64_t)g.g * p.G + h) * D + ch * 8;
            auto advance = [&]() {  // RPI rows on
                r += RPI;
                h += step_h;
                src += ((int64_t)step_t * p.hq + step_h) * D;
                if (h >= p.G) {     // the next drafted token's first heads
                    h -= p.G;
                    src += (int64_t)(p.hq - p.G) * D;
                }
            };
            while (r - sub < M) {
                if constexpr (!F8) {
                    if (r < M) rx::cp_async_16(sbase + dst + sw128(r, ch, L::BLK), p.q + src, 16);
                    advance();
                } else {
                    const int rbase = r;
                    uint4 x[UQ];
#pragma unroll
                    for (int u = 0; u < UQ; ++u) {
                        x[u] = make_uint4(0, 0, 0, 0);
                        if (r < M) x[u] = rx::ld_stream(p.q + src);
                        advance();
                    }
#pragma unroll
                    for (int u = 0; u < UQ; ++u) {
                        const int ru = rbase + u * RPI;
                        const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
                        uint32_t top = 0;  // largest magnitude (bf16 bits) of the row
#pragma unroll
                        for (int k = 0; k < 4; ++k) top = max(top, max(w[k] & 0x7FFFu, (w[k] >> 16) & 0x7FFFu));
#pragma unroll
                        for (int d = CPR / 2; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
                        const int e = max((int)(top >> 7) - 127, -100);
                        const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);  // 2^(14 - e)
                        uint32_t y[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            y[k] = rx::pack_f16(__uint_as_float(w[k] << 16) * up, __uint_as_float(w[k] & 0xFFFF0000u) * up);
                        if (ru < M) {
                            *reinterpret_cast<uint4 *>(smem + dst + sw128(ru, ch, L::BLK)) = make_uint4(y[0], y[1], y[2], y[3]);
                            // never 0 or infinite: a masked place's score is
                            // -inf times it (a finite one is below 2^31)
                            if (ch == 0)
                                reinterpret_cast<float *>(smem + L::OFF_QS)[(s % kRing) * kRows + ru] =
                                    fminf(fmaxf(p.scale_log2 * __uint_as_float((uint32_t)(127 - 14 + e) << 23), 0x1p-126f),
                                          0x1.fffffep127f);
                        }
                    }
                }
            }
            if constexpr (F8) {
                rx::fence_proxy_async_smem();
                rx::mbar_arrive(bar + 8 * (L::B_QFULL + buf));
            } else {
                rx::cp_async_mbar_arrive(bar + 8 * (L::B_QFULL + buf));
            }
        }
        if (!ok || g.last) break;
    }
    rx::cp_async_wait_all();
}

// ---------------------------------------------------------------------------
// the two MMA threads
// ---------------------------------------------------------------------------

// The CTA's items: for every position tile n (all segments in a row) the
// segment's row tiles t.  S = Q_t K_n^T waits for an S buffer whose scores the
// softmax has in registers, O_t += P V_n for P.
//
// One row tile: S and P have two buffers each, which the items take in turn, and
// barriers for each: whoever waits for one product knows that the one two items
// before has completed, and a phase's parity is never ambiguous.  Two row tiles:
// a P and barriers for each, so again each barrier is waited for phase by phase
// by one group of warps; TMEM has room for one S, which the next item of either
// takes once the last one's scores are in registers.
//
// S and P V are issued by a thread each: a thread spends as long on the waits
// and commits around an operation's eight MMAs as on the MMAs, and with one
// thread for both the tensor core idled meanwhile (long chat 0.252 against
// 0.242 ms).
struct Item {
    int c, n, t;                   // c: of its row tile; before: the item before it, if any
    int before_t, before_c;
    int use;                       // row tiles before this one in its O (and Q) buffer
    int seg;
    bool t0, t1;                   // the first, the last row tile of the position tile
    bool first, last;              // the row tile's first, last position tile
};

// f(item) for every item, until it or a wait gives up.
template <typename L, int NT, typename F>
__device__ __forceinline__ void for_items(const TParams &p, unsigned char *smem, uint32_t sbase, F f)
{
    int c0 = 0, c1 = 0, n = 0, s2 = 0;  // s2: segments with two row tiles
    int before_t = 0, before_c = -1;
    for (int s = 0;; ++s) {
        Seg g;
        if (!get_seg<L>(s, g, smem, sbase, p.status)) return;
        free_seg<L>(s, sbase);
        const int nt = NT == 1 ? 1 : g.nt;
        for (int j = g.j0; j < g.j1; ++j, ++n)
            for (int t = 0; t < nt; ++t) {
                const int c = t == 0 ? c0++ : c1++;
                if (!f(Item{c, n, t, before_t, before_c, t == 0 ? s : s2, s, NT == 1 || t == 0, NT == 1 || t == nt - 1, j == g.j0,
                            j == g.j1 - 1}))
                    return;
                before_t = t;
                before_c = c;
            }
        s2 += nt == 2;
        if (g.last) return;
    }
}

template <int D, bool F8, int NT>
__device__ void issue_qk(const TParams &p, unsigned char *smem, uint32_t sbase)
{
    using L = TL<D, F8>;
    using M = Tm<NT>;
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + L::OFF_TMEM);
    const uint32_t bar = sbase + L::OFF_BAR;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::OFF_ABORT);
    constexpr uint32_t idesc = F8 ? rx::idesc_f16(kRows, kBN, false, false) : rx::idesc_bf16(kRows, kBN, false, false);
    auto wait = [&](int b, uint32_t parity) { return wait_or_abort(bar + 8 * b, parity, abort_flag, p.status); };
    const uint64_t dq = rx::sdesc_sw128(sbase + L::OFF_Q, 16, 1024);
    const uint64_t dk = rx::sdesc_sw128(sbase + L::OFF_K, 16, 1024);
    for_items<L, NT>(p, smem, sbase, [&](const Item &m) -> bool {
        const int st = m.n % kStages;
        const Turn<NT> turn(m.t, m.c);
        const int qb = NT == 1 ? m.seg % L::QB : m.t, quse = NT == 1 ? m.seg / L::QB : m.use;
        if (m.first && !wait(L::B_QFULL + qb, quse & 1)) return false;
        if (m.t0 && !wait(L::B_KFULL + st, (m.n / kStages) & 1)) return false;
        // its S: of the item two before, or with one for both row tiles of the item before
        if constexpr (NT == 1) {
            if (m.c >= 2 && !wait(L::B_SEMPTY + turn.b, (turn.phase - 1) & 1)) return false;
        } else {
            if (m.before_c >= 0 && !wait(L::B_SEMPTY + m.before_t, m.before_c & 1)) return false;
        }
        rx::fence_proxy_async_smem();  // rows landed by cp.async -> async proxy
        rx::tc_fence_after();
        const uint64_t dks = dk + (uint64_t)((st * L::NB * L::BLK) >> 4);
        const uint64_t dqs = dq + (uint64_t)((qb * L::NB * L::BLK) >> 4);
#pragma unroll
        for (int kb = 0; kb < D / 16; ++kb) {
            const uint64_t off = (uint64_t)(((kb >> 2) * L::BLK + (kb & 3) * 32) >> 4);
            rx::tc_mma(tmem + M::s(turn.b), dqs + off, dks + off, idesc, kb > 0);
        }
        rx::tc_commit(bar + 8 * (L::B_SFULL + turn.b));
        if (m.t1) rx::tc_commit(bar + 8 * (L::B_KEMPTY + st));
        if (m.last) rx::tc_commit(bar + 8 * (L::B_QEMPTY + qb));
        return true;
    });
    // everything issued has finished before TMEM is released
    rx::tc_commit(bar + 8 * L::B_FINAL);
    rx::drain_wait(bar + 8 * L::B_FINAL, 0, p.status);
}

template <int D, bool F8, int NT>
__device__ void issue_pv(const TParams &p, unsigned char *smem, uint32_t sbase)
{
    using L = TL<D, F8>;
    using M = Tm<NT>;
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + L::OFF_TMEM);
    const uint32_t bar = sbase + L::OFF_BAR;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::OFF_ABORT);
    constexpr uint32_t idesc = rx::idesc_bf16(kRows, D, false, true);
    auto wait = [&](int b, uint32_t parity) { return wait_or_abort(bar + 8 * b, parity, abort_flag, p.status); };
    const uint64_t dv = rx::sdesc_sw128(sbase + L::OFF_V, L::BLK, 1024);
    for_items<L, NT>(p, smem, sbase, [&](const Item &m) -> bool {
        const int st = m.n % kStages;
        const Turn<NT> turn(m.t, m.c);
        if (m.t0 && !wait(L::B_VFULL + st, (m.n / kStages) & 1)) return false;
        if (m.first && m.use >= 1 && !wait(L::B_OEMPTY + m.t, (m.use - 1) & 1)) return false;
        if (!wait(L::B_PFULL + turn.b, turn.phase & 1)) return false;
        rx::fence_proxy_async_smem();  // V rows landed by cp.async
        rx::tc_fence_after();
        const uint64_t dvs = dv + (uint64_t)((st * L::NB * L::BLK) >> 4);
#pragma unroll
        for (int ks = 0; ks < kBN / 16; ++ks)
            rx::tc_mma_ts(tmem + M::o(m.t), tmem + M::p(turn.b) + ks * 8, dvs + (uint64_t)((ks * 16 * 128) >> 4), idesc,
                          (!m.first || ks > 0) ? 1u : 0u);
        rx::tc_commit(bar + 8 * (L::B_PVDONE + turn.b));
        if (m.t1) rx::tc_commit(bar + 8 * (L::B_VEMPTY + st));
        return true;
    });
    rx::tc_commit(bar + 8 * (L::B_FINAL + 1));
    rx::drain_wait(bar + 8 * (L::B_FINAL + 1), 0, p.status);
}

// ---------------------------------------------------------------------------
// softmax warps: one query row per thread
// ---------------------------------------------------------------------------

// The NaN and infinities of V at drafted positions that a row sees, added to
// its written result: o (part < 0) or the partial row `part`.
template <int D, bool F8>
__device__ __noinline__ void add_not_finite(const TParams &p, const uint32_t *nf, const uint32_t *mrow, int words, int node,
                                            int row, int g, int P, int T, int64_t part, int64_t orow)
{
    for (int w = 0; w < (T + 31) / 32; ++w)
        for (uint32_t bad = nf[w] & mask_word(mrow, words, node, T, w); bad; bad &= bad - 1) {
            const int pos = P + 32 * w + __ffs(bad) - 1;
            const int64_t slot = __ldg(p.rtt + (int64_t)row * p.rtt_stride + pos);
            const int64_t at = (slot * p.hkv + g) * D;
            for (int i = 0; i < D; ++i) {
                float v;
                if constexpr (F8) {
                    const uint32_t h = rx::e4m3x2_to_f16x2(__ldg(p.v + at + i));
                    v = __half2float(__ushort_as_half((unsigned short)(h & 0xFFFFu)));
                } else {
                    v = __bfloat162float(reinterpret_cast<const bf16 *>(p.v)[at + i]);
                }
                if (isfinite(v)) continue;
                if (part >= 0) p.part_o[part * D + i] += v;
                else p.o[orow * D + i] = __float2bfloat16_rn(__bfloat162float(p.o[orow * D + i]) + v);
            }
        }
}

// What a thread keeps of its row of one row tile.
struct RowState {
    float m, l;    // running maximum (log2 units) and sum
    float sl2;     // log2 units of a score
};

template <int D, bool F8, int NT>
__device__ void softmax_rows(const TParams &p, unsigned char *smem, uint32_t sbase)
{
    using L = TL<D, F8>;
    using TM = Tm<NT>;
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + L::OFF_TMEM);
    const uint32_t bar = sbase + L::OFF_BAR;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::OFF_ABORT);
    const int row = threadIdx.x & (kRows - 1);         // = TMEM lane
    const int t = NT == 1 ? 0 : threadIdx.x / kRows;   // the warps' row tile
    const uint32_t lanes = (uint32_t)(row & ~31) << 16;
    const int rt = row / p.G, rh = row - rt * p.G;     // drafted token of the row tile, q head of the kv head
    int c = 0;                                         // the row tile's items so far
    for (int s = 0;; ++s) {
        Seg g;
        if (!__all_sync(0xffffffffu, get_seg<L>(s, g, smem, sbase, p.status))) return;
        if (NT == 2 && t >= g.nt) {  // the segment has one row tile
            __syncwarp();
            if ((row & 31) == 0) free_seg<L>(s, sbase);
            if (g.last) return;
            continue;
        }
        // the mask row of drafted token rt + t * tb of the segment
        const uint32_t *masks = !p.mask ? nullptr
                                : g.T <= kMaskT ? reinterpret_cast<const uint32_t *>(smem + L::OFF_MASK) + (s % kSegs) * (kMaskT * (kMaskT / 32))
                                                : p.mask + (int64_t)g.tok * p.words;
        const int words = g.T <= kMaskT ? kMaskT / 32 : p.words;
        RowState a{-INFINITY, 0.f, p.scale_log2};
        for (int j = g.j0; j < g.j1; ++j, ++c) {
                const int M = min(p.tb, g.ntok - t * p.tb) * p.G, node = rt + t * p.tb;
                const bool valid = row < M, warp_on = (row & ~31) < M;
                const uint32_t tO = tmem + TM::o(t) + lanes;
                const Turn<NT> turn(t, c);
                const uint32_t tS = tmem + TM::s(turn.b) + lanes, tP = tmem + TM::p(turn.b) + lanes;
                if (!warp_wait(bar + 8 * (L::B_SFULL + turn.b), turn.phase & 1, abort_flag, p.status)) return;
                rx::tc_fence_after();
                auto release_s = [&]() {
                    rx::tc_fence_before();
                    rx::mbar_arrive(bar + 8 * (L::B_SEMPTY + turn.b));
                };
                // the product before in these columns has read P (a warp without
                // rows waits too, or it could arrive twice in a phase)
                auto p_free = [&]() {
                    const bool ok = turn.phase < 1 || warp_wait(bar + 8 * (L::B_PVDONE + turn.b), (turn.phase - 1) & 1, abort_flag, p.status);
                    rx::tc_fence_after();
                    return ok;
                };
                if (!warp_on) {
                    release_s();
                    if (!p_free()) return;
                } else {
                    // the row's scores of this tile, loaded once (four loads in
                    // flight): a load takes about 200 cycles to come back
                    uint32_t sv[kBN];
#pragma unroll
                    for (int k = 0; k < kBN / 32; ++k) rx::tmem_ld32(tS + k * 32, *reinterpret_cast<uint32_t(*)[32]>(sv + 32 * k));
                    if (F8 && j == g.j0) a.sl2 = reinterpret_cast<const float *>(smem + L::OFF_QS)[(s % kRing) * kRows + row];
                    const int kbase = j * kBN;
                    if (kbase + kBN > g.P) {   // drafted positions, or past the last
                        const int off = kbase - g.P, w0 = off >> 5;
                        const uint32_t *mrow = masks && valid ? masks + (int64_t)node * words : nullptr;
                        uint32_t w[5];
#pragma unroll
                        for (int k = 0; k < 5; ++k) w[k] = mask_word(mrow, words, g.node + node, g.T, w0 + k);
                        rx::tmem_wait_ld();
                        release_s();
#pragma unroll
                        for (int k = 0; k < kBN / 32; ++k) {
                            const uint32_t bits = __funnelshift_r(w[k], w[k + 1], off & 31);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!((bits >> e) & 1u)) sv[32 * k + e] = 0xFF800000u;  // -inf
                        }
                    } else {
                        rx::tmem_wait_ld();
                        release_s();
                    }
                    float mx;
                    {
                        float a0 = -INFINITY, a1 = -INFINITY, a2 = -INFINITY, a3 = -INFINITY;
#pragma unroll
                        for (int k = 0; k < kBN / 8; ++k) {
                            a0 = rx::fmax3(a0, u2f(sv[8 * k]), u2f(sv[8 * k + 1]));
                            a1 = rx::fmax3(a1, u2f(sv[8 * k + 2]), u2f(sv[8 * k + 3]));
                            a2 = rx::fmax3(a2, u2f(sv[8 * k + 4]), u2f(sv[8 * k + 5]));
                            a3 = rx::fmax3(a3, u2f(sv[8 * k + 6]), u2f(sv[8 * k + 7]));
                        }
                        mx = rx::fmax3(fmaxf(a0, a1), a2, a3);
                    }
                    const float m_new = fmaxf(a.m, mx * a.sl2);
                    const bool need = valid && (a.m == -INFINITY || m_new > a.m + kRescale);
                    const bool scale_o = need && a.m != -INFINITY;
                    const float alpha = scale_o ? rx::fast_exp2(a.m - m_new) : 1.f;
                    if (need) {
                        a.l *= alpha;
                        a.m = m_new;
                    }
                    const float mu = a.m == -INFINITY ? 0.f : a.m;
                    const uint64_t scale2 = rx::f2(a.sl2, a.sl2), negm2 = rx::f2(-mu, -mu);
                    uint64_t acc[4] = {0, 0, 0, 0};
                    if (!p_free()) return;
#pragma unroll
                    for (int k = 0; k < kBN / 64; ++k) {
                        uint32_t pk[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            float x0, x1;
                            rx::f2_split(rx::f2_fma(rx::f2(u2f(sv[64 * k + 2 * e]), u2f(sv[64 * k + 2 * e + 1])), scale2, negm2), x0, x1);
                            const float e0 = rx::fast_exp2(x0), e1 = rx::fast_exp2(x1);
                            acc[e & 3] = rx::f2_add(acc[e & 3], rx::f2(e0, e1));
                            // the weights are rounded to bf16 for the tensor core
                            // (their sum is not), over FP8 pools too: f16 would keep
                            // three more bits of weights near the largest, but none of
                            // those 17 nats below it, which a long context adds up
                            pk[e] = rx::pack_bf16(e0, e1);
                        }
                        rx::tmem_st32(tP + k * 32, pk);
                    }
                    float a0, a1;
                    rx::f2_split(rx::f2_add(rx::f2_add(acc[0], acc[1]), rx::f2_add(acc[2], acc[3])), a0, a1);
                    a.l += a0 + a1;
                    if (__any_sync(0xffffffffu, scale_o)) {
                        // the row tile's product before has to be complete; that
                        // of the item two before is
                        if (NT == 1 && !warp_wait(bar + 8 * (L::B_PVDONE + ((c - 1) & 1)), ((c - 1) >> 1) & 1, abort_flag, p.status))
                            return;
                        rx::tc_fence_after();
#pragma unroll
                        for (int k = 0; k < D / 32; ++k) {
                            uint32_t x[32];
                            rx::tmem_ld32(tO + k * 32, x);
                            rx::tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(u2f(x[e]) * alpha);
                            rx::tmem_st32(tO + k * 32, x);
                        }
                    }
                    rx::tmem_wait_st();
                }
                rx::tc_fence_before();
                rx::mbar_arrive(bar + 8 * (L::B_PFULL + turn.b));
            }
        // the segment's results, once the row tile's last product is complete
        const uint32_t *nf = reinterpret_cast<const uint32_t *>(smem + L::OFF_NF) + (s % kSegs) * 32;
        {
            const Turn<NT> end(t, c - 1);
            const int M = min(p.tb, g.ntok - t * p.tb) * p.G, node = rt + t * p.tb;
            const bool valid = row < M, warp_on = (row & ~31) < M;
            const uint32_t tO = tmem + TM::o(t) + lanes;
            if (!warp_wait(bar + 8 * (L::B_PVDONE + end.b), end.phase & 1, abort_flag, p.status)) return;
            rx::tc_fence_after();
            const float inv = a.l == 0.f ? 0.f : p.v_scale / a.l;
            const int64_t orow = (int64_t)(g.tok + node) * p.hq + (int64_t)g.g * p.G + rh;
            const int64_t prow = ((int64_t)(2 * blockIdx.x + (g.j0 == 0 ? 1 : 0)) * NT + t) * kRows + row;
            if (warp_on) {
                // not unrolled: straight-line code that runs once a segment is
                // fetched more slowly than it runs
#pragma unroll 1
                for (int k = 0; k < D / 32; ++k) {
                    uint32_t x[32];
                    rx::tmem_ld32(tO + k * 32, x);
                    rx::tmem_wait_ld();
                    if (valid) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = a.l == 0.f ? 0u : __float_as_uint(u2f(x[e]) * inv);
                    if (g.whole) {
                        uint4 *dst = reinterpret_cast<uint4 *>(p.o + orow * D + k * 32);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            dst[e] = make_uint4(rx::pack_bf16(u2f(x[8 * e]), u2f(x[8 * e + 1])),
                                                rx::pack_bf16(u2f(x[8 * e + 2]), u2f(x[8 * e + 3])),
                                                rx::pack_bf16(u2f(x[8 * e + 4]), u2f(x[8 * e + 5])),
                                                rx::pack_bf16(u2f(x[8 * e + 6]), u2f(x[8 * e + 7])));
                    } else {
                        uint4 *dst = reinterpret_cast<uint4 *>(p.part_o + prow * D + k * 32);
#pragma unroll
                        for (int e = 0; e < 8; ++e) dst[e] = make_uint4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
                    }
                    }
                    __syncwarp();
                }
                if (valid) {
                    const float l2 = a.l == 0.f ? -INFINITY : a.m + log2f(a.l);
                    if (!g.whole) p.part_l[prow] = l2;
                    else if (p.lse) p.lse[orow] = l2 * rx::kLn2;
                }
                __syncwarp();
            }
            rx::tc_fence_before();
            rx::mbar_arrive(bar + 8 * (L::B_OEMPTY + t));
            if (g.j1 * kBN > g.P) {
                uint32_t any = 0;
                for (int w = 0; w < (g.T + 31) / 32; ++w) any |= nf[w];
                if (any && valid)
                    add_not_finite<D, F8>(p, nf, masks ? masks + (int64_t)node * words : nullptr, words, g.node + node, g.row, g.g,
                                          g.P, g.T, g.whole ? -1 : prow, orow);
            }
        }
        __syncwarp();
        if ((row & 31) == 0) free_seg<L>(s, sbase);
        if (g.last) return;
    }
}

template <int D, bool F8, int NT>
__global__ void __launch_bounds__(Ro<NT>::THREADS, 1) tree_kernel(const __grid_constant__ TParams p)
{
    using L = TL<D, F8>;
    using W = Ro<NT>;
    constexpr int kThreads = W::THREADS;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = rx::smem_u32(smem_raw);
    unsigned char *smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);  // 1024-aligned swizzle atoms
    const uint32_t sbase = rx::smem_u32(smem);
    const uint32_t bar = sbase + L::OFF_BAR;
    const int warp = threadIdx.x >> 5;
    rx::pdl_launch_dependents();  // the merge kernel may launch and wait on the device

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            rx::mbar_init(bar + 8 * (L::B_KFULL + i), 32 * W::PROD);
            rx::mbar_init(bar + 8 * (L::B_VFULL + i), 32 * W::PROD);
            rx::mbar_init(bar + 8 * (L::B_KEMPTY + i), 1);
            rx::mbar_init(bar + 8 * (L::B_VEMPTY + i), 1);
        }
        for (int i = 0; i < L::QB; ++i) {
            rx::mbar_init(bar + 8 * (L::B_QFULL + i), 32);
            rx::mbar_init(bar + 8 * (L::B_QEMPTY + i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            rx::mbar_init(bar + 8 * (L::B_SFULL + i), 1);
            rx::mbar_init(bar + 8 * (L::B_SEMPTY + i), kRows);
            rx::mbar_init(bar + 8 * (L::B_PFULL + i), kRows);
            rx::mbar_init(bar + 8 * (L::B_PVDONE + i), 1);
            rx::mbar_init(bar + 8 * (L::B_OEMPTY + i), kRows);
        }
        for (int i = 0; i < kSegs; ++i) {
            rx::mbar_init(bar + 8 * (L::B_SEGFULL + i), 32 + 1);  // the scheduler's lanes' copies, and the segment
            rx::mbar_init(bar + 8 * (L::B_SEGEMPTY + i), W::SOFT + 2 * W::PROD + 3);
        }
        rx::mbar_init(bar + 8 * L::B_FINAL, 1);
        rx::mbar_init(bar + 8 * (L::B_FINAL + 1), 1);
        *reinterpret_cast<volatile int *>(smem + L::OFF_ABORT) = 0;
        rx::fence_mbar_init();
    }
    for (int i = threadIdx.x; i < kSegs * 32; i += kThreads) reinterpret_cast<uint32_t *>(smem + L::OFF_NF)[i] = 0;
    int64_t *pre = reinterpret_cast<int64_t *>(smem + L::OFF_MASK);
    const int per = (p.batch + kThreads - 1) / kThreads;
    const int64_t per_head = scan_units<kThreads>(p, pre, per, blockIdx.x == 0);
    const int64_t total = per_head * p.hkv;
    const int ctas = (int)min((int64_t)gridDim.x, total);
    if ((int)blockIdx.x >= ctas || total / ctas >= INT_MAX) {  // nothing to do, or lengths of no real pool
        if (threadIdx.x == 0) {
            p.cuts[blockIdx.x] = Cut{0, 0, 0, 0};
            if (ctas > 0 && total / ctas >= INT_MAX && p.status) atomicOr(p.status, RX_DEV_BAD_LEN);
        }
        return;
    }
    static_assert(sizeof(Start) <= 32, "the start's room");
    if (threadIdx.x == 0) {
        const int64_t u0 = first_unit(total, ctas, blockIdx.x);
        Req r;
        Start c = locate<kThreads>(p, pre, per, per_head, u0, r);
        c.left = (int)(first_unit(total, ctas, blockIdx.x + 1) - u0);
        *reinterpret_cast<Start *>(smem + L::OFF_START) = c;
    }
    if (warp == W::MMA) rx::tmem_alloc(sbase + L::OFF_TMEM, kTmemCols);
    rx::tc_fence_before();
    __syncthreads();  // from here on the scan's room holds masks
    rx::tc_fence_after();

    if (warp < W::SOFT) {
        rx::reg_inc<W::R_SOFT>();
        softmax_rows<D, F8, NT>(p, smem, sbase);
    } else if (warp < W::Q) {
        rx::reg_dec<W::R_REST>();
        if (warp < W::SOFT + W::PROD) producer<D, F8, NT, false>(p, smem, sbase);
        else producer<D, F8, NT, true>(p, smem, sbase);
    } else {
        rx::reg_dec<W::R_REST>();
        if (warp == W::Q) {
            query_loader<D, F8, NT>(p, smem, sbase);
        } else if (warp == W::MMA) {
            if ((threadIdx.x & 31) == 0) issue_qk<D, F8, NT>(p, smem, sbase);
            __syncwarp();
        } else if (warp == W::PV) {
            if ((threadIdx.x & 31) == 0) issue_pv<D, F8, NT>(p, smem, sbase);
            __syncwarp();
        } else if (warp == W::SCHED) {
            scheduler<D, F8>(p, smem, sbase);
        }
    }
    rx::tc_fence_before();
    __syncthreads();
    if (warp == W::MMA) {
        rx::tc_fence_after();
        rx::tmem_dealloc(*reinterpret_cast<volatile uint32_t *>(smem + L::OFF_TMEM), kTmemCols);
    }
}

// ---------------------------------------------------------------------------
// joining the partial results
// ---------------------------------------------------------------------------

// The parts of cut x = blockIdx.x, a warp a row: with m the largest
// log2-sum-exp, w = 2^(l - m): o = sum w o / sum w.  The first two parts'
// results are on their way before it has their weights; with four rows a warp,
// one after the other, the call for one small request took 17.5 us, with four
// rows' loads together 16, with one row 13.
template <int D>
__global__ void __launch_bounds__(kMergeThreads) tree_merge_kernel(const __grid_constant__ TParams p)
{
    const int x0 = (int)blockIdx.x;
    rx::pdl_wait();  // the cuts and the partial results are written by the kernel before this one
    const int4 raw = __ldcg(reinterpret_cast<const int4 *>(p.cuts + x0));
    const Cut c{raw.x, raw.y, raw.z, raw.w};
    const int parts = c.parts;
    if (parts == 0) return;

    constexpr int V = D / 32;  // values of a lane
    const int lane = threadIdx.x & 31;
    const int row = (int)blockIdx.y * kMergeRows + (int)(threadIdx.x >> 5);  // of the group's nt * 128
    const int t = row / kRows, r = row % kRows;
    if (t >= p.nt || r >= min(p.tb, c.ntok - t * p.tb) * p.G) return;
    using Vec = std::conditional_t<V == 4, float4, float2>;
    auto at = [&](int s) { return (int64_t)(2 * (x0 + s) + (s == 0 ? 1 : 0)) * p.nt * kRows + row; };
    auto part = [&](int s) { return __ldcg(reinterpret_cast<const Vec *>(p.part_o + at(s) * D) + lane); };
    const float l = lane < parts ? __ldcg(p.part_l + at(lane)) : -INFINITY;
    const Vec v0 = part(0), v1 = part(1);
    float m = l;
    for (int s = lane + 32; s < parts; s += 32) m = fmaxf(m, __ldcg(p.part_l + at(s)));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float mu = m == -INFINITY ? 0.f : m;
    float acc[V] = {}, tot = 0.f;
    auto add = [&](float ls, const Vec &x) {
        const float w = rx::fast_exp2(ls - mu);
        tot += w;
        acc[0] = fmaf(w, x.x, acc[0]);
        acc[1] = fmaf(w, x.y, acc[1]);
        if constexpr (V == 4) {
            acc[2] = fmaf(w, x.z, acc[2]);
            acc[3] = fmaf(w, x.w, acc[3]);
        }
    };
    add(__shfl_sync(0xffffffffu, l, 0), v0);
    add(__shfl_sync(0xffffffffu, l, 1), v1);
#pragma unroll 4
    for (int s = 2; s < parts; ++s) add(s < 32 ? __shfl_sync(0xffffffffu, l, s) : __ldcg(p.part_l + at(s)), part(s));
    const float inv = tot == 0.f ? 0.f : 1.f / tot;
    const int64_t orow = ((int64_t)c.tok + t * p.tb + r / p.G) * p.hq + (int64_t)c.g * p.G + r % p.G;
    uint32_t *dst = reinterpret_cast<uint32_t *>(p.o + orow * D + lane * V);
    dst[0] = rx::pack_bf16(acc[0] * inv, acc[1] * inv);
    if constexpr (V == 4) dst[1] = rx::pack_bf16(acc[2] * inv, acc[3] * inv);
    if (p.lse && lane == 0) p.lse[orow] = tot == 0.f ? -INFINITY : (m + log2f(tot)) * rx::kLn2;
}

size_t part_bytes(int32_t nt, int32_t head_dim) { return (size_t)2 * kCtas * nt * kRows * head_dim * sizeof(float); }

// Row tiles that share a K/V tile: two where some tree may have more than one
// (64-token trees over 64/8 heads, 8k contexts: 121 us, one at a time 134 us).
// The second brings softmax warps of its own; one group for both took 133 us.
// The call takes it for bf16 pools only: an FP8 tile has one query buffer, and
// the same trees over E4M3 pools gather every K/V tile once a row tile, 213 us.
// The workspace has room for either.
int row_tiles(int32_t hq, int32_t hkv, int32_t max_tree) { return (int64_t)max_tree > kRows / (hq / hkv) ? kMaxNt : 1; }

struct TreePool {
    const void *k, *v;
    int64_t num_slots;
    int hkv, D;
    bool f8;
    float k_scale, v_scale;
};

bool tree_shape_ok(int32_t batch, int32_t hq, int32_t hkv, int32_t D, int32_t max_tree)
{
    return batch >= 0 && batch <= 65535 && hq > 0 && hkv > 0 && hkv <= 8192 && hq % hkv == 0 && hq / hkv <= 128 &&
           (D == 64 || D == 128) && max_tree >= 1 && max_tree <= kMaxTree;
}

// The registers that the kernel is launched with: the shares of the roles are
// granted out of them, and a share that is not there would be waited for.
template <int D, bool F8, int NT>
bool registers_ok()
{
    cudaFuncAttributes a;
    return cudaFuncGetAttributes(&a, tree_kernel<D, F8, NT>) == cudaSuccess && a.numRegs >= Ro<NT>::R_LAUNCH;
}

template <int D, bool F8, int NT = 1>
int launch(const TParams &p, cudaStream_t st)
{
    static const bool ok = registers_ok<D, F8, NT>();
    if (!ok) return rx_set_error(RX_ERR_UNSUPPORTED, "tree attention: the kernel was built with too few registers");
    // per device; cheap, and right whichever device is current
    RX_CUDA_CHECK(cudaFuncSetAttribute(tree_kernel<D, F8, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (TL<D, F8>::BYTES)));
    tree_kernel<D, F8, NT><<<kCtas, Ro<NT>::THREADS, (TL<D, F8>::BYTES), st>>>(p);
    RX_CUDA_CHECK(cudaGetLastError());
    // a programmatic dependent: it is launched meanwhile and waits on the device
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCtas - 1, (unsigned)(p.nt == 1 ? (std::min(p.max_tree, p.tb) * p.G + kMergeRows - 1) / kMergeRows : p.nt * kRows / kMergeRows));
    cfg.blockDim = dim3(kMergeThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    RX_CUDA_CHECK(cudaLaunchKernelEx(&cfg, tree_merge_kernel<D>, p));
    return RX_OK;
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
    if (rx_misaligned16(q) || rx_misaligned16(o) || rx_misaligned16(pool.k) || rx_misaligned16(pool.v) ||
        (reinterpret_cast<uintptr_t>(lse) & 3) != 0 || (reinterpret_cast<uintptr_t>(mask) & 3) != 0)
        return rx_set_error(RX_ERR_INVALID, "%s: q, o and the pools must be 16-byte aligned", who);
    const float scale_log2 = sm_scale * pool.k_scale * rx::kLog2e;
    if (!(scale_log2 >= 0x1p-126f && scale_log2 < INFINITY))
        return rx_set_error(RX_ERR_INVALID, "%s: sm_scale %g (times K's scale %g) outside fp32's normal range", who, sm_scale,
                            pool.k_scale);
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
    p.k = (const unsigned char *)pool.k;
    p.v = (const unsigned char *)pool.v;
    p.num_slots = pool.num_slots;
    p.hq = hq;
    p.hkv = pool.hkv;
    p.G = hq / pool.hkv;
    p.tb = kRows / p.G;
    p.nt = pool.f8 ? 1 : row_tiles(hq, pool.hkv, max_tree);
    p.qo_indptr = qo_indptr;
    p.req_idx = req_idx;
    p.prefix_len = prefix_len;
    p.mask = mask;
    p.words = words;
    p.rtt = rtt;
    p.rtt_stride = rtt_stride;
    p.batch = batch;
    p.max_tree = max_tree;
    p.scale_log2 = scale_log2;
    p.v_scale = pool.v_scale;
    p.status = dev_status;
    p.part_o = (float *)workspace;
    p.part_l = (float *)((char *)workspace + part_bytes(p.nt, pool.D));
    p.cuts = (Cut *)(p.part_l + (size_t)2 * kCtas * p.nt * kRows);
    cudaStream_t st = (cudaStream_t)stream;
    if (pool.D == 128)
        return pool.f8 ? launch<128, true>(p, st) : p.nt == 1 ? launch<128, false>(p, st) : launch<128, false, kMaxNt>(p, st);
    return pool.f8 ? launch<64, true>(p, st) : p.nt == 1 ? launch<64, false>(p, st) : launch<64, false, kMaxNt>(p, st);
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
