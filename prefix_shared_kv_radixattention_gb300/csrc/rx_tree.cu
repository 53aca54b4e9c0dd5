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
//   - K/V rows are gathered through the slot list by eight producer warps with
//     16-byte loads into registers and stores into the swizzled tile that the
//     tensor core reads.  Rows of 256 bytes at random slots stream at 6.6 TB/s
//     this way with 64 KB in flight an SM (2.9 TB/s as bulk copies, 2.8 TB/s
//     through three warps of cp.async), so no copy of the context is needed
//     first;
//   - the work is cut evenly: the (kv head, request, row tile, position tile)
//     units are one long list of which every CTA takes a contiguous share; a
//     (kv head, request, row tile) cut by a CTA's end leaves fp32 partial
//     results that a second kernel joins by the log-sum-exp identity.  The
//     heads are outermost, so with 8 heads on 152 SMs nineteen CTAs walk each
//     head in step and the rows of one slot are read at about the same time;
//   - S = Q K^T goes to one of two TMEM buffers in turn, so that the tensor
//     core works on the next tile while four softmax warps (one row a thread)
//     turn this one into P, written over S and read from there by O += P V.
//
// All lengths are read on the device, by every CTA for itself: a scan of the
// batch's lengths in shared memory finds its share.
#include <math.h>

#include <algorithm>
#include <climits>

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
constexpr int kRows = 128;           // query rows of a tile (MMA M)
constexpr int kBN = 128;             // positions of a K/V tile
constexpr int kStages = 2;           // K ring and V ring depth
constexpr int kProdWarps = 8;        // for K, and as many for V
constexpr int kProdRows = kBN / kProdWarps;  // rows of a tile each producer warp gathers
constexpr int kSoftWarps = 4;        // one query row a thread
constexpr int kWarpQ = kSoftWarps + 2 * kProdWarps;  // loads the query rows
constexpr int kWarpMma = kWarpQ + 1;
constexpr int kThreads = 32 * (kWarpQ + 4);          // two warps idle: register shares go by warpgroup
// registers a thread, by role (a softmax thread holds a row's 128 scores):
// 128 x 192 + 512 x 56 + 128 x 56 of the 768 x 80 launched
constexpr int kRegsSoft = 192, kRegsProd = 56, kRegsMisc = 56, kRegsLaunch = 80;
static_assert(32 * (kSoftWarps * kRegsSoft + 2 * kProdWarps * kRegsProd + 4 * kRegsMisc) <= kThreads * kRegsLaunch,
              "a share is granted out of the launched registers only");
static_assert(kThreads * kRegsLaunch <= 65536, "registers of an SM");
constexpr int kRing = 4;             // per-segment words kept this many segments (see nf, qscale)
constexpr int kCodeBufs = 3;         // FP8: half tiles of codes in flight, for K and for V
constexpr uint32_t kTmemCols = 512;  // buffer i: S (then P) at 256 i, O at 256 i + 128
constexpr float kRescale = 8.f;      // log2 units the running max may lag
constexpr int kMergeRows = 16;       // rows of one merge CTA
constexpr int kMergeThreads = 128;

template <int D, bool F8>
struct TL {
    static constexpr int NB = D / 64;             // 128-byte column blocks of a row
    static constexpr int BLK = kRows * 128;       // bytes of one column block of a tile
    static constexpr int QB = F8 ? 1 : 2;         // query buffers (FP8: their room goes to the codes)
    static constexpr int CODE = F8 ? kBN * D / 2 : 0;  // bytes of half a tile of codes
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = OFF_Q + QB * NB * BLK;
    static constexpr int OFF_V = OFF_K + kStages * NB * BLK;
    static constexpr int OFF_CODE = OFF_V + kStages * NB * BLK;
    static constexpr int OFF_NF = OFF_CODE + 2 * kCodeBufs * CODE;        // kRing x 32 words
    static constexpr int OFF_QS = OFF_NF + kRing * 32 * 4;            // kRing x 128 floats
    static constexpr int OFF_SCAN = OFF_QS + kRing * kRows * 4;       // kThreads + 1 int64
    static constexpr int OFF_BAR = OFF_SCAN + (kThreads + 1) * 8;
    static constexpr int B_KFULL = 0, B_KEMPTY = B_KFULL + kStages, B_VFULL = B_KEMPTY + kStages,
                         B_VEMPTY = B_VFULL + kStages, B_QFULL = B_VEMPTY + kStages, B_QEMPTY = B_QFULL + QB,
                         B_SFULL = B_QEMPTY + QB, B_PFULL = B_SFULL + 2, B_PVDONE = B_PFULL + 2,
                         B_OEMPTY = B_PVDONE + 1, B_FINAL = B_OEMPTY + 2, N_BAR = B_FINAL + 1;
    static constexpr int OFF_TMEM = OFF_BAR + N_BAR * 8;
    static constexpr int OFF_ABORT = OFF_TMEM + 8;
    static constexpr int OFF_START = OFF_ABORT + 8;                   // Cursor of the CTA's first unit
    static constexpr int BYTES = OFF_START + 64 + 1024;               // + room to align the base to 1024
};
static_assert(TL<128, false>::BYTES <= 226 * 1024 && TL<128, true>::BYTES <= 226 * 1024, "shared memory budget");
static_assert(TL<128, false>::OFF_SCAN % 8 == 0 && TL<128, false>::OFF_BAR % 8 == 0, "alignment");

struct TParams {
    const bf16 *q;
    bf16 *o;
    float *lse;
    const unsigned char *k;
    const unsigned char *v;
    int64_t num_slots;
    int hq, hkv, G, tb;     // tb: drafted tokens of a row tile, 128 / G
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
    float *part_o;      // [2 kCtas][128][D] partial results, normalised
    float *part_l;      // [2 kCtas][128] their log2-sum-exps
    int32_t *status;
};

// ---------------------------------------------------------------------------
// the list of work
// ---------------------------------------------------------------------------

struct Req {
    int T, P;
    int row;          // of req_to_token
    int ntiles, nqt;  // 0 where there is nothing to do (no drafted token, or lengths out of range)

    __device__ __forceinline__ int64_t units() const { return (int64_t)ntiles * nqt; }
};

__device__ __forceinline__ Req load_req(const TParams &p, int b, bool flag = false)
{
    Req r;
    r.T = __ldg(p.qo_indptr + b + 1) - __ldg(p.qo_indptr + b);
    r.P = __ldg(p.prefix_len + b);
    r.row = __ldg(p.req_idx + b);
    r.ntiles = r.nqt = 0;
    if (r.T == 0) return r;
    if (r.T < 0 || r.T > p.max_tree || r.P < 0 || (int64_t)r.P + r.T > p.rtt_stride) {
        if (flag && p.status) atomicOr(p.status, RX_DEV_BAD_LEN);
        return r;
    }
    r.ntiles = (int)(((int64_t)r.P + r.T + kBN - 1) / kBN);
    r.nqt = (r.T + p.tb - 1) / p.tb;
    return r;
}

// A place in the list: kv head g, request b, row tile qt, position tile j.
struct Cursor {
    int left;  // units of this CTA from here on
    int g, b, qt, j;
    Req r;

    // position tiles of the segment (g, b, qt) that are this CTA's, from j on
    __device__ __forceinline__ int end() const { return left < r.ntiles - j ? j + left : r.ntiles; }
    // to the CTA's next segment; false when there is none
    __device__ __forceinline__ bool next(const TParams &p)
    {
        left -= end() - j;
        if (left <= 0) return false;
        j = 0;
        if (++qt < r.nqt) return true;
        qt = 0;
        do {
            if (++b == p.batch) {
                b = 0;
                ++g;
            }
            r = load_req(p, b);
        } while (r.ntiles == 0);
        return true;
    }
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

// The place of unit u (0 <= u < hkv * per_head).
template <int THREADS>
__device__ Cursor locate(const TParams &p, const int64_t *pre, int per, int64_t per_head, int64_t u)
{
    Cursor c;
    c.left = 0;
    c.g = (int)(u / per_head);
    int64_t r = u - c.g * per_head;
    int lo = 0, hi = THREADS - 1;  // the thread whose requests hold unit r
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (pre[mid] <= r) lo = mid; else hi = mid - 1;
    }
    r -= pre[lo];
    c.b = lo * per;
    for (c.r = load_req(p, c.b); r >= c.r.units(); c.r = load_req(p, c.b)) {
        r -= c.r.units();
        ++c.b;
    }
    c.qt = (int)(r / c.r.ntiles);
    c.j = (int)(r - (int64_t)c.qt * c.r.ntiles);
    return c;
}

// The CTA's first place, as thread 0 left it in shared memory.
template <typename L>
__device__ __forceinline__ Cursor start_of(const unsigned char *smem)
{
    const volatile int *w = reinterpret_cast<const volatile int *>(smem + L::OFF_START);
    Cursor c;
    int *d = reinterpret_cast<int *>(&c);
#pragma unroll
    for (int i = 0; i < (int)(sizeof(Cursor) / 4); ++i) d[i] = w[i];
    return c;
}

// First unit of CTA c out of `ctas` (no more CTAs than units: none is empty).
__device__ __forceinline__ int64_t first_unit(int64_t total, int ctas, int c) { return total * c / ctas; }

// ---------------------------------------------------------------------------
// which drafted tokens a row sees
// ---------------------------------------------------------------------------

// Word i of drafted token `node`'s mask: prefix positions (i < 0) are seen,
// bits at and past T are not.  Without branches around the load, so that the
// loads of several words go out together.
__device__ __forceinline__ uint32_t mask_word(const TParams &p, const uint32_t *row, int node, int T, int i)
{
    uint32_t w = 0xFFFFFFFFu;
    int n = T - 32 * i;  // drafted tokens from bit 0 of this word on
    if (row) w = __ldg(row + min(max(i, 0), p.words - 1));
    else n = min(n, node + 1 - 32 * i);
    w = n >= 32 ? w : n <= 0 ? 0u : w & ((1u << (n & 31)) - 1u);
    return i < 0 ? 0xFFFFFFFFu : w;
}

// ---------------------------------------------------------------------------
// producer warps
// ---------------------------------------------------------------------------

// Which halves of a word are NaN or infinite (bf16 / f16 pairs): 0xFFFF masks.
template <bool F8>
__device__ __forceinline__ uint32_t not_finite(uint32_t w)
{
    constexpr uint32_t E = F8 ? 0x7C00u : 0x7F80u;
    return ((w & E) == E ? 0xFFFFu : 0u) | ((w & (E << 16)) == (E << 16) ? 0xFFFF0000u : 0u);
}
template <bool F8>
__device__ __forceinline__ bool drop_not_finite(uint4 &x)
{
    const uint32_t a = not_finite<F8>(x.x), b = not_finite<F8>(x.y), c = not_finite<F8>(x.z), d = not_finite<F8>(x.w);
    x = make_uint4(x.x & ~a, x.y & ~b, x.z & ~c, x.w & ~d);
    return (a | b | c | d) != 0u;
}

// Eight E4M3 codes as eight f16 (exact).
__device__ __forceinline__ uint4 widen_f16(uint32_t lo, uint32_t hi)
{
    return make_uint4(rx::e4m3x2_to_f16x2((uint16_t)lo), rx::e4m3x2_to_f16x2((uint16_t)(lo >> 16)),
                      rx::e4m3x2_to_f16x2((uint16_t)hi), rx::e4m3x2_to_f16x2((uint16_t)(hi >> 16)));
}

// Eight producer warps for K and eight for V (V's wait for the softmax does
// not hold up K); warp w gathers rows [16 w, 16 w + 16) of every tile with
// 16-byte async copies, slot ids two tiles ahead.  (Loads into registers go
// through L1, which this kernel's shared memory leaves 28 KB: with 64 KB meant
// to be in flight they ran at half the rate.)
//
// bf16 pools: the copies land in the swizzled tile itself and report to its
// barrier.  FP8 pools: they land in a ring of three half tiles of codes; each
// thread widens the chunks that it copied (E4M3 to f16 is exact) and stores
// them to the tile.
//
// V at drafted positions passes through registers in both: a NaN or infinity
// there would reach rows that do not see the position (0 * inf), so it is
// dropped, noted, and added back to the rows that see it at the end.
template <int D, bool F8, bool IS_V>
__device__ void producer(const TParams &p, unsigned char *smem, uint32_t sbase)
{
    using L = TL<D, F8>;
    Cursor c = start_of<L>(smem);
    constexpr int EB = F8 ? 1 : 2;                    // bytes of a value
    constexpr int CPR = D * EB / 16;                  // 16-byte chunks of a row
    constexpr int RPI = 32 / CPR;                     // rows of one instruction
    constexpr int U = kProdRows / RPI;                // instructions for this warp's rows
    const uint32_t bar_full = sbase + L::OFF_BAR + 8 * (IS_V ? L::B_VFULL : L::B_KFULL);
    const uint32_t bar_empty = sbase + L::OFF_BAR + 8 * (IS_V ? L::B_VEMPTY : L::B_KEMPTY);
    const unsigned char *pool = IS_V ? p.v : p.k;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::OFF_ABORT);
    const int lane = threadIdx.x & 31, pw = ((int)(threadIdx.x >> 5) - kSoftWarps) % kProdWarps;
    const int r0 = pw * kProdRows;
    const int sub = lane / CPR, ch = lane % CPR;
    const int row_bytes = p.hkv * D * EB;             // at most 2^15 heads (host check)

    struct Tile {
        int32_t slot;  // lane l < 16: slot of row r0 + l, in flight until check() looks at it
        int g;
        int rel;       // the tile's first position, from the first drafted one
        int seg;       // segment mod kRing; -1: no tile
        bool in;       // row r0 + l is a position of the request
    };
    int seg = 0;
    // the tile at the cursor, with the loads of its slot ids; then on to the next
    auto take = [&](Tile &t) {
        t.seg = t.slot = -1;
        t.g = t.rel = 0;
        t.in = false;
        if (c.left <= 0) return;
        t.g = c.g;
        t.rel = c.j * kBN - c.r.P;
        t.seg = seg % kRing;
        const int pos = c.j * kBN + r0 + lane;
        t.in = lane < kProdRows && pos < c.r.P + c.r.T;
        if (t.in) t.slot = rx::ld_stream_b32(p.rtt + (int64_t)c.r.row * p.rtt_stride + pos);
        if (c.j + 1 < c.r.ntiles) {
            ++c.j;
            --c.left;
        } else {
            ++seg;
            c.next(p);  // the tile at j is the segment's last
        }
    };
    // slots past the end or outside the pool (flagged) become -1
    auto check = [&](Tile &t) {
        const bool ok = t.in && t.slot >= 0 && (int64_t)t.slot < p.num_slots;
        if (t.in && !ok && p.status) atomicOr(p.status, RX_DEV_BAD_SLOT);
        if (!ok) t.slot = -1;
    };
    auto source = [&](const Tile &t, int u, bool &ok) {
        const int32_t s = __shfl_sync(0xffffffffu, t.slot, u * RPI + sub);
        ok = s >= 0;
        return pool + (ok ? (int64_t)s * row_bytes : 0) + (t.g * (D * EB) + ch * 16);
    };
    auto note = [&](const Tile &t, int r) {
        const int e = t.rel + r;
        atomicOr(reinterpret_cast<uint32_t *>(smem + L::OFF_NF) + t.seg * 32 + (e >> 5), 1u << (e & 31));
    };

    Tile cur, nxt, nx2;
    take(cur);
    take(nxt);
    if constexpr (!F8) {
        for (int n = 0; cur.seg >= 0; ++n) {
            const int st = n % kStages;
            take(nx2);
            check(cur);
            const uint32_t off = (IS_V ? L::OFF_V : L::OFF_K) + st * L::NB * L::BLK;
            if (n >= kStages && !warp_wait(bar_empty + 8 * st, (n / kStages - 1) & 1, abort_flag, p.status)) break;
            if (!IS_V || cur.rel + kBN <= 0) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    bool ok;
                    const unsigned char *src = source(cur, u, ok);
                    rx::cp_async_16(sbase + off + sw128(r0 + u * RPI + sub, ch, L::BLK), src, ok ? 16 : 0);
                }
                rx::cp_async_mbar_arrive(bar_full + 8 * st);
            } else {
                constexpr int H = U / 2;  // half the rows at a time
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint4 x[H];
#pragma unroll
                    for (int u = 0; u < H; ++u) {
                        bool ok;
                        const unsigned char *src = source(cur, h * H + u, ok);
                        x[u] = make_uint4(0, 0, 0, 0);
                        if (ok) x[u] = rx::ld_stream(src);
                    }
#pragma unroll
                    for (int u = 0; u < H; ++u) {
                        const int r = r0 + (h * H + u) * RPI + sub;
                        if (cur.rel + r >= 0 && drop_not_finite<false>(x[u])) note(cur, r);
                        *reinterpret_cast<uint4 *>(smem + off + sw128(r, ch, L::BLK)) = x[u];
                    }
                }
                rx::fence_proxy_async_smem();
                rx::mbar_arrive(bar_full + 8 * st);
            }
            cur = nxt;
            nxt = nx2;
        }
    } else {
        constexpr int H = U / 2;  // instructions of half a tile
        // chunk u of half-tile buffer b: + b CODE + 512 u
        const uint32_t mine = L::OFF_CODE + (IS_V ? kCodeBufs * L::CODE : 0) + (uint32_t)(pw * H * 32 + lane) * 16;
        auto fetch = [&](const Tile &t, int item) {  // item = 2 n + half
#pragma unroll
            for (int u = 0; u < H; ++u) {
                bool ok;
                const unsigned char *src = source(t, (item & 1) * H + u, ok);
                rx::cp_async_16(sbase + mine + (item % kCodeBufs) * L::CODE + u * 512, src, ok ? 16 : 0);
            }
            rx::cp_async_commit();
        };
        // this thread's chunks of a landed half into the tile at `off`
        auto widen = [&](uint32_t off, const Tile &t, int item) {
            const bool drafted = IS_V && t.rel + kBN > 0;
#pragma unroll
            for (int u = 0; u < H; ++u) {
                const uint4 x = *reinterpret_cast<const uint4 *>(smem + mine + (item % kCodeBufs) * L::CODE + u * 512);
                uint4 a = widen_f16(x.x, x.y), b = widen_f16(x.z, x.w);
                const int r = r0 + ((item & 1) * H + u) * RPI + sub;
                if (drafted && t.rel + r >= 0) {
                    bool nf = drop_not_finite<true>(a);
                    nf |= drop_not_finite<true>(b);
                    if (nf) note(t, r);
                }
                // the upper lanes of a row store their second chunk first: the
                // two column blocks of a row lie on the same banks
                const int swap = D == 128 ? (ch >> 2) & 1 : 0;
                *reinterpret_cast<uint4 *>(smem + off + sw128(r, 2 * ch + swap, L::BLK)) = swap ? b : a;
                *reinterpret_cast<uint4 *>(smem + off + sw128(r, 2 * ch + 1 - swap, L::BLK)) = swap ? a : b;
            }
        };
        check(cur);
        check(nxt);
        fetch(cur, 0);
        fetch(cur, 1);
        fetch(nxt, 2);
        for (int n = 0; cur.seg >= 0; ++n) {
            const int st = n % kStages;
            const uint32_t off = (IS_V ? L::OFF_V : L::OFF_K) + st * L::NB * L::BLK;
            take(nx2);
            rx::cp_async_wait<2>();     // the first half of tile n
            if (n >= kStages && !warp_wait(bar_empty + 8 * st, (n / kStages - 1) & 1, abort_flag, p.status)) break;
            widen(off, cur, 2 * n);
            fetch(nxt, 2 * n + 3);
            rx::cp_async_wait<2>();     // the second
            widen(off, cur, 2 * n + 1);
            rx::fence_proxy_async_smem();
            rx::mbar_arrive(bar_full + 8 * st);
            check(nx2);
            fetch(nx2, 2 * n + 4);
            cur = nxt;
            nxt = nx2;
        }
    }
    rx::cp_async_wait_all();  // nothing may still be landing when the CTA exits
}

// ---------------------------------------------------------------------------
// query rows
// ---------------------------------------------------------------------------

// One warp copies each segment's query rows (row r: drafted token r / G of the
// row tile, q head g G + r % G) into a query buffer.  bf16 pools: 16-byte
// async copies.  FP8 pools: the products run in f16, which holds every E4M3
// value; a query row is brought to f16 times a power of two that puts its
// largest value just below 2^15 (values 2^-29 of that and above stay exact),
// and the power goes into the row's score scale.
template <int D, bool F8>
__device__ void query_loader(const TParams &p, unsigned char *smem, uint32_t sbase)
{
    using L = TL<D, F8>;
    Cursor c = start_of<L>(smem);
    constexpr int CPR = D / 8;
    const uint32_t bar = sbase + L::OFF_BAR;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::OFF_ABORT);
    const int lane = threadIdx.x & 31;
    for (int s = 0;; ++s) {
        const int buf = s % L::QB;
        const int t0 = c.qt * p.tb, M = min(p.tb, c.r.T - t0) * p.G;
        const int64_t tok0 = (int64_t)__ldg(p.qo_indptr + c.b) + t0;
        if (s >= L::QB && !warp_wait(bar + 8 * (L::B_QEMPTY + buf), (s / L::QB - 1) & 1, abort_flag, p.status)) break;
        const uint32_t dst = sbase + L::OFF_Q + buf * L::NB * L::BLK;
        for (int i0 = 0; i0 < M * CPR; i0 += 32) {
            const int i = i0 + lane, r = i / CPR, ch = i % CPR;
            const bool in = i < M * CPR;
            const bf16 *src = in ? p.q + ((tok0 + r / p.G) * p.hq + (int64_t)c.g * p.G + r % p.G) * D + ch * 8 : p.q;
            if constexpr (!F8) {
                if (in) rx::cp_async_16(dst + sw128(r, ch, L::BLK), src, 16);
            } else {
                uint4 x = make_uint4(0, 0, 0, 0);
                if (in) x = __ldg(reinterpret_cast<const uint4 *>(src));
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
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
                if (in) {
                    *reinterpret_cast<uint4 *>(smem + (dst - sbase) + sw128(r, ch, L::BLK)) = make_uint4(y[0], y[1], y[2], y[3]);
                    if (ch == 0)
                        reinterpret_cast<float *>(smem + L::OFF_QS)[(s % kRing) * kRows + r] =
                            __uint_as_float((uint32_t)(127 - 14 + e) << 23);
                }
            }
        }
        if constexpr (F8) {
            rx::fence_proxy_async_smem();
            rx::mbar_arrive(bar + 8 * (L::B_QFULL + buf));
        } else {
            rx::cp_async_mbar_arrive(bar + 8 * (L::B_QFULL + buf));
        }
        if (!c.next(p)) break;
    }
    rx::cp_async_wait_all();
}

// ---------------------------------------------------------------------------
// MMA thread
// ---------------------------------------------------------------------------

// Over the CTA's tiles n = 0, 1, ... (all segments in a row): S(n) into buffer
// n & 1, then O += P V of tile n - 1, O of segment s in buffer s & 1.  P(n - 2)
// sits in the columns that S(n) overwrites, so S(n) waits for that product's
// completion.
template <int D, bool F8>
__device__ void mma_issuer(const TParams &p, unsigned char *smem, uint32_t sbase)
{
    using L = TL<D, F8>;
    Cursor c = start_of<L>(smem);
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + L::OFF_TMEM);
    const uint32_t bar = sbase + L::OFF_BAR;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::OFF_ABORT);
    constexpr uint32_t idesc_qk = F8 ? rx::idesc_f16(kRows, kBN, false, false) : rx::idesc_bf16(kRows, kBN, false, false);
    constexpr uint32_t idesc_pv = F8 ? rx::idesc_f16(kRows, D, false, true) : rx::idesc_bf16(kRows, D, false, true);
    auto wait = [&](int b, uint32_t parity) { return wait_or_abort(bar + 8 * b, parity, abort_flag, p.status); };
    const uint64_t dq = rx::sdesc_sw128(sbase + L::OFF_Q, 16, 1024);
    const uint64_t dk = rx::sdesc_sw128(sbase + L::OFF_K, 16, 1024);
    const uint64_t dv = rx::sdesc_sw128(sbase + L::OFF_V, L::BLK, 1024);

    auto issue_s = [&](int n, int s, bool first, bool last) -> bool {
        const int st = n % kStages, buf = n & 1;
        if (first && !wait(L::B_QFULL + s % L::QB, (s / L::QB) & 1)) return false;
        if (!wait(L::B_KFULL + st, (n / kStages) & 1)) return false;
        if (n >= 2 && !wait(L::B_PVDONE, n & 1)) return false;  // O += P V of tile n - 2 (the same parity)
        rx::fence_proxy_async_smem();  // rows landed by cp.async -> async proxy
        rx::tc_fence_after();
        const uint64_t dks = dk + (uint64_t)((st * L::NB * L::BLK) >> 4);
        const uint64_t dqs = dq + (uint64_t)(((s % L::QB) * L::NB * L::BLK) >> 4);
#pragma unroll
        for (int kb = 0; kb < D / 16; ++kb) {
            const uint64_t off = (uint64_t)(((kb >> 2) * L::BLK + (kb & 3) * 32) >> 4);
            rx::tc_mma(tmem + buf * 256, dqs + off, dks + off, idesc_qk, kb > 0);
        }
        rx::tc_commit(bar + 8 * (L::B_SFULL + buf));
        rx::tc_commit(bar + 8 * (L::B_KEMPTY + st));
        if (last) rx::tc_commit(bar + 8 * (L::B_QEMPTY + s % L::QB));
        return true;
    };
    auto issue_pv = [&](int n, int s, bool first) -> bool {
        const int st = n % kStages, buf = n & 1;
        if (!wait(L::B_PFULL + buf, (n >> 1) & 1)) return false;
        if (!wait(L::B_VFULL + st, (n / kStages) & 1)) return false;
        if (first && s >= 2 && !wait(L::B_OEMPTY + (s & 1), ((s >> 1) - 1) & 1)) return false;
        rx::fence_proxy_async_smem();  // V rows landed by cp.async
        rx::tc_fence_after();
        const uint64_t dvs = dv + (uint64_t)((st * L::NB * L::BLK) >> 4);
#pragma unroll
        for (int ks = 0; ks < kBN / 16; ++ks)
            rx::tc_mma_ts(tmem + (s & 1) * 256 + 128, tmem + buf * 256 + ks * 8, dvs + (uint64_t)((ks * 16 * 128) >> 4),
                          idesc_pv, (!first || ks > 0) ? 1u : 0u);
        rx::tc_commit(bar + 8 * L::B_PVDONE);
        rx::tc_commit(bar + 8 * (L::B_VEMPTY + st));
        return true;
    };
    bool ok = true, prev_first = false;
    int n = 0, prev_s = 0;
    for (int s = 0; ok; ++s) {
        const int j0 = c.j, j1 = c.end();
        for (int j = j0; j < j1 && ok; ++j, ++n) {
            ok = issue_s(n, s, j == j0, j == j1 - 1);
            if (ok && n > 0) ok = issue_pv(n - 1, prev_s, prev_first);
            prev_s = s;
            prev_first = j == j0;
        }
        if (!ok || !c.next(p)) break;
    }
    if (ok) issue_pv(n - 1, prev_s, prev_first);
    // everything issued has finished before TMEM is released
    rx::tc_commit(bar + 8 * L::B_FINAL);
    rx::drain_wait(bar + 8 * L::B_FINAL, 0, p.status);
}

// ---------------------------------------------------------------------------
// softmax warps: one query row per thread
// ---------------------------------------------------------------------------

// The NaN and infinities of V at drafted positions that a row sees, added to
// its written result: o (part < 0) or the partial row `part`.
template <int D, bool F8>
__device__ __noinline__ void add_not_finite(const TParams &p, const uint32_t *nf, const uint32_t *mrow, int node, int b,
                                            int g, int P, int T, int64_t part, int64_t orow)
{
    for (int w = 0; w < (T + 31) / 32; ++w)
        for (uint32_t bad = nf[w] & mask_word(p, mrow, node, T, w); bad; bad &= bad - 1) {
            const int pos = P + 32 * w + __ffs(bad) - 1;
            const int64_t slot = __ldg(p.rtt + (int64_t)__ldg(p.req_idx + b) * p.rtt_stride + pos);
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

template <int D, bool F8>
__device__ void softmax_rows(const TParams &p, unsigned char *smem, uint32_t sbase)
{
    using L = TL<D, F8>;
    Cursor c = start_of<L>(smem);
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + L::OFF_TMEM);
    const uint32_t bar = sbase + L::OFF_BAR;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::OFF_ABORT);
    const int row = threadIdx.x;                       // = TMEM lane
    const uint32_t lanes = (uint32_t)(row & ~31) << 16;
    int n = 0;
    for (int s = 0;; ++s) {
        const int j0 = c.j, j1 = c.end(), P = c.r.P, T = c.r.T;
        const int t0 = c.qt * p.tb, M = min(p.tb, T - t0) * p.G;
        const bool valid = row < M, warp_on = (row & ~31) < M;
        const int node = t0 + row / p.G;
        const int64_t tok = (int64_t)__ldg(p.qo_indptr + c.b) + node;
        const uint32_t *mrow = p.mask && valid ? p.mask + tok * p.words : nullptr;
        const uint32_t tO = tmem + (s & 1) * 256 + 128 + lanes;
        float m_used = -INFINITY, l = 0.f, sl2 = p.scale_log2;
        for (int j = j0; j < j1; ++j, ++n) {
            const int buf = n & 1;
            const uint32_t tS = tmem + buf * 256 + lanes;
            if (!warp_wait(bar + 8 * (L::B_SFULL + buf), (n >> 1) & 1, abort_flag, p.status)) return;
            rx::tc_fence_after();
            if (warp_on) {
                // the row's scores of this tile, loaded once (four loads in
                // flight): a load takes about 200 cycles to come back
                uint32_t sv[kBN];
#pragma unroll
                for (int k = 0; k < kBN / 32; ++k) rx::tmem_ld32(tS + k * 32, *reinterpret_cast<uint32_t(*)[32]>(sv + 32 * k));
                if (F8 && j == j0) sl2 = p.scale_log2 * reinterpret_cast<const float *>(smem + L::OFF_QS)[(s % kRing) * kRows + row];
                const int kbase = j * kBN;
                if (kbase + kBN > P) {   // drafted positions, or past the last
                    const int off = kbase - P, w0 = off >> 5;
                    uint32_t w[5];
#pragma unroll
                    for (int k = 0; k < 5; ++k) w[k] = mask_word(p, mrow, node, T, w0 + k);
                    rx::tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < kBN / 32; ++k) {
                        const uint32_t bits = __funnelshift_r(w[k], w[k + 1], off & 31);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!((bits >> i) & 1u)) sv[32 * k + i] = 0xFF800000u;  // -inf
                    }
                } else {
                    rx::tmem_wait_ld();
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
                const float m_new = fmaxf(m_used, mx * sl2);
                const bool need = valid && (m_used == -INFINITY || m_new > m_used + kRescale);
                const bool scale_o = need && m_used != -INFINITY;
                const float alpha = scale_o ? rx::fast_exp2(m_used - m_new) : 1.f;
                if (need) {
                    l *= alpha;
                    m_used = m_new;
                }
                const float mu = m_used == -INFINITY ? 0.f : m_used;
                const uint64_t scale2 = rx::f2(sl2, sl2), negm2 = rx::f2(-mu, -mu);
                uint64_t acc[4] = {0, 0, 0, 0};
#pragma unroll
                for (int k = 0; k < kBN / 64; ++k) {
                    uint32_t pk[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        float x0, x1;
                        rx::f2_split(rx::f2_fma(rx::f2(u2f(sv[64 * k + 2 * i]), u2f(sv[64 * k + 2 * i + 1])), scale2, negm2), x0, x1);
                        const float e0 = rx::fast_exp2(x0), e1 = rx::fast_exp2(x1);
                        acc[i & 3] = rx::f2_add(acc[i & 3], rx::f2(e0, e1));
                        // the weights are rounded to the type of V's tile for
                        // the tensor core; their sum is not
                        pk[i] = F8 ? rx::pack_f16(e0, e1) : rx::pack_bf16(e0, e1);
                    }
                    rx::tmem_st32(tS + k * 32, pk);  // over scores already read
                }
                float a0, a1;
                rx::f2_split(rx::f2_add(rx::f2_add(acc[0], acc[1]), rx::f2_add(acc[2], acc[3])), a0, a1);
                l += a0 + a1;
                if (__any_sync(0xffffffffu, scale_o)) {
                    // O += P V of the tile before has to be complete
                    if (!warp_wait(bar + 8 * L::B_PVDONE, (n - 1) & 1, abort_flag, p.status)) return;
                    rx::tc_fence_after();
#pragma unroll
                    for (int k = 0; k < D / 32; ++k) {
                        uint32_t x[32];
                        rx::tmem_ld32(tO + k * 32, x);
                        rx::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(u2f(x[i]) * alpha);
                        rx::tmem_st32(tO + k * 32, x);
                    }
                }
                rx::tmem_wait_st();
            }
            rx::tc_fence_before();
            rx::mbar_arrive(bar + 8 * (L::B_PFULL + buf));
        }
        // the segment's result
        if (!warp_wait(bar + 8 * L::B_PVDONE, (n - 1) & 1, abort_flag, p.status)) return;
        rx::tc_fence_after();
        uint32_t *nf = reinterpret_cast<uint32_t *>(smem + L::OFF_NF) + (s % kRing) * 32;
        uint32_t any = 0;
        if (j1 * kBN > P)
            for (int i = 0; i < (T + 31) / 32; ++i) any |= nf[i];
        const bool whole = j0 == 0 && j1 == c.r.ntiles;
        const float inv = l == 0.f ? 0.f : p.v_scale / l;
        const int64_t orow = tok * p.hq + (int64_t)c.g * p.G + row % p.G;
        const int64_t prow = (int64_t)(2 * blockIdx.x + (j0 == 0 ? 1 : 0)) * kRows + row;
        if (warp_on) {
            uint32_t r[D];
#pragma unroll
            for (int k = 0; k < D / 32; ++k) rx::tmem_ld32(tO + k * 32, *reinterpret_cast<uint32_t(*)[32]>(r + 32 * k));
            rx::tmem_wait_ld();
            if (valid) {
                if (whole) {
                    uint4 *dst = reinterpret_cast<uint4 *>(p.o + orow * D);
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {
                        uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) w[k] = rx::pack_bf16(u2f(r[8 * i + 2 * k]) * inv, u2f(r[8 * i + 2 * k + 1]) * inv);
                        dst[i] = l == 0.f ? make_uint4(0, 0, 0, 0) : make_uint4(w[0], w[1], w[2], w[3]);
                    }
                } else {
                    float4 *dst = reinterpret_cast<float4 *>(p.part_o + prow * D);
#pragma unroll
                    for (int i = 0; i < D / 4; ++i)
                        dst[i] = l == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                                          : make_float4(u2f(r[4 * i]) * inv, u2f(r[4 * i + 1]) * inv,
                                                        u2f(r[4 * i + 2]) * inv, u2f(r[4 * i + 3]) * inv);
                }
                const float l2 = l == 0.f ? -INFINITY : m_used + log2f(l);
                if (!whole) p.part_l[prow] = l2;
                else if (p.lse) p.lse[orow] = l2 * rx::kLn2;
            }
            __syncwarp();
        }
        rx::tc_fence_before();
        rx::mbar_arrive(bar + 8 * (L::B_OEMPTY + (s & 1)));
        if (any) {  // the same for every thread: all have read the words, then they are cleared
            if (valid) add_not_finite<D, F8>(p, nf, mrow, node, c.b, c.g, P, T, whole ? -1 : prow, orow);
            rx::named_bar_sync(1, 32 * kSoftWarps);
            if (row < 32) nf[row] = 0;
        }
        if (!c.next(p)) return;
    }
}

template <int D, bool F8>
__global__ void __launch_bounds__(kThreads, 1) tree_kernel(const __grid_constant__ TParams p)
{
    using L = TL<D, F8>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = rx::smem_u32(smem_raw);
    unsigned char *smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);  // 1024-aligned swizzle atoms
    const uint32_t sbase = rx::smem_u32(smem);
    const uint32_t bar = sbase + L::OFF_BAR;
    const int warp = threadIdx.x >> 5;
    rx::pdl_launch_dependents();  // the merge kernel may launch and wait on the device

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            rx::mbar_init(bar + 8 * (L::B_KFULL + i), 32 * kProdWarps);
            rx::mbar_init(bar + 8 * (L::B_VFULL + i), 32 * kProdWarps);
            rx::mbar_init(bar + 8 * (L::B_KEMPTY + i), 1);
            rx::mbar_init(bar + 8 * (L::B_VEMPTY + i), 1);
        }
        for (int i = 0; i < L::QB; ++i) {
            rx::mbar_init(bar + 8 * (L::B_QFULL + i), 32);
            rx::mbar_init(bar + 8 * (L::B_QEMPTY + i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            rx::mbar_init(bar + 8 * (L::B_SFULL + i), 1);
            rx::mbar_init(bar + 8 * (L::B_PFULL + i), kRows);
            rx::mbar_init(bar + 8 * (L::B_OEMPTY + i), kRows);
        }
        rx::mbar_init(bar + 8 * L::B_PVDONE, 1);
        rx::mbar_init(bar + 8 * L::B_FINAL, 1);
        *reinterpret_cast<volatile int *>(smem + L::OFF_ABORT) = 0;
        rx::fence_mbar_init();
    }
    for (int i = threadIdx.x; i < kRing * 32; i += kThreads) reinterpret_cast<uint32_t *>(smem + L::OFF_NF)[i] = 0;
    int64_t *pre = reinterpret_cast<int64_t *>(smem + L::OFF_SCAN);
    const int per = (p.batch + kThreads - 1) / kThreads;
    const int64_t per_head = scan_units<kThreads>(p, pre, per, blockIdx.x == 0);
    const int64_t total = per_head * p.hkv;
    const int ctas = (int)min((int64_t)gridDim.x, total);
    if ((int)blockIdx.x >= ctas) return;
    if (total / ctas >= INT_MAX) {  // lengths of no real pool
        if (p.status && threadIdx.x == 0) atomicOr(p.status, RX_DEV_BAD_LEN);
        return;
    }
    static_assert(sizeof(Cursor) <= 64, "the start cursor's room");
    if (threadIdx.x == 0) {
        const int64_t u0 = first_unit(total, ctas, blockIdx.x);
        Cursor c = locate<kThreads>(p, pre, per, per_head, u0);
        c.left = (int)(first_unit(total, ctas, blockIdx.x + 1) - u0);
        *reinterpret_cast<Cursor *>(smem + L::OFF_START) = c;
    }
    if (warp == kWarpMma) rx::tmem_alloc(sbase + L::OFF_TMEM, kTmemCols);
    rx::tc_fence_before();
    __syncthreads();
    rx::tc_fence_after();

    if (warp < kSoftWarps) {
        rx::reg_inc<kRegsSoft>();
        softmax_rows<D, F8>(p, smem, sbase);
    } else if (warp < kWarpQ) {
        rx::reg_dec<kRegsProd>();
        if (warp < kSoftWarps + kProdWarps) producer<D, F8, false>(p, smem, sbase);
        else producer<D, F8, true>(p, smem, sbase);
    } else {
        rx::reg_dec<kRegsMisc>();
        if (warp == kWarpQ) {
            query_loader<D, F8>(p, smem, sbase);
        } else if (warp == kWarpMma) {
            if ((threadIdx.x & 31) == 0) mma_issuer<D, F8>(p, smem, sbase);
            __syncwarp();
        }
    }
    rx::tc_fence_before();
    __syncthreads();
    if (warp == kWarpMma) {
        rx::tc_fence_after();
        rx::tmem_dealloc(*reinterpret_cast<volatile uint32_t *>(smem + L::OFF_TMEM), kTmemCols);
    }
}

// ---------------------------------------------------------------------------
// joining the partial results
// ---------------------------------------------------------------------------

// The (kv head, request, row tile) that the boundary between CTAs x and x + 1
// cuts, x = blockIdx.x, when it is the first boundary inside: its parts are
// CTA x's last segment (slot 1) and the first segments (slot 0) of the CTAs
// after it, as far as it reaches.  One warp a row: with m the largest
// log2-sum-exp, w = 2^(l - m): o = sum w o / sum w.  kMergeRows rows a CTA.
template <int D>
__global__ void __launch_bounds__(kMergeThreads) tree_merge_kernel(const __grid_constant__ TParams p, int main_ctas)
{
    __shared__ int64_t pre[kMergeThreads + 1];
    const int per = (p.batch + kMergeThreads - 1) / kMergeThreads;
    const int64_t per_head = scan_units<kMergeThreads>(p, pre, per, false);
    const int64_t total = per_head * p.hkv;
    const int ctas = (int)min((int64_t)main_ctas, total);
    const int x0 = (int)blockIdx.x;
    rx::pdl_wait();  // the partial results are written by the kernel before this one
    if (x0 + 1 >= ctas || total / ctas >= INT_MAX) return;
    const int64_t cut = first_unit(total, ctas, x0 + 1);
    const Cursor c = locate<kMergeThreads>(p, pre, per, per_head, cut);
    const int64_t begin = cut - c.j, end = begin + c.r.ntiles;
    if (c.j == 0 || begin < first_unit(total, ctas, x0)) return;
    int parts = 2;
    while (x0 + parts < ctas && first_unit(total, ctas, x0 + parts) < end) ++parts;

    constexpr int V = D / 32;  // values of a lane
    const int lane = threadIdx.x & 31;
    const int t0 = c.qt * p.tb, M = min(p.tb, c.r.T - t0) * p.G;
    const int64_t tok0 = (int64_t)__ldg(p.qo_indptr + c.b) + t0;
    for (int i = threadIdx.x >> 5; i < kMergeRows; i += kMergeThreads / 32) {
        const int row = (int)blockIdx.y * kMergeRows + i;
        if (row >= M) break;
        auto at = [&](int s) { return (int64_t)(2 * (x0 + s) + (s == 0 ? 1 : 0)) * kRows + row; };
        float m = -INFINITY;
        for (int s = lane; s < parts; s += 32) m = fmaxf(m, __ldcg(p.part_l + at(s)));
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        const float mu = m == -INFINITY ? 0.f : m;
        float acc[V] = {}, tot = 0.f;
#pragma unroll 4
        for (int s = 0; s < parts; ++s) {
            const float w = exp2f(__ldcg(p.part_l + at(s)) - mu);
            const float *src = p.part_o + at(s) * D + lane * V;
            tot += w;
            if constexpr (V == 4) {
                const float4 v = __ldcg(reinterpret_cast<const float4 *>(src));
                acc[0] = fmaf(w, v.x, acc[0]);
                acc[1] = fmaf(w, v.y, acc[1]);
                acc[2] = fmaf(w, v.z, acc[2]);
                acc[3] = fmaf(w, v.w, acc[3]);
            } else {
                const float2 v = __ldcg(reinterpret_cast<const float2 *>(src));
                acc[0] = fmaf(w, v.x, acc[0]);
                acc[1] = fmaf(w, v.y, acc[1]);
            }
        }
        const float inv = tot == 0.f ? 0.f : 1.f / tot;
        const int64_t orow = (tok0 + row / p.G) * p.hq + (int64_t)c.g * p.G + row % p.G;
        uint32_t *dst = reinterpret_cast<uint32_t *>(p.o + orow * D + lane * V);
        dst[0] = rx::pack_bf16(acc[0] * inv, acc[1] * inv);
        if constexpr (V == 4) dst[1] = rx::pack_bf16(acc[2] * inv, acc[3] * inv);
        if (p.lse && lane == 0) p.lse[orow] = tot == 0.f ? -INFINITY : (m + log2f(tot)) * rx::kLn2;
    }
}

size_t part_bytes(int32_t head_dim) { return (size_t)2 * kCtas * kRows * head_dim * sizeof(float); }

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

template <int D, bool F8>
int launch(const TParams &p, cudaStream_t st)
{
    // per device; cheap, and right whichever device is current
    RX_CUDA_CHECK(cudaFuncSetAttribute(tree_kernel<D, F8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (TL<D, F8>::BYTES)));
    tree_kernel<D, F8><<<kCtas, kThreads, (TL<D, F8>::BYTES), st>>>(p);
    RX_CUDA_CHECK(cudaGetLastError());
    // a programmatic dependent: it finds its part of the work, then waits on the device
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCtas - 1, (unsigned)((std::min(p.max_tree, p.tb) * p.G + kMergeRows - 1) / kMergeRows));
    cfg.blockDim = dim3(kMergeThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    RX_CUDA_CHECK(cudaLaunchKernelEx(&cfg, tree_merge_kernel<D>, p, (int)kCtas));
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
    p.part_o = (float *)workspace;
    p.part_l = (float *)((char *)workspace + part_bytes(pool.D));
    cudaStream_t st = (cudaStream_t)stream;
    if (pool.D == 128) return pool.f8 ? launch<128, true>(p, st) : launch<128, false>(p, st);
    return pool.f8 ? launch<64, true>(p, st) : launch<64, false>(p, st);
}

}  // namespace

extern "C" size_t rx_attn_tree_workspace(int32_t batch, int32_t hq, int32_t hkv, int32_t head_dim, int32_t max_tree)
{
    if (!tree_shape_ok(batch, hq, hkv, head_dim, max_tree)) {
        rx_set_error(RX_ERR_INVALID, "rx_attn_tree_workspace: invalid argument");
        return 0;
    }
    return part_bytes(head_dim) + (size_t)2 * kCtas * kRows * sizeof(float);
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
