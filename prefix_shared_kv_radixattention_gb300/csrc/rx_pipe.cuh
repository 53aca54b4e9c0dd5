// rx_pipe.cuh -- bounded waits and the swizzled tile layout shared by the
// tensor-core attention kernels (rx_extend.cu, rx_tree.cu).
#pragma once

#include "rx_common.cuh"

namespace rx {

// Bounded wait of one thread; false when it gave up (or another role did).
__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                              int32_t *status)
{
    if (mbar_test_wait(bar, parity)) return true;  // already flipped: no suspend
    const long long t0 = clock64();
    do {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
    } while (clock64() - t0 < kWaitCycles);
    *abort_flag = 1;
    if (status) atomicOr(status, RX_DEV_TIMEOUT);
    return false;
}
// The same for a whole warp, with one answer for all its lanes (the warp-wide
// tcgen05.ld / st that follow need every lane).
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                          int32_t *status)
{
    return __all_sync(0xffffffffu, wait_or_abort(bar, parity, abort_flag, status));
}

// Bounded wait that ignores the abort flag: used only to let copies already
// issued finish landing before the CTA exits.
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity, int32_t *status)
{
    const long long t0 = clock64();
    do {
        if (mbar_try_wait(bar, parity)) return;
    } while (clock64() - t0 < kWaitCycles);
    if (status) atomicOr(status, RX_DEV_TIMEOUT);
}

// byte offset of 16-byte chunk c of row r in a 128-byte-swizzled K-major
// tile whose 128-byte column blocks are blk bytes apart
__device__ __forceinline__ uint32_t sw128(int r, int c, int blk)
{
    return (uint32_t)((c >> 3) * blk + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

__device__ __forceinline__ float u2f(uint32_t u) { return __uint_as_float(u); }

}  // namespace rx
