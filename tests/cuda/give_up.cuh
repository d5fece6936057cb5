// give_up.cuh -- the attention kernels' waits with a short limit, one of which gives up on
// demand: included ahead of a kernel's source file.
//
// The n-th wait of one warp of one CTA gives up in the lanes of a mask, without waiting; every
// other wait is the kernels' own, bounded by 50 ms. What the CTA does next is the kernels' code.
#pragma once

#define warp_wait plain_warp_wait
#include "gdn_paged.cuh"
#undef warp_wait

namespace gdn {

struct GiveUp {
    int cta, warp, nth;  // cta -1: nowhere
    unsigned lanes;
};

__device__ GiveUp g_give_up = {-1, 0, 0, 0u};
__device__ volatile int g_waits;  // of that warp so far, in this launch and those before

// By a whole warp: whether this lane's wait gives up.
__device__ __forceinline__ bool gives_up() {
    const GiveUp g = g_give_up;
    if (static_cast<int>(blockIdx.x) != g.cta || static_cast<int>(threadIdx.x >> 5) != g.warp) return false;
    const int n = g_waits;
    __syncwarp();
    if ((threadIdx.x & 31) == 0) g_waits = n + 1;
    __syncwarp();
    return n == g.nth && ((g.lanes >> (threadIdx.x & 31)) & 1u);
}

__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *dead,
                                          unsigned *watchdog) {
    const bool now = gives_up();
    if (__all_sync(FULL_MASK, !now && mbar_test(bar, parity))) return true;
    const uint64_t t0 = global_timer_ns();
    while (!__all_sync(FULL_MASK, !now && mbar_try_wait(bar, parity))) {
        const bool late = now || global_timer_ns() - t0 > 50000000ull;
        if (__any_sync(FULL_MASK, late || *dead)) {
            if (late) atomicOr(watchdog, WD_STAGE_COPY);
            *dead = 1;
            return false;
        }
    }
    return true;
}

}  // namespace gdn

extern "C" int give_up_arm(int cta, int warp, int nth, unsigned lanes) {
    const gdn::GiveUp g{cta, warp, nth, lanes};
    const int zero = 0;
    return cudaMemcpyToSymbol(gdn::g_give_up, &g, sizeof(g)) != cudaSuccess ||
           cudaMemcpyToSymbol(gdn::g_waits, &zero, sizeof(zero)) != cudaSuccess;
}

// Waits of the armed warp since it was armed.
extern "C" int give_up_waits() {
    int n = -1;
    cudaMemcpyFromSymbol(&n, gdn::g_waits, sizeof(n));
    return n;
}
