// A producer's record of its loads into shared memory: a CTA must not end while one is in flight,
// also where a bounded wait ran out.
#pragma once
#include "ll_device.cuh"

namespace ll {

// Which stages a producer has loaded, and the phase of their barriers that each load completes.
struct Issued {
    uint32_t stages = 0, phases = 0;
    __device__ __forceinline__ void add(int stage, uint32_t phase) {
        stages |= 1u << stage;
        phases = (phases & ~(1u << stage)) | (phase << stage);
    }
};
// Waits, up to one limit in all, for those stages' barriers; returns the stages still on their way.
// By a whole warp, which stays together.
__device__ __forceinline__ uint32_t wait_for_loads(uint64_t* bars, const Issued& issued,
                                                   uint64_t limit_ns) {
    uint32_t left = issued.stages;
    const uint64_t t0 = globaltimer_ns();
    while (left) {
        for (uint32_t todo = left; todo; todo &= todo - 1) {
            const int s = __ffs(todo) - 1;
            if (__all_sync(0xffffffffu, mbar_try_wait_cl(&bars[s], (issued.phases >> s) & 1u)))
                left &= ~(1u << s);
        }
        if (__any_sync(0xffffffffu, globaltimer_ns() - t0 > limit_ns)) break;
    }
    return left;
}
// The same for a CTA pair's leader, whose barriers count both CTAs' loads (`bytes` of either a
// stage).  gave_up: it may have stopped ahead of loads that the other CTA still issued.
__device__ __forceinline__ void wait_for_pair_loads(uint64_t* bars, const Issued& issued, int stages,
                                                    uint32_t bytes, bool gave_up, uint64_t limit_ns) {
    const uint32_t late = wait_for_loads(bars, issued, limit_ns);
    if (!gave_up) return;
    Issued other;
    for (int s = 0; s < stages; ++s)
        if (!((late >> s) & 1u)) {
            if ((threadIdx.x & 31) == 0) mbar_arrive_expect_tx(&bars[s], bytes);
            other.add(s, (issued.stages >> s) & 1u ? ((issued.phases >> s) & 1u) ^ 1u : 0u);
        }
    __syncwarp();
    wait_for_loads(bars, other, limit_ns);
}

}  // namespace ll
