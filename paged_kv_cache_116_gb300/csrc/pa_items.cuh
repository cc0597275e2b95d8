// pa_items.cuh -- work items handed out to all warps of a CTA through a small
// ring in shared memory: one warp draws them, every warp takes each in turn.
#pragma once

#include <stdint.h>

#include "pa_device.cuh"

namespace pa {

// What a warp gets instead of an item (items are not negative): there are no
// more, or a wait ran out -- two different ends, since work is lost with the
// second and copies may be in flight.
constexpr int kItemsDone = -1, kItemsExpired = -2;

// N slots (a power of two).  full: one arrival each, by the drawing warp;
// empty: one by every warp of the CTA.
template <int N>
struct ItemRing {
    uint64_t* full;
    uint64_t* empty;
    volatile int* slot;
    int n = 0;  // items taken by this warp

    // The next item; draw() gives it (or kItemsDone) in the drawing warp.
    // The whole warp calls it and gets one answer.
    template <typename Draw>
    __device__ __forceinline__ int next(bool drawing, uint64_t limit_ns, Draw draw) {
        const int k = n & (N - 1);
        const uint32_t turn = (uint32_t)(n / N) & 1u;
        const bool first = (threadIdx.x & 31) == 0;
        if (drawing) {
            int ok = 0;
            if (first && (ok = mbar_wait_ns(&empty[k], turn ^ 1u, limit_ns))) {
                slot[k] = draw();
                mbar_arrive(&full[k]);
            }
            if (!__shfl_sync(0xffffffffu, ok, 0)) return kItemsExpired;
        }
        if (!mbar_wait_ns_warp(&full[k], turn, limit_ns)) return kItemsExpired;
        const int it = slot[k];
        __syncwarp();
        if (first) mbar_arrive(&empty[k]);
        ++n;
        return it;
    }
};

}  // namespace pa
