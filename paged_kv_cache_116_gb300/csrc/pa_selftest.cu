// pa_selftest.cu -- a fault-free exercise of the kernels' failure path: the
// warps of one CTA wait on shared-memory barriers that nothing completes, with
// the same bounded waits the kernels use -- one as the decode kernel does, one
// for a work item that nobody draws, one to hand out an item into a ring that
// nobody empties --, give up and record the expiry in a device status word
// that pa_device_status reads like the kernels' own.  The bit is set only if
// every one of them saw its expiry as one (an item that never comes is not the
// end of the items).
#include <cuda_runtime.h>
#include <stdint.h>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_items.cuh"

namespace pa {
namespace {

__device__ unsigned int g_selftest_status;

__global__ void selftest_wait_kernel(uint32_t polls) {
    constexpr int N = 4;
    constexpr uint64_t kLimitNs = 200000;
    __shared__ uint64_t bar, full[2][N], empty[2][N];
    __shared__ int slot[2][N];
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        for (int i = 0; i < 2 * N; ++i) {
            mbar_init(full[0] + i, 1);
            mbar_init(empty[0] + i, 2);  // (the drawing warp's arrival alone does not empty a slot)
        }
        mbar_fence_init();
    }
    __syncthreads();
    const int warp = threadIdx.x >> 5;
    bool expired = false;
    if (warp == 0) {
        if (threadIdx.x == 0) expired = !mbar_wait_bounded(&bar, 0u, polls);
        expired = __shfl_sync(0xffffffffu, (int)expired, 0) != 0;
    } else if (warp == 1) {
        ItemRing<N> ring{full[0], empty[0], slot[0]};
        expired = ring.next(false, kLimitNs, [] { return kItemsDone; }) == kItemsExpired;
    } else {
        ItemRing<N> ring{full[1], empty[1], slot[1]};
        int got = 0, it;
        while (got <= N && (it = ring.next(true, kLimitNs, [&] { return got; })) == got) ++got;
        expired = got == N && it == kItemsExpired;
    }
    if (__syncthreads_and(expired) && threadIdx.x == 0) atomicOr(&g_selftest_status, kStatusTimeout);
}

}  // namespace

cudaError_t launch_selftest_wait(uint32_t polls, cudaStream_t stream) {
    selftest_wait_kernel<<<1, 96, 0, stream>>>(polls);
    return cudaGetLastError();
}

uint32_t selftest_status(bool clear) {
    unsigned int v = 0;
    cudaMemcpyFromSymbol(&v, g_selftest_status, sizeof(v));
    if (clear) {
        const unsigned int z = 0;
        cudaMemcpyToSymbol(g_selftest_status, &z, sizeof(z));
    }
    return v;
}

}  // namespace pa
