// pa_weights.cuh -- what the kernels of the attention-weight passes share:
// a request's rows and keys, and the list of tiles over a batch.
#pragma once

#include <stdint.h>

#include "pa_internal.h"

namespace pa {

struct WeightSeq {
    int s;       // request
    int L;       // keys
    int n;       // new tokens
    int rows;    // of them counted: the last min(n, window)
    int row0;    // row of q of the first counted one
    int stat0;   // row of its statistics
};

__device__ __forceinline__ WeightSeq weight_seq(const WeightArgs& a, int s) {
    WeightSeq q;
    q.s = s;
    q.L = a.seq_lens[s];
    q.n = 1;
    int end = s + 1;
    if (a.cu != nullptr) {
        end = a.cu[s + 1];
        q.n = end - a.cu[s];
    }
    if (q.L <= 0) q.L = q.n = 0;
    q.rows = a.window > 0 ? min(q.n, a.window) : q.n;
    q.row0 = end - q.rows;
    q.stat0 = a.stat_pitch ? s * a.stat_pitch : q.row0;
    return q;
}

// Exclusive prefix over the batch of count(request), into shared memory
// (prefix[S + 1]).  Every thread of the block calls it; it ends with a block
// barrier.
template <typename Count>
__device__ __forceinline__ void work_prefix(const WeightArgs& a, int32_t* prefix, Count count) {
    const int S = a.num_seqs, lane = threadIdx.x & 31;
    for (int s = threadIdx.x; s < S; s += blockDim.x) prefix[s + 1] = count(weight_seq(a, s));
    if (threadIdx.x == 0) prefix[0] = 0;
    __syncthreads();
    if (threadIdx.x < 32) {
        const int per = (S + 31) / 32;
        const int lo = 1 + lane * per, hi = min(S + 1, lo + per);
        int sum = 0;
        for (int i = lo; i < hi; ++i) sum += prefix[i];
        int incl = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += v;
        }
        int run = incl - sum;
        for (int i = lo; i < hi; ++i) {
            run += prefix[i];
            prefix[i] = run;
        }
    }
    __syncthreads();
}

// Work item -> (request, KV head, tile): a request's items are its tiles, all
// heads of a tile before the next (the callers put the long tiles first).
__device__ __forceinline__ void locate_work(const int32_t* prefix, int S, int Hkv, int64_t item, int& s, int& h,
                                            int& tile) {
    int lo = 0, hi = S - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((int64_t)prefix[mid] * Hkv <= item) lo = mid;
        else hi = mid - 1;
    }
    const int64_t rem = item - (int64_t)prefix[lo] * Hkv;
    s = lo;
    tile = (int)(rem / Hkv);
    h = (int)(rem - (int64_t)tile * Hkv);
}

}  // namespace pa
