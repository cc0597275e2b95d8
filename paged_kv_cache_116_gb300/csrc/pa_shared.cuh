// pa_shared.cuh -- how the work of shared prefixes is cut: the same on the
// kernel that does it (pa_prefix_umma.cu) and the one that joins its records
// (pa_decode_shared.cu).
//
// A unit is (group, KV head, tile of up to T members): 128 query rows that
// share the group's prefix, 128 keys at a time.  The units' key tiles, and
// kPrefixUnit more a unit for its queries, first maxima and output, form one
// flat list that is cut into equal runs, one per CTA.  A unit's first piece
// goes to its query rows' own records, every later one is the first piece of
// its CTA's run and goes to the CTA's records.
#pragma once

#include <stdint.h>

namespace pa {

constexpr int kPrefixKeys = 128;  // keys per tile
constexpr int kPrefixUnit = 2;

struct SharedGroups {
    const int32_t* starts;       // [groups + 1]
    const int32_t* prefix_lens;  // [groups]
    int32_t groups;
    int32_t num_kv_heads;
    int32_t tokens;      // members per tile: floor(128 / query heads per KV head)
    int32_t block_size;
    float* rows;  // [num_seqs * num_heads][head_dim + 4]: o, m, l
    float* cont;  // [CTAs][128][head_dim + 4]
};

// Tokens of group g's prefix that are worked once for all members: whole
// groups of 16 and whole blocks; none for a group of one.
__device__ __forceinline__ int shared_tokens(const SharedGroups& p, int g) {
    if (p.starts[g + 1] - p.starts[g] < 2) return 0;
    const int step = max(p.block_size, 16);
    return max(p.prefix_lens[g], 0) / step * step;
}
__device__ __forceinline__ int shared_row_tiles(const SharedGroups& p, int g) {
    return (p.starts[g + 1] - p.starts[g] + p.tokens - 1) / p.tokens;
}
__device__ __forceinline__ int shared_cost(const SharedGroups& p, int g) {
    const int nk = (shared_tokens(p, g) + kPrefixKeys - 1) / kPrefixKeys;
    return nk ? p.num_kv_heads * shared_row_tiles(p, g) * (nk + kPrefixUnit) : 0;
}
// CTAs that the list of cost W is cut for: runs of four at least, so that a
// row's pieces are few (and no run is empty).
__device__ __forceinline__ int shared_ctas(int64_t W, int ctas) { return (int)max(min((int64_t)ctas, W / 4), (int64_t)1); }
// Exclusive prefix of the groups' costs, in shared memory (every thread of the
// block; ends with a block barrier).
__device__ __forceinline__ void shared_prefix(const SharedGroups& p, int32_t* prefix) {
    for (int g = threadIdx.x; g < p.groups; g += blockDim.x) prefix[g + 1] = shared_cost(p, g);
    if (threadIdx.x == 0) prefix[0] = 0;
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x, per = (p.groups + 31) / 32;
        const int lo = 1 + lane * per, hi = min(p.groups + 1, lo + per);
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

}  // namespace pa
