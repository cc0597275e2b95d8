// pa_evict.cu -- eviction from the paged cache by accumulated attention
// weight.
//
// For each (sequence, KV head) with L cached tokens and a budget of `keep`:
// if L > keep, the tokens whose position is below num_sink or among the
// num_recent newest are held, and the others are taken by weight, largest
// first (a NaN counts above every number, equal weights go to the lower
// index), until `keep` are.  The kept rows are then brought to the front of
// the sequence with as few moves as there can be: a kept token with index
// below `keep` stays where it is, and the i-th hole below `keep` gets the
// i-th kept token from `keep` on.  Sources (index >= keep) and destinations
// (index < keep) are disjoint, so the moves need no order and no staging; the
// price is that a head's rows are in no particular order afterwards, which
// attention does not see (keys carry their rotation with them), and that the
// token positions move along with the rows.
//
// Destination rows are addressed through a second block table: the
// sequence's own blocks (in place: only the holes are written), or others
// where its blocks are shared with someone else (every kept row is copied
// there, into the same places).
//
// Two kernels.  evict_select_kernel, one CTA per (sequence, KV head), finds
// the keep-th largest key by a radix selection of four 8-bit digits over
// order-preserving integers of the weights, then writes the source index of
// every destination index.  evict_move_kernel copies the rows, one warp per
// destination row at a time.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_launch.cuh"

namespace pa {
namespace {

constexpr int kSelThreads = 1024;

// Position of cached token j: recorded by an earlier eviction, or (appended
// since) counted back from the newest.
__device__ __forceinline__ int token_position(const EvictArgs& a, const int32_t* pos, int j, int L, int c, int seen) {
    return j < c ? pos[j] : seen - L + j;
}

// Larger weight -> larger key; -0 and +0 alike, NaN above +infinity.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (isnan(w)) return 0xfffffffeu;
    const uint32_t b = __float_as_uint(w + 0.f);
    return (b >> 31) ? ~b : b | 0x80000000u;
}

struct EvictUnit {
    int s, h, L, c, seen;
    int64_t row;  // of weights and positions
};
__device__ __forceinline__ EvictUnit evict_unit(const EvictArgs& a, int u) {
    EvictUnit e;
    e.s = u / a.num_kv_heads;
    e.h = u - e.s * a.num_kv_heads;
    e.L = max(0, a.context_lens[e.s]);
    e.c = a.recorded_lens ? min(max(0, a.recorded_lens[e.s]), e.L) : 0;
    e.seen = a.seen_lens ? a.seen_lens[e.s] : e.L;
    e.row = ((int64_t)e.s * a.num_kv_heads + e.h) * a.stride;
    return e;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a) {
    __shared__ uint32_t hist[256];
    __shared__ uint32_t sh_prefix;
    __shared__ int sh_need, sh_cnt[32], sh_cnt2[32];
    pdl_wait_primary();
    pdl_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const EvictUnit e = evict_unit(a, blockIdx.x);
    const int L = e.L, keep = a.keep;
    if (tid == 0 && e.h == 0) a.new_lens[e.s] = min(L, keep);
    if (L <= keep) return;  // everything stays; the move kernel copies by index
    const float* w = a.weights + e.row;
    const int32_t* pos = a.positions + e.row;  // read below recorded_lens only
    int32_t* map = a.map + (int64_t)blockIdx.x * a.map_stride;
    auto key = [&](int j) -> uint32_t {
        const int p = token_position(a, pos, j, L, e.c, e.seen);
        if (p < a.num_sink || p >= e.seen - a.num_recent) return 0xffffffffu;
        return weight_key(w[j]);
    };
    // the keep-th largest key: digit by digit from the top
    uint32_t prefix = 0, mask = 0;
    int need = keep;
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        for (int j = tid; j < L; j += kSelThreads) {
            const uint32_t k = key(j);
            if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1u);
        }
        __syncthreads();
        if (tid == 0) {
            int left = need;
            int d = 255;
            while (d > 0 && (int)hist[d] < left) left -= (int)hist[d--];
            sh_prefix = prefix | ((uint32_t)d << shift);
            sh_need = left;
        }
        __syncthreads();
        prefix = sh_prefix;
        need = sh_need;
        mask |= 255u << shift;
        __syncthreads();
    }
    // kept: key above the threshold, or equal to it and among its first `need`.
    // Warps own contiguous index ranges; ranks come from counts per warp.
    const int per = ((L + 31) / 32 + 31) / 32 * 32;
    const int lo = min(L, warp * per), hi = min(L, lo + per);
    int eq = 0;
    for (int j0 = lo; j0 < hi; j0 += 32) {
        const bool is = j0 + lane < hi && key(j0 + lane) == prefix;
        eq += __popc(__ballot_sync(0xffffffffu, is));
    }
    if (lane == 0) sh_cnt[warp] = eq;
    __syncthreads();
    int eq0 = 0;
    for (int i = 0; i < warp; ++i) eq0 += sh_cnt[i];
    __syncthreads();
    // walk: is token j0 + lane kept, given the warp's equal keys before j0
    auto kept_mask = [&](int j0, int& eqs) -> uint32_t {
        const uint32_t k = j0 + lane < hi ? key(j0 + lane) : 0u;
        const uint32_t em = __ballot_sync(0xffffffffu, j0 + lane < hi && k == prefix);
        const int rank = eqs + __popc(em & ((1u << lane) - 1u));
        const bool kept = j0 + lane < hi && (k > prefix || (k == prefix && rank < need));
        eqs += __popc(em);
        return __ballot_sync(0xffffffffu, kept);
    };
    int holes = 0, movers = 0, eqs = eq0;
    for (int j0 = lo; j0 < hi; j0 += 32) {
        const uint32_t km = kept_mask(j0, eqs);
        const uint32_t below = j0 + 32 <= keep ? 0xffffffffu : (j0 >= keep ? 0u : (1u << (keep - j0)) - 1u);
        const uint32_t live = j0 + 32 <= hi ? 0xffffffffu : (1u << (hi - j0)) - 1u;
        holes += __popc(~km & below & live);
        movers += __popc(km & ~below);
    }
    if (lane == 0) {
        sh_cnt[warp] = holes;
        sh_cnt2[warp] = movers;
    }
    __syncthreads();
    int hole0 = 0, mover0 = 0;
    for (int i = 0; i < warp; ++i) {
        hole0 += sh_cnt[i];
        mover0 += sh_cnt2[i];
    }
    // destinations of holes and sources of movers, by rank, then joined
    int32_t* hole_at = map + keep;
    int32_t* mover_at = map + 2 * keep;
    eqs = eq0;
    for (int j0 = lo; j0 < hi; j0 += 32) {
        const uint32_t km = kept_mask(j0, eqs);
        const uint32_t below = j0 + 32 <= keep ? 0xffffffffu : (j0 >= keep ? 0u : (1u << (keep - j0)) - 1u);
        const uint32_t live = j0 + 32 <= hi ? 0xffffffffu : (1u << (hi - j0)) - 1u;
        const uint32_t hm = ~km & below & live, mm = km & ~below, lt = (1u << lane) - 1u;
        const int j = j0 + lane;
        if ((hm >> lane) & 1u) hole_at[hole0 + __popc(hm & lt)] = j;
        else if (j < min(hi, keep)) map[j] = j;
        if ((mm >> lane) & 1u) mover_at[mover0 + __popc(mm & lt)] = j;
        hole0 += __popc(hm);
        mover0 += __popc(mm);
    }
    __syncthreads();
    int total = 0;
    for (int i = 0; i < 32; ++i) total += sh_cnt[i];
    for (int i = tid; i < total; i += kSelThreads) map[hole_at[i]] = mover_at[i];
}

// VB: bytes per vector of a row.
template <int VB> struct VecOf;
template <> struct VecOf<16> { using V = uint4; };
template <> struct VecOf<8> { using V = uint2; };
template <> struct VecOf<4> { using V = uint32_t; };
template <> struct VecOf<2> { using V = uint16_t; };
template <> struct VecOf<1> { using V = uint8_t; };

constexpr int kMoveWarps = 8, kMoveRows = 64;  // destination rows per CTA

template <int VB>
__global__ void __launch_bounds__(kMoveWarps * 32) evict_move_kernel(const EvictArgs a, int chunks) {
    using V = typename VecOf<VB>::V;
    pdl_wait_primary();
    pdl_launch_dependents();
    const int u = blockIdx.x / chunks, i0 = (blockIdx.x - u * chunks) * kMoveRows;
    const EvictUnit e = evict_unit(a, u);
    const int count = min(e.L, a.keep);
    if (i0 >= count) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, bs = a.block_size, Hkv = a.num_kv_heads;
    const int32_t* map = e.L > a.keep ? a.map + (int64_t)u * a.map_stride : nullptr;
    const int32_t* from_tb = a.block_tables + (int64_t)e.s * a.max_blocks;
    const int32_t* to_tb = a.new_block_tables + (int64_t)e.s * a.new_max_blocks;
    const int64_t rv = a.row_bytes / VB;
    for (int i = i0 + warp; i < min(count, i0 + kMoveRows); i += kMoveWarps) {
        const int src = map ? map[i] : i;
        if (lane == 0) {
            const float w = a.weights[e.row + src];
            const int p = token_position(a, a.positions + e.row, src, e.L, e.c, e.seen);
            a.weights_out[e.row + i] = w;
            if (a.positions_out) a.positions_out[e.row + i] = p;
        }
        const int64_t fb = from_tb[src / bs], tb = to_tb[i / bs];
        if (src == i && fb == tb) continue;
        const int64_t fo = ((fb * bs + src % bs) * Hkv + e.h) * rv, to = ((tb * bs + i % bs) * Hkv + e.h) * rv;
        for (int x = lane; x < rv; x += 32) {
            const V kv = static_cast<const V*>(a.k_cache)[fo + x], vv = static_cast<const V*>(a.v_cache)[fo + x];
            static_cast<V*>(a.k_cache)[to + x] = kv;
            static_cast<V*>(a.v_cache)[to + x] = vv;
        }
        if (a.k_scales && lane < 2) {
            float* sc = lane ? a.v_scales : a.k_scales;
            sc[(tb * Hkv + e.h) * bs + i % bs] = sc[(fb * Hkv + e.h) * bs + src % bs];
        }
    }
}

}  // namespace

size_t evict_workspace(int32_t num_seqs, int32_t num_kv_heads, int32_t max_context, int32_t keep) {
    if (max_context <= keep) return 0;
    return (size_t)num_seqs * num_kv_heads * 3 * keep * sizeof(int32_t);
}

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream) {
    const int64_t units = (int64_t)a.num_seqs * a.num_kv_heads;
    EvictArgs p = a;
    p.map_stride = 3 * (int64_t)a.keep;
    cudaError_t e = launch_pdl(evict_select_kernel, dim3((unsigned)units), dim3(kSelThreads), stream, p);
    if (e != cudaSuccess) return e;
    const int rows = std::min(a.keep, a.max_context);
    const int chunks = std::max(1, (rows + kMoveRows - 1) / kMoveRows);
    const dim3 grid((unsigned)(units * chunks)), block(kMoveWarps * 32);
    const int64_t rb = a.row_bytes;
    if (rb % 16 == 0) return launch_pdl(evict_move_kernel<16>, grid, block, stream, p, chunks);
    if (rb % 8 == 0) return launch_pdl(evict_move_kernel<8>, grid, block, stream, p, chunks);
    if (rb % 4 == 0) return launch_pdl(evict_move_kernel<4>, grid, block, stream, p, chunks);
    if (rb % 2 == 0) return launch_pdl(evict_move_kernel<2>, grid, block, stream, p, chunks);
    return launch_pdl(evict_move_kernel<1>, grid, block, stream, p, chunks);
}

}  // namespace pa
