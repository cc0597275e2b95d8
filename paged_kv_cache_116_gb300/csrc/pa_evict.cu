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
// Two kernels.
//   evict_select_kernel, one CTA per (sequence, KV head): the tokens' keys
//   (order-preserving integers of the weights, the held ones above all) are
//   read once into shared memory; the keep-th largest is found by a radix
//   selection of 11, 11 and 10 bits, which ends as soon as a digit's bucket is
//   taken whole; the kept tokens are marked in a bit mask, holes and movers are
//   ranked by a prefix over its words, and the threads then write each
//   destination index's weight and position and list the rows to copy.
//   evict_move_kernel copies the listed rows, all of the GPU's warps over all
//   units' lists.
// Bound: the select kernel by the latency of its few passes over shared
// memory (512 heads of 1,040 tokens: 11 us, of which 2 us each for loading,
// the two digits, ranking and writing; 64 heads of 32,768: 21 us, a third of
// it the first pass), the move kernel by HBM (each listed row is read and
// written once: 262,144 rows of 2 x 256 bytes in 43 us, 6.2 TB/s).
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_launch.cuh"

namespace pa {
namespace {

constexpr int kStageMax = 48 * 1024;  // keys held in shared memory; longer contexts re-read the weights
constexpr int kBins = 2048;

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
    e.L = min(max(0, a.context_lens[e.s]), a.max_context);  // (shared memory holds no more)
    e.c = a.recorded_lens ? min(max(0, a.recorded_lens[e.s]), e.L) : 0;
    e.seen = a.seen_lens ? a.seen_lens[e.s] : e.L;
    e.row = ((int64_t)e.s * a.num_kv_heads + e.h) * a.stride;
    return e;
}

// Dynamic shared memory: kept-token mask and holes before each of its words,
// then (staged) the keys, whose place the movers take.
size_t select_smem(int32_t max_context) {
    const size_t words = ((size_t)max_context + 31) / 32;
    return words * 8 + (max_context <= kStageMax ? (size_t)max_context * 4 : 0);
}

// Longest context of the select kernel's forms, by threads.
constexpr int select_max(int threads, bool staged) {
    return !staged ? kEvictMaxContext : threads == 256 ? 2048 : threads == 512 ? 8192 : kStageMax;
}

// NT threads; STAGED: the context fits in shared memory.
template <int NT, bool STAGED>
__global__ void __launch_bounds__(NT) evict_select_kernel(const EvictArgs a) {
    constexpr int NW = NT / 32, PER = kBins / NT;  // warps; buckets per thread
    extern __shared__ uint32_t dyn[];
    __shared__ alignas(16) uint32_t hist[kBins];
    __shared__ int sh_warp[NW];
    __shared__ uint64_t sh_both[NW];
    __shared__ int sh_digit, sh_left, sh_count, sh_rows;
    const int words_max = (a.max_context + 31) / 32;
    uint32_t* mask = dyn;
    int* holes_before = reinterpret_cast<int*>(dyn + words_max);
    uint32_t* keys = dyn + 2 * words_max;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_wait_primary();
    pdl_launch_dependents();
    const EvictUnit e = evict_unit(a, blockIdx.x);
    const int L = e.L, keep = a.keep, count = min(L, keep);
    if (tid == 0) {
        if (e.h == 0) a.new_lens[e.s] = count;
        sh_rows = 0;
    }
    const float* w = a.weights + e.row;
    const int32_t* pos = a.positions + e.row;  // read below recorded_lens only
    float* wo = a.weights_out + e.row;
    int32_t* po = a.positions_out ? a.positions_out + e.row : nullptr;
    if (L <= keep) {  // everything stays where it is; the move kernel copies by index
        if (tid == 0 && a.counts) a.counts[blockIdx.x] = -1;
        for (int i = tid; i < L; i += NT) {
            if (wo != w) wo[i] = w[i];
            if (po) po[i] = token_position(a, pos, i, L, e.c, e.seen);
        }
        return;
    }
    int* movers = STAGED ? reinterpret_cast<int*>(keys) : a.movers + (int64_t)blockIdx.x * a.list_stride;
    auto to_key = [&](int p, float x) -> uint32_t {
        return p < a.num_sink || p >= e.seen - a.num_recent ? 0xffffffffu : weight_key(x);
    };
    auto key_at = [&](int j) -> uint32_t {
        return STAGED ? keys[j] : to_key(token_position(a, pos, j, L, e.c, e.seen), w[j]);
    };
    for (int b = tid; b < kBins; b += NT) hist[b] = 0;
    __syncthreads();

    // the keep-th largest key, digit by digit from the top: `prefix` under
    // `bits`, of whose tokens `need` are taken
    uint32_t prefix = 0, bits = 0;
    int need = keep;
    bool tied = false;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, width = pass == 2 ? 1024 : 2048;
        if (pass == 0) {
            constexpr int U = 8;  // tokens in flight per thread
            for (int j0 = tid; j0 < L; j0 += NT * U) {
                float x[U];
                int p[U];
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    const int j = j0 + i * NT;
                    x[i] = j < L ? w[j] : 0.f;
                    p[i] = j < L ? token_position(a, pos, j, L, e.c, e.seen) : 0;
                }
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    const int j = j0 + i * NT;
                    if (j >= L) break;
                    const uint32_t k = to_key(p[i], x[i]);
                    if (STAGED) keys[j] = k;
                    atomicAdd(&hist[k >> shift], 1u);
                }
            }
        } else {
#pragma unroll 4
            for (int j = tid; j < L; j += NT) {
                const uint32_t k = key_at(j);
                if ((k & bits) == prefix) atomicAdd(&hist[(k >> shift) & (width - 1)], 1u);
            }
        }
        __syncthreads();
        // buckets from the top: thread t holds PER of them
        // (as vectors, whose lanes fall into different banks)
        using BV = typename std::conditional<PER == 2, uint2, uint4>::type;
        constexpr int VE = sizeof(BV) / 4, NV = PER / VE;
        int mine[PER], sum = 0;
        BV* own = reinterpret_cast<BV*>(hist + kBins - (tid + 1) * PER);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const BV b = own[v];
            memcpy(mine + v * VE, &b, sizeof(b));
            own[v] = BV{};
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) sum += mine[i];
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) sh_warp[warp] = incl;
        __syncthreads();
        int before = incl - sum + __reduce_add_sync(0xffffffffu, lane < warp ? sh_warp[lane] : 0);
        if (before < need && need <= before + sum) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int n = mine[PER - 1 - i];
                if (before < need && need <= before + n) {
                    sh_digit = kBins - 1 - (tid * PER + i);
                    sh_left = need - before;
                    sh_count = n;
                }
                before += n;
            }
        }
        __syncthreads();
        prefix |= (uint32_t)sh_digit << shift;
        bits |= (uint32_t)(width - 1) << shift;
        need = sh_left;
        tied = sh_count != need;
        if (!tied) break;  // the whole bucket is taken: lower digits decide nothing
        __syncthreads();
    }

    // Kept: above the threshold, or equal to it and among its first `need`.
    // One bit per token, a warp per mask word.
    const int words = (L + 31) / 32;
    if (!tied) {
#pragma unroll 4
        for (int x = warp; x < words; x += NW) {
            const int j = 32 * x + lane;
            const uint32_t kept = __ballot_sync(0xffffffffu, j < L && (key_at(j) & bits) >= prefix);
            if (lane == 0) mask[x] = kept;
        }
        __syncthreads();
    } else {  // ranks among equal keys: warps own contiguous runs of words
        const int per = (words + NW - 1) / NW, w0 = min(words, warp * per), w1 = min(words, w0 + per);
        int equal = 0;
        for (int x = w0; x < w1; ++x) {
            const int j = 32 * x + lane;
            equal += __popc(__ballot_sync(0xffffffffu, j < L && key_at(j) == prefix));
        }
        if (lane == 0) sh_warp[warp] = equal;
        __syncthreads();
        equal = 0;
        for (int i = 0; i < warp; ++i) equal += sh_warp[i];
        for (int x = w0; x < w1; ++x) {
            const int j = 32 * x + lane;
            const uint32_t k = j < L ? key_at(j) : 0u;
            const uint32_t same = __ballot_sync(0xffffffffu, j < L && k == prefix);
            const int rank = equal + __popc(same & ((1u << lane) - 1u));
            const uint32_t kept = __ballot_sync(0xffffffffu, j < L && (k > prefix || (k == prefix && rank < need)));
            equal += __popc(same);
            if (lane == 0) mask[x] = kept;
        }
        __syncthreads();
    }
    // Holes below `keep` and movers from there on, ranked: a thread per run of
    // words, a block-wide prefix of both counts (fields of 32 bits).
    auto below = [&](int x) -> uint32_t {  // tokens of word x with index below keep (each is a token: keep < L)
        const int n = keep - 32 * x;
        return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
    };
    const int run = (words + NT - 1) / NT, x0 = min(words, tid * run), x1 = min(words, x0 + run);
    uint64_t both = 0;
    for (int x = x0; x < x1; ++x)
        both += (uint64_t)__popc(~mask[x] & below(x)) | (uint64_t)__popc(mask[x] & ~below(x)) << 32;
    uint64_t incl = both;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) sh_both[warp] = incl;
    __syncthreads();
    both = incl - both;
#pragma unroll
    for (int i = 0; i < NW; ++i) both += i < warp ? sh_both[i] : 0;
    int holes = (int)(uint32_t)both, moved = (int)(both >> 32);
    for (int x = x0; x < x1; ++x) {
        holes_before[x] = holes;
        holes += __popc(~mask[x] & below(x));
        for (uint32_t late = mask[x] & ~below(x); late; late &= late - 1) movers[moved++] = 32 * x + __ffs(late) - 1;
    }
    __syncthreads();
    const int32_t* from_tb = a.block_tables + (int64_t)e.s * a.max_blocks;
    const int32_t* to_tb = a.new_block_tables + (int64_t)e.s * a.new_max_blocks;
    const int bs = a.block_size, sh = (bs & (bs - 1)) == 0 ? 31 - __clz(bs) : -1;
    auto block_of = [&](int x) { return sh >= 0 ? x >> sh : x / bs; };
    int2* list = a.list + (int64_t)blockIdx.x * a.list_stride;
    constexpr int U = 4;  // destinations in flight per thread
    for (int i0 = 32 * warp; i0 < keep; i0 += NT * U) {
        int src[U], p[U], fb[U], tb[U];
        int2 off[U];
        float x[U];
#pragma unroll
        for (int q = 0; q < U; ++q) {
            const int i = i0 + q * NT + lane;
            src[q] = -1;
            fb[q] = tb[q] = 0;
            if (i >= keep) continue;
            const uint32_t kept = mask[i >> 5];
            src[q] = (kept >> lane) & 1u ? i : movers[holes_before[i >> 5] + __popc(~kept & ((1u << lane) - 1u))];
            x[q] = w[src[q]];
            p[q] = token_position(a, pos, src[q], L, e.c, e.seen);
            const int bf = block_of(src[q]), bt = block_of(i);
            fb[q] = from_tb[bf];
            tb[q] = to_tb[bt];
            off[q] = make_int2(src[q] - bf * bs, i - bt * bs);
        }
#pragma unroll
        for (int q = 0; q < U; ++q) {
            const int i = i0 + q * NT + lane;
            if (i0 + q * NT >= keep) break;  // (uniform for the warp)
            if (src[q] >= 0) {
                wo[i] = x[q];
                if (po) po[i] = p[q];
            }
            const bool copy = src[q] >= 0 && (src[q] != i || fb[q] != tb[q]);
            const uint32_t c = __ballot_sync(0xffffffffu, copy);
            int at = 0;
            if (lane == 0 && c) at = atomicAdd(&sh_rows, __popc(c));
            at = __shfl_sync(0xffffffffu, at, 0) + __popc(c & ((1u << lane) - 1u));
            if (copy)  // source and destination slots (in any order: the rows are disjoint)
                list[at] = make_int2(fb[q] * bs + off[q].x, tb[q] * bs + off[q].y);
        }
    }
    __syncthreads();
    if (tid == 0) a.counts[blockIdx.x] = sh_rows;
}

// VB: bytes per vector of a row.
template <int VB> struct VecOf;
template <> struct VecOf<16> { using V = uint4; };
template <> struct VecOf<8> { using V = uint2; };
template <> struct VecOf<4> { using V = uint32_t; };
template <> struct VecOf<2> { using V = uint16_t; };
template <> struct VecOf<1> { using V = uint8_t; };

constexpr int kWarpRows = 8, kMoveWarps = 4;
constexpr int kMoveCtas = kSms * 16;  // wanted over all units

// Each unit has `ctas` CTAs, whose warps take eight rows of its list in turn
// (few enough that a short list spreads, and nobody visits what no list
// holds); a warp's lanes copy the rows' K and V vectors, U of them in flight
// each, six CTAs per SM (five: 2 us more on moves of 35-50 us; eight spill).
template <int VB>
__global__ void __launch_bounds__(kMoveWarps * 32, 6) evict_move_kernel(const EvictArgs a, int ctas) {
    using V = typename VecOf<VB>::V;
    constexpr int U = 8;
    pdl_wait_primary();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, bs = a.block_size, Hkv = a.num_kv_heads;
    const uint32_t rv = (uint32_t)(a.row_bytes / VB), per = 2 * rv;
    const int u = blockIdx.x / ctas, s = u / Hkv, h = u - s * Hkv;
    int first = ((blockIdx.x - u * ctas) * kMoveWarps + warp) * kWarpRows;
    // the unit's rows: those listed, or (-1) all of them by index; the first
    // list entries are read together with the count, not after it
    auto listed_row = [&](int r) {
        return a.counts && lane < kWarpRows && r < a.keep ? __ldcg(a.list + (int64_t)u * a.list_stride + r)
                                                          : make_int2(0, 0);
    };
    int2 entry = listed_row(first + lane);
    const int listed = a.counts ? __ldcg(a.counts + u) : -1;
    const int rows = listed >= 0 ? listed : min(max(0, a.context_lens[s]), min(a.keep, a.max_context));
    int2 ahead = entry;
    const int stride = ctas * kMoveWarps * kWarpRows;
    for (; first < rows; first += stride) {
        const int r = first + lane;
        entry = ahead;
        ahead = listed_row(r + stride);
        int from = 0, to = 0;  // this lane's row: its slots (equal ones: nothing to copy)
        if (lane < kWarpRows && r < rows) {
            if (listed < 0)
                entry = make_int2(a.block_tables[(int64_t)s * a.max_blocks + r / bs] * bs + r % bs,
                                  a.new_block_tables[(int64_t)s * a.new_max_blocks + r / bs] * bs + r % bs);
            from = entry.x;
            to = entry.y;
        }
        if (!__any_sync(0xffffffffu, from != to)) continue;
        const bool scaled = a.k_scales && from != to;
        float ks = 0.f, vs = 0.f;  // stored after the rows' loads are out
        if (scaled) {
            const int64_t f = ((int64_t)(from / bs) * Hkv + h) * bs + from % bs;
            ks = a.k_scales[f];
            vs = a.v_scales[f];
        }
        const uint32_t n = min(kWarpRows, rows - first) * per;
        const V* k = static_cast<const V*>(a.k_cache);
        const V* v = static_cast<const V*>(a.v_cache);
        for (uint32_t e0 = 0; e0 < n; e0 += 32 * U) {
            V x[U];
            int64_t dst[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const uint32_t it = e0 + 32 * i + lane, row = min(it / per, 31u), c = it - row * per;
                const int f = __shfl_sync(0xffffffffu, from, row), d = __shfl_sync(0xffffffffu, to, row);
                const uint32_t col = c < rv ? c : c - rv;
                dst[i] = it < n && f != d ? (((int64_t)d * Hkv + h) * rv + col) * 2 + (c < rv ? 0 : 1) : -1;
                if (dst[i] >= 0) x[i] = (c < rv ? k : v)[((int64_t)f * Hkv + h) * rv + col];
            }
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (dst[i] >= 0) static_cast<V*>(dst[i] & 1 ? a.v_cache : a.k_cache)[dst[i] >> 1] = x[i];
        }
        if (scaled) {
            const int64_t d = ((int64_t)(to / bs) * Hkv + h) * bs + to % bs;
            a.k_scales[d] = ks;
            a.v_scales[d] = vs;
        }
    }
}

// Workspace: rows listed per unit, the lists, and (contexts beyond shared
// memory) the movers.  Nothing where no sequence can exceed the budget.
struct EvictSpace {
    size_t counts = 0, list = 0, movers = 0;
};
EvictSpace evict_space(int64_t units, int32_t max_context, int32_t keep) {
    EvictSpace w;
    if (max_context <= keep) return w;
    auto round = [](size_t b) { return (b + 255) / 256 * 256; };
    w.counts = round((size_t)units * sizeof(int32_t));
    w.list = round((size_t)units * keep * sizeof(int2));
    if (max_context > kStageMax) w.movers = (size_t)units * keep * sizeof(int32_t);
    return w;
}

template <int NT, bool STAGED>
cudaError_t launch_select(const EvictArgs& a, int64_t units, cudaStream_t stream) {
    const size_t most = select_smem(select_max(NT, STAGED));
    if (most > 32 * 1024) {  // (with the static arrays beyond what every kernel may have)
        cudaError_t e = allow_smem(reinterpret_cast<const void*>(&evict_select_kernel<NT, STAGED>), most);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl_smem(evict_select_kernel<NT, STAGED>, dim3((unsigned)units), dim3(NT), select_smem(a.max_context),
                           stream, a);
}

}  // namespace

size_t evict_workspace(int32_t num_seqs, int32_t num_kv_heads, int32_t max_context, int32_t keep) {
    const EvictSpace w = evict_space((int64_t)num_seqs * num_kv_heads, max_context, keep);
    return w.counts + w.list + w.movers;
}

cudaError_t launch_evict(const EvictArgs& a, void* workspace, cudaStream_t stream) {
    const int64_t units = (int64_t)a.num_seqs * a.num_kv_heads;
    const EvictSpace w = evict_space(units, a.max_context, a.keep);
    EvictArgs p = a;
    p.list_stride = a.keep;
    if (w.list) {
        uint8_t* ws = static_cast<uint8_t*>(workspace);
        p.counts = reinterpret_cast<int32_t*>(ws);
        p.list = reinterpret_cast<int2*>(ws + w.counts);
        p.movers = reinterpret_cast<int32_t*>(ws + w.counts + w.list);
    }
    // short contexts: several small CTAs per SM; long ones: a CTA of 1,024
    // threads holds an SM's shared memory anyway
    cudaError_t e = a.max_context > select_max(1024, true)  ? launch_select<1024, false>(p, units, stream)
                    : a.max_context > select_max(512, true) ? launch_select<1024, true>(p, units, stream)
                    : a.max_context > select_max(256, true) ? launch_select<512, true>(p, units, stream)
                                                            : launch_select<256, true>(p, units, stream);
    if (e != cudaSuccess) return e;
    const int rows = std::max(1, std::min(a.keep, a.max_context));
    const int ctas = (int)std::max<int64_t>(
        1, std::min<int64_t>(kMoveCtas / units, (rows + kMoveWarps * kWarpRows - 1) / (kMoveWarps * kWarpRows)));
    const dim3 grid((unsigned)(units * ctas)), block(32 * kMoveWarps);
    const int64_t rb = a.row_bytes;
    if (rb % 16 == 0) return launch_pdl(evict_move_kernel<16>, grid, block, stream, p, ctas);
    if (rb % 8 == 0) return launch_pdl(evict_move_kernel<8>, grid, block, stream, p, ctas);
    if (rb % 4 == 0) return launch_pdl(evict_move_kernel<4>, grid, block, stream, p, ctas);
    if (rb % 2 == 0) return launch_pdl(evict_move_kernel<2>, grid, block, stream, p, ctas);
    return launch_pdl(evict_move_kernel<1>, grid, block, stream, p, ctas);
}

}  // namespace pa
