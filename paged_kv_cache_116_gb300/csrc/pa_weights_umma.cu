// pa_weights_umma.cu -- attention weights of a request's cached tokens on the
// 5th-generation tensor cores (tcgen05.mma, accumulators in tensor memory):
// bf16/f16 queries, head_dim 64, 128 or 256.  The definition stands at the head of pa_weights_simt.cu; the two
// passes over Q K^T are here one kernel in two forms:
//
//   pass 1 (row statistics)  stationary A = 128 query rows, streamed B = the
//                            128-key tiles they see; a thread owns a row and
//                            keeps its running maximum and sum;
//   pass 2 (key weights)     stationary A = 128 keys, streamed B = the tiles
//                            of 128 query rows that see them; a thread owns a
//                            key and sums exp2(x - M_row) / l_row over the
//                            rows.
//
//   pass 2 for few rows      (all counted rows of a request fit the
//                            stationary tiles) the other way round: the query
//                            tiles stay as B, the keys stream through as A.
//
// In all of them the reduction runs along the columns of the accumulator,
// that is within one thread's tensor-memory lane: no shuffle, no atomics, a
// fixed order.  A query tile is T = floor(128 / G) consecutive new tokens with
// the G query heads of a KV head (row t G + g).
//
// Up to head_dim 128 a CTA keeps two stationary tiles, so that every streamed
// tile feeds two MMAs: with one the streamed tiles crossed from L2 twice as
// often, a third more time in all (8,192-token prompt, 32 / 8 heads of 128).
//
// Bound: the groups' work on the columns, by issue slots and the exponential
// unit (32 per cycle and SM, 512 cycles per accumulator, as many as its MMAs
// take); a pass spends about 1,120 cycles per accumulator, 255 and 268 us on
// 8,192 tokens with 32 / 8 heads (550 GFLOP in both: 1.05 PFLOP/s).  With a
// short window over long contexts: the two reads of the keys (4 x 32,768 keys
// of 8 heads, 32 rows: 61 and 71 us, 3.9-4.5 TB/s).
//
// Pools with block_size 8 or a multiple of 16 up to 256 are read in place.
// Others, and code pools, are first laid out densely in the workspace, codes
// as their exact values in the query's type; a code row's scale multiplies the
// fp32 score (of the key's column in pass 1, of its lane in pass 2).
//
// Where there are few stationary tiles the streamed axis is split: pass 1's
// pieces of (maximum, sum) are joined by a small kernel, pass 2's partial
// weights added by another.
//
// Roles (20 warps up to head_dim 128): four groups of four warps work the
// accumulator tiles, one row or key per thread; two warps load tiles by TMA
// (128-byte swizzle; keys through the block table, one 16-token group per
// box); one warp per stationary tile issues its MMAs (one warp for both: 3 % slower
// on 8,192 tokens).
// Accumulators are (stationary tile x, parity of the streamed tile within its
// item), 128 columns each; the parity decides which group adds what up, so it
// may not depend on what a CTA worked before.  In pass 1 a group owns one of them; in pass 2 it owns half of
// the columns of both tiles' accumulators of a parity, so that every column
// statistic it reads from shared memory serves two keys.  Every wait is
// bounded; on expiry the CTA sets a status bit, abandons its work, waits
// (bounded) for its loads in flight and frees its tensor memory.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <string>
#include <type_traits>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_items.cuh"
#include "pa_launch.cuh"
#include "pa_tmap.cuh"
#include "pa_weights.cuh"

namespace pa {
namespace {


// One lane of a converged warp.  MMAs issued under it, with operands that the
// compiler knows to be the same in every lane (shuffled from lane 0), go out
// one per 64 cycles; the same loop under `if (lane == 0)` takes 115-138 cycles
// per MMA (128 x 128 x 16), because every descriptor then has to be moved to
// uniform registers one by one.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ uint32_t lane0(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
// Shared-memory matrix descriptor of a 128-byte-swizzled tile from its low
// word (address >> 4 | leading byte offset): stride 1024 bytes, version 1.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t lo) {
    return (uint64_t)((1024u >> 4) | (1u << 14) | (2u << 29)) << 32 | lo;
}

__device__ unsigned int g_weights_status;

constexpr int TM = 128;                       // rows of A and columns of B
constexpr int GRP = 16;                       // keys per TMA box (two boxes of 8 with 8-token blocks)
constexpr int NGRP = TM / GRP;
constexpr uint64_t WAIT_NS = 2000000000ull;   // 2 s

template <int HD>
struct WGeo {
    static constexpr int NA = HD <= 128 ? 2 : 1;    // stationary tiles
    static constexpr int RING = HD == 64 ? 6 : HD == 128 ? 4 : 2;  // streamed tiles in flight
    static constexpr int NWG = 2 * NA;              // accumulators and their warp groups
    static constexpr int NPROD = 2;                 // loading warps
    static constexpr int W_PROD = 4 * NWG, W_MMA = W_PROD + NPROD, NTHREADS = 32 * (W_MMA + NA);
    static constexpr uint32_t TMEM_COLS = NWG * TM;
    static constexpr int CH = HD / 64;        // 128-byte chunks of a row
    static constexpr int CHB = TM * 128;      // bytes of one chunk of a tile
    static constexpr int TILE = CH * CHB;
    static constexpr int RING_OFF = NA * TILE;
    // pass 2: the streamed query tiles' statistics, SRING x {-M, 1 / l}[128];
    // few rows: the stationary ones', [NA]{-M, 1 / l}[128]
    static constexpr int SRING = 8;
    static constexpr int STAT_OFF = RING_OFF + RING * TILE;
    static constexpr int JOIN_OFF = STAT_OFF + SRING * 2 * TM * 4;  // results handed over, float2[3][128]
    static constexpr int BAR_OFF = JOIN_OFF + 3 * TM * 8;
    // a_full, a_empty, b_full[RING], b_empty[RING], d_full[NWG],
    // s_full[SRING], i_full[IRING], d_empty[NWG], s_empty[SRING],
    // i_empty[IRING], g_bar, j_full[3], j_empty[3]
    static constexpr int IRING = 4;  // work items handed to the CTA's warps
    static constexpr int NBAR = 2 + 2 * RING + 2 * NWG + 2 * SRING + 2 * IRING + 7;
    static constexpr int ITEM_OFF = BAR_OFF + NBAR * 8;  // int[IRING]
    static constexpr int ADDR_OFF = ITEM_OFF + IRING * 4;
    static constexpr int PREF_OFF = ADDR_OFF + 16;
};
static_assert(1024 + WGeo<128>::PREF_OFF + (kWeightMaxSeqsPerLaunch + 1) * 4 <= 232448 &&
                  1024 + WGeo<256>::PREF_OFF + (kWeightMaxSeqsPerLaunch + 1) * 4 <= 232448,
              "tiles and the batch's prefix fit in shared memory");
template <int HD>
size_t weights_smem(int num_seqs) { return 1024 + WGeo<HD>::PREF_OFF + (size_t)(num_seqs + 1) * 4; }

// One work item, as every role sees it.
struct Item {
    WeightSeq sq;
    int h;
    int a0, na;  // first stationary tile (query tile, or key tile in pass 2) and how many
    int b0, b1;  // streamed tiles
    int z;       // piece of the streamed axis
};

// What pass 2 needs of a row, (-M, 1 / l): its weights are exp2(x - M) / l.
// One number -(M + log2 l) would spare half of pass 2's reads of statistics
// (8,192 tokens: 517 instead of 533 us), but its rounding, 2^-24 of its size,
// would be in every weight of the row: against 64 bits the whole prompt's
// weights are off by 3.4e-7 in norm (one number: 3.9e-7), 16 chunks' by
// 1.6e-7 (1.9e-7).  What is left is the tensor cores' accumulation, which cuts
// where fp32 addition rounds: neither exp2f in place of ex2.approx nor
// compensated sums of the tiles change it.  A row with only scores of
// -infinity (l = 0) gets 1 / l infinite, hence NaN weights, as its softmax has.
__device__ __forceinline__ float2 row_stat(float m, float l) {
    return make_float2(m == -INFINITY ? 0.f : -m, 1.f / l);
}

// The statistics of one row (an index into a piece of p.stats), joined over
// pass 1's key splits.
__device__ __forceinline__ float2 joined_stat(const WeightArgs& p, int64_t row) {
    const int64_t part = (int64_t)p.stat_rows * p.num_heads;
    constexpr int B = 8;  // pieces in flight
    float2 s = make_float2(-INFINITY, 0.f);
    for (int z0 = 0; z0 < p.key_splits; z0 += B) {
        float2 o[B];
#pragma unroll
        for (int b = 0; b < B; ++b)
            o[b] = z0 + b < p.key_splits ? __ldcg(p.stats + (z0 + b) * part + row) : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const float mn = fmaxf(s.x, o[b].x);
            if (mn == -INFINITY) {  // no key, or none with a number for a score
                s.y += o[b].y;
                continue;
            }
            s.y = s.y * exp2f(s.x - mn) + o[b].y * exp2f(o[b].x - mn);
            s.x = mn;
        }
    }
    return row_stat(s.x, s.y);
}

enum Pass { kRowStats = 1, kKeyWeights = 2, kFewRows = 3 };

// T: the element type of q and the keys.  SC: keys have scales
// (p.key_scales, the score's scale in them).
template <typename T, int HD, int PASS, bool SC>
__global__ void __launch_bounds__(WGeo<HD>::NTHREADS, 1)
    weights_umma_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const WeightArgs p) {
    using Gm = WGeo<HD>;
    constexpr int NA = Gm::NA, RING = Gm::RING, NTH = Gm::NTHREADS;
    constexpr bool kBF16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr bool kKeysStream = PASS != kKeyWeights;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(base + Gm::BAR_OFF);
    uint64_t* a_full = bars;
    uint64_t* a_empty = bars + 1;
    uint64_t* b_full = bars + 2;
    uint64_t* b_empty = b_full + RING;
    uint64_t* d_full = b_empty + RING;
    uint64_t* s_full = d_full + Gm::NWG;
    uint64_t* i_full = s_full + Gm::SRING;
    uint64_t* d_empty = i_full + Gm::IRING;
    uint64_t* s_empty = d_empty + Gm::NWG;
    uint64_t* i_empty = s_empty + Gm::SRING;
    uint64_t* g_bar = i_empty + Gm::IRING;
    volatile int* item_s = reinterpret_cast<volatile int*>(base + Gm::ITEM_OFF);
    uint64_t* j_full = g_bar + 1;
    uint64_t* j_empty = j_full + 3;
    float* stat_s = reinterpret_cast<float*>(base + Gm::STAT_OFF);
    // keys streamed with their scales: kScaleRing x [128] behind the stationary statistics
    constexpr int kScaleRing = 4, kRing = PASS == kKeyWeights ? Gm::SRING : kScaleRing;
    float* scale_s = stat_s + NA * 2 * TM;
    static_assert(kScaleRing + 2 * NA <= 2 * Gm::SRING, "scales fit behind the statistics");
    float2* join_s = reinterpret_cast<float2*>(base + Gm::JOIN_OFF);
    volatile uint32_t* taddr_slot = reinterpret_cast<volatile uint32_t*>(base + Gm::ADDR_OFF);
    int32_t* prefix = reinterpret_cast<int32_t*>(base + Gm::PREF_OFF);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = p.num_heads / p.num_kv_heads, Hkv = p.num_kv_heads, TT = TM / G;

    if (threadIdx.x == 32 * Gm::W_PROD) {
        prefetch_tmap(&tmQ);
        prefetch_tmap(&tmK);
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < Gm::NBAR; ++i) {
            const uint64_t* b = bars + i;
            // a_empty, b_empty: one commit per issuing warp; from d_empty on
            // one arrival per warp: of the groups that work the accumulator
            // or tile, of all warps (i_empty), of all groups (g_bar), of one
            // group (j_*)
            const uint32_t groups =
                b >= j_full ? 1 : b >= g_bar ? Gm::NWG : b < s_empty && PASS == kRowStats ? 1 : NA;
            const bool per_mma = b == a_empty || (b >= b_empty && b < d_full), each_warp = b >= i_empty && b < g_bar;
            mbar_init(bars + i, each_warp ? NTH / 32 : b >= d_empty ? 4 * groups : per_mma ? NA : 1u);
        }
        mbar_fence_init();
    }
    // tensor memory is taken after the previous grid is done: its CTAs may
    // still be waiting for theirs on this SM
    pdl_wait_primary();
    pdl_launch_dependents();
    work_prefix(p, prefix, [&](const WeightSeq& sq) {
        if (PASS == kFewRows) return sq.rows ? 1 : 0;
        const int tiles = PASS == kRowStats ? (sq.rows + TT - 1) / TT : sq.rows ? (sq.L + TM - 1) / TM : 0;
        return (tiles + NA - 1) / NA;
    });
    // an item is a piece of the streamed axis of a (request, KV head, group of
    // stationary tiles)
    const int splits = PASS == kRowStats ? p.key_splits : p.row_splits;
    const int64_t items = (int64_t)prefix[p.num_seqs] * Hkv * splits;
    if (blockIdx.x >= items) return;  // uniform for the CTA
    if (warp == Gm::W_MMA) {
        tmem_alloc(const_cast<uint32_t*>(taddr_slot), Gm::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *taddr_slot;

    auto item_at = [&](int64_t it) -> Item {
        Item w;
        int s, tile;
        const int64_t unit = it / splits;
        w.z = (int)(it - unit * splits);
        locate_work(prefix, p.num_seqs, Hkv, unit, s, w.h, tile);
        w.sq = weight_seq(p, s);
        const int q_tiles = (w.sq.rows + TT - 1) / TT, k_tiles = (w.sq.L + TM - 1) / TM;
        int n;
        if (PASS == kKeyWeights) {
            w.a0 = tile * NA;
            w.na = min(NA, k_tiles - w.a0);
            w.b0 = p.causal ? max(0, w.a0 * TM - (w.sq.L - w.sq.rows)) / TT : 0;
            n = q_tiles - w.b0;
        } else {
            // late tiles see the most keys under a causal mask: they go first
            w.a0 = PASS == kFewRows ? 0 : ((q_tiles + NA - 1) / NA - 1 - tile) * NA;
            w.na = min(NA, q_tiles - w.a0);
            const int last = min(w.sq.rows, (w.a0 + w.na) * TT);
            const int seen = p.causal ? w.sq.L - w.sq.rows + last : w.sq.L;
            w.b0 = 0;
            n = (max(seen, 0) + TM - 1) / TM;
        }
        w.b1 = w.b0 + (int)((int64_t)n * (w.z + 1) / splits);
        w.b0 += (int)((int64_t)n * w.z / splits);
        return w;
    };
    // where query tile t of a request keeps its statistics: distinct for every
    // (request, tile), since a request's ceil(rows / T) tiles fit between its
    // floor(stat0 / T) + s and the next request's
    auto stat_tile = [&](const WeightSeq& sq, int h, int t) -> int64_t {
        return (int64_t)h * p.stat_tiles + sq.stat0 / TT + sq.s + t;
    };
    // The CTA's items: its own number first, then whatever is next in the grid
    // (items differ in length; dealt out in advance they left SMs idle).  The
    // first producer draws them as it gets to them; every warp takes each in
    // turn.
    auto fail = [&]() { atomicOr(&g_weights_status, kStatusTimeout); };
    ItemRing<Gm::IRING> ring{i_full, i_empty, item_s};
    auto next_item = [&](bool& run) -> int {
        const int it = ring.next(warp == Gm::W_PROD, WAIT_NS, [&]() -> int {
            // (drawn only now: an item drawn ahead would wait for this CTA
            // while others run dry, 10 % more time on 8,192 tokens)
            const int64_t i = ring.n == 0 ? blockIdx.x : (int64_t)gridDim.x + atomicAdd(p.next_item + (PASS > 1), 1u);
            return i < items ? (int)i : kItemsDone;
        });
        if (it == kItemsExpired) {  // the other items are lost: reported here, in whatever role
            run = false;
            if (lane == 0) fail();
        }
        return it;
    };
    // (in pass 2 a group works both stationary tiles' accumulators of a parity;
    // a lone tile, which only the last keys of a request are, keeps to the first)
    constexpr bool spread_alone = PASS != kKeyWeights;

    if (warp >= Gm::W_PROD && warp < Gm::W_MMA) {
        // ---------------- producer `me` of every NPROD-th streamed tile; the first also loads the stationary ones
        const int me = warp - Gm::W_PROD;
        const uint64_t pol = l2_policy_evict_last();  // keys are read twice, query tiles by every key tile
        const int bsz = p.block_size, halves = !p.dense_stride && bsz == 8 ? 2 : 1;
        const int nbox = NGRP * halves;  // boxes along the keys of a tile
        int na = 0, nb = 0;
        bool run = true;
        // pool row of box `lane` of key tile kt (where the second half of a
        // group holds no context, the first half's; never read past it)
        auto key_row = [&](const Item& w, int kt) -> int32_t {
            if (lane >= nbox) return 0;
            if (p.dense_stride) return w.sq.s * p.dense_stride + kt * TM + lane * GRP;
            const int32_t* table = p.block_tables + (int64_t)w.sq.s * p.max_blocks;
            int tok = kt * TM + lane * (GRP / halves);
            if (halves == 2 && (lane & 1) && tok >= w.sq.L) tok -= 8;
            if (tok >= w.sq.L) return 0;
            return table[tok / bsz] * bsz + tok % bsz;
        };
        auto key_groups = [&](const Item& w, int kt) { return min(NGRP, (w.sq.L - kt * TM + GRP - 1) / GRP); };
        auto load_keys = [&](const Item& w, int kt, int32_t row, uint8_t* dst, uint64_t* bar) {
            const int boxes = key_groups(w, kt) * halves * Gm::CH;
            for (int e0 = 0; e0 < boxes; e0 += 32) {
                const int e = e0 + lane, b = e / Gm::CH, c = e - b * Gm::CH;  // box along the keys, chunk
                const int32_t r = __shfl_sync(0xffffffffu, row, min(b, 31));
                if (e < boxes)
                    tma_load_3d(dst + c * Gm::CHB + b * (GRP / halves) * 128, &tmK, bar, 0, w.h * Gm::CH + c, r, pol);
            }
        };
        auto load_queries = [&](const Item& w, int tile, uint8_t* dst, uint64_t* bar) {
            if (lane < Gm::CH)
                tma_load_3d(dst + lane * Gm::CHB, &tmQ, bar, 64 * lane, w.h * G, w.sq.row0 + tile * TT, pol);
        };
        const uint32_t group_bytes = GRP * 128 * Gm::CH, query_bytes = Gm::CH * 128 * G * TT;
        auto expect = [&](uint64_t* bar, uint32_t bytes) {
            if (lane == 0) {
                fence_proxy_async_smem();
                mbar_arrive_expect_tx(bar, bytes);
            }
            __syncwarp();
        };
        auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
            int ok = 0;
            if (lane == 0) {
                ok = mbar_wait_ns(bar, parity, WAIT_NS);
                if (!ok) fail();
            }
            return __shfl_sync(0xffffffffu, ok, 0) != 0;
        };
        for (int it; run && (it = next_item(run)) >= 0;) {
            const Item w = item_at(it);
            if (w.b0 >= w.b1) continue;
            const int mine = w.b0 + (nb + me) % Gm::NPROD;  // this warp's first tile of the item
            int32_t row = kKeysStream && mine < w.b1 ? key_row(w, mine) : 0;
            if (me == 0 && !(run = wait(a_empty, (uint32_t)(na & 1) ^ 1u))) break;
            if (me != 0) {
                // (the first producer's)
            } else if (kKeysStream) {
                expect(a_full, w.na * query_bytes);
                for (int x = 0; x < w.na; ++x) load_queries(w, w.a0 + x, base + x * Gm::TILE, a_full);
            } else {
                uint32_t bytes = 0;
                for (int x = 0; x < w.na; ++x) bytes += key_groups(w, w.a0 + x) * group_bytes;
                expect(a_full, bytes);
                for (int x = 0; x < w.na; ++x)
                    load_keys(w, w.a0 + x, key_row(w, w.a0 + x), base + x * Gm::TILE, a_full);
            }
            ++na;
            for (int t = w.b0; t < w.b1; ++t, ++nb) {
                if ((nb + me) % Gm::NPROD) continue;
                const int slot = nb % RING;
                uint8_t* dst = base + Gm::RING_OFF + slot * Gm::TILE;
                if (!(run = wait(&b_empty[slot], (uint32_t)(nb / RING & 1) ^ 1u))) break;
                if (kKeysStream) {
                    expect(&b_full[slot], key_groups(w, t) * group_bytes);
                    load_keys(w, t, row, dst, &b_full[slot]);
                    if (t + Gm::NPROD < w.b1) row = key_row(w, t + Gm::NPROD);
                    if constexpr (SC) {
                        const int sl = nb % kScaleRing;
                        if (!(run = wait(&s_empty[sl], (uint32_t)(nb / kScaleRing & 1) ^ 1u))) break;
                        expect(&s_full[sl], TM * 4);
                        if (lane == 0)
                            bulk_g2s(scale_s + sl * TM, p.key_scales + ((int64_t)w.sq.s * Hkv + w.h) * p.dense_stride + t * TM,
                                     TM * 4, &s_full[sl]);
                    }
                } else {
                    expect(&b_full[slot], query_bytes);
                    load_queries(w, t, dst, &b_full[slot]);
                    const int sl = nb % Gm::SRING;
                    if (!(run = wait(&s_empty[sl], (uint32_t)(nb / Gm::SRING & 1) ^ 1u))) break;
                    expect(&s_full[sl], 2 * TM * 4);
                    if (lane == 0)
                        bulk_g2s(stat_s + sl * 2 * TM, p.tile_stats + stat_tile(w.sq, w.h, t) * 2 * TM, 2 * TM * 4,
                                 &s_full[sl]);
                }
            }
        }
        if (!run) {  // copies in flight land before the CTA's shared memory is given up
            if (me == 0 && na) mbar_wait_ns(a_full, (uint32_t)(na - 1) & 1u, WAIT_NS);
            for (int j = max(0, nb - RING); j <= nb; ++j)
                if ((j + me) % Gm::NPROD == 0 && j < nb + (PASS == kKeyWeights || SC))
                    mbar_wait_ns(&b_full[j % RING], (uint32_t)(j / RING) & 1u, WAIT_NS);
            if (PASS == kKeyWeights || SC)
                for (int j = max(0, nb - kRing); j < nb; ++j)
                    if ((j + me) % Gm::NPROD == 0)
                        mbar_wait_ns(&s_full[j % kRing], (uint32_t)(j / kRing) & 1u, WAIT_NS);
        }
    } else if (warp >= Gm::W_MMA) {
        // ---------------- MMA issuer of stationary tile x
        const uint32_t x = lane0(warp - Gm::W_MMA);
        const uint32_t idesc = umma_idesc_f16(TM, TM, kBF16, false);
        const uint32_t s_lo = lane0(smem_u32(base) >> 4 | 1u << 16);
        const uint32_t d_x = lane0(tmem) + x * 2 * TM;
        int na = 0, nb = 0, nd[2] = {0, 0}, last = -1;  // items, streamed tiles, accumulators of each parity
        bool run = true;
        for (int it; run && (it = next_item(run)) >= 0;) {
            const Item w = item_at(it);
            if (w.b0 >= w.b1) continue;
            if (!(run = mbar_wait_ns_warp(a_full, (uint32_t)na & 1u, WAIT_NS))) break;
            ++na;
            const bool alone = NA == 2 && w.na == 1;  // one stationary tile: its tiles take all four accumulators in turn
            const uint32_t a_lo = lane0(s_lo + (alone ? 0 : x) * (Gm::TILE / 16));
            for (int t = w.b0; t < w.b1; ++t, ++nb) {
                const int slot = nb % RING, par = (t - w.b0) & 1, turn = par ? nd[1] : nd[0];
                const bool mine = alone ? spread_alone && ((t - w.b0) >> 1 & 1) == (int)x || !spread_alone && x == 0 : true;
                run = __all_sync(0xffffffffu, mbar_wait_ns(&b_full[slot], (uint32_t)(nb / RING) & 1u, WAIT_NS) &&
                                                  (!mine || mbar_wait_ns(&d_empty[2 * x + par],
                                                                         ((uint32_t)turn & 1u) ^ 1u, WAIT_NS)));
                if (!run) break;
                tc_fence_after();
                const uint32_t b_lo = lane0(s_lo + (Gm::RING_OFF + slot * Gm::TILE) / 16);
                // the accumulator's lanes are query rows, or keys
                const uint32_t l_lo = PASS == kFewRows ? b_lo : a_lo, c_lo = PASS == kFewRows ? a_lo : b_lo;
                const uint32_t d = lane0(d_x + par * TM);
                if (elect_one()) {
                    if (mine) {
#pragma unroll
                        for (int kk = 0; kk < HD / 16; ++kk) {
                            const uint32_t off = ((kk >> 2) * Gm::CHB + (kk & 3) * 32) / 16;
                            umma_f16(d, sw128_desc(l_lo + off), sw128_desc(c_lo + off), idesc, kk > 0 ? 1u : 0u);
                        }
                        umma_commit(&d_full[2 * x + par]);
                    }
                    umma_commit(&b_empty[slot]);
                    if (t == w.b1 - 1) umma_commit(a_empty);
                }
                __syncwarp();
                if (mine) {
                    ++(par ? nd[1] : nd[0]);
                    last = par;
                }
            }
        }
        if (!run) {
            if (lane == 0) fail();
            if (last >= 0)  // MMAs in flight
                mbar_wait_ns(&d_full[2 * x + last], (uint32_t)((last ? nd[1] : nd[0]) - 1) & 1u, WAIT_NS);
        }
    } else {
        // ---------------- accumulator tiles: one row or key per thread.  Group
        // (hi, par): the streamed tiles of parity par; in pass 1 stationary
        // tile hi, in pass 2 columns 64 hi .. 64 hi + 63 of every tile.
        const int wg = warp >> 2, hi = wg >> 1, par = wg & 1, m = threadIdx.x & 127;
        constexpr int HC = TM / NA;  // columns of a group in pass 2
        const uint32_t acc = tmem + ((uint32_t)((warp & 3) * 32) << 16) + par * TM;  // + 2 TM x
        const float sl = p.scale_log2;
        const int64_t part = (int64_t)p.stat_rows * p.num_heads;  // rows of one split's statistics
        int nx = 0, n_meet = 0;              // streamed tiles; barriers gone through
        int n_join[3] = {0, 0, 0};           // handovers through each buffer
        int n_d[2] = {0, 0};                 // accumulators of x worked by this group
        bool run = true;
        auto release = [&](int x) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&d_empty[2 * x + par]);
        };
        // (each lane's own answer: the warp's is the vote of all, one for the waits of a tile)
        auto acquire = [&](int x) -> bool {
            const bool ok = mbar_wait_ns(&d_full[2 * x + par], (uint32_t)n_d[x]++ & 1u, WAIT_NS);
            tc_fence_after();
            return ok;
        };
        // a giving group hands its values to the receiving one through buffer j;
        // the turns of each buffer are counted by all groups
        auto give = [&](int j, float2 v) -> bool {
            if (!mbar_wait_ns_warp(&j_empty[j], ((uint32_t)n_join[j] & 1u) ^ 1u, WAIT_NS)) return false;
            join_s[j * TM + m] = v;
            __syncwarp();
            if (lane == 0) mbar_arrive(&j_full[j]);
            return true;
        };
        auto take = [&](int j, float2& v) -> bool {
            if (!mbar_wait_ns_warp(&j_full[j], (uint32_t)n_join[j] & 1u, WAIT_NS)) return false;
            v = join_s[j * TM + m];
            __syncwarp();
            if (lane == 0) mbar_arrive(&j_empty[j]);
            return true;
        };
        // this warp is done with what slot sl of the statistics (or scales) ring holds
        auto used = [&](int sl_) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_empty[sl_]);
        };
        // a bounded barrier of all groups
        auto meet = [&]() -> bool {
            __syncwarp();
            if (lane == 0) mbar_arrive(g_bar);
            return mbar_wait_ns_warp(g_bar, (uint32_t)n_meet++ & 1u, WAIT_NS);
        };
        // exp2(x - M) / l of 16 columns of one or both stationary tiles'
        // accumulators, added to v[] and v2[] of this thread's keys (nm: the
        // columns' -M, TM further on their 1 / l)
        auto add_whole = [&](auto count, const float (&a)[2][16], const float (&ks)[2], const float* nm,
                             unsigned long long (&v2)[2]) {
            constexpr int N = decltype(count)::value;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 n4 = *reinterpret_cast<const float4*>(nm + 4 * j);
                const float4 i4 = *reinterpret_cast<const float4*>(nm + TM + 4 * j);
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const unsigned long long sv = f32x2_pack(ks[k], ks[k]);
                    float x0, x1, x2, x3;
                    f32x2_unpack(fma_f32x2(f32x2_pack(a[k][4 * j], a[k][4 * j + 1]), sv, f32x2_pack(n4.x, n4.y)), x0, x1);
                    f32x2_unpack(fma_f32x2(f32x2_pack(a[k][4 * j + 2], a[k][4 * j + 3]), sv, f32x2_pack(n4.z, n4.w)), x2, x3);
                    v2[k] = fma_f32x2(f32x2_pack(fast_exp2(x0), fast_exp2(x1)), f32x2_pack(i4.x, i4.y), v2[k]);
                    v2[k] = fma_f32x2(f32x2_pack(fast_exp2(x2), fast_exp2(x3)), f32x2_pack(i4.z, i4.w), v2[k]);
                }
            }
        };
        // the same where a mask may cut: column c0 + j counts if lo[] <= c0 + j < end
        auto add_columns = [&](auto count, const float (&a)[2][16], const float (&ks)[2], const float* nm, int c0, bool whole, const int (&lo)[2], int end, float (&v)[2],
                               unsigned long long (&v2)[2]) {
            constexpr int N = decltype(count)::value;
            // columns past the tile's T G rows hold whatever was there
            if (whole && c0 + 16 <= TT * G) {
                add_whole(count, a, ks, nm, v2);
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j)
#pragma unroll
                    for (int k = 0; k < N; ++k)
                        if (c0 + j >= lo[k] && c0 + j < end)
                            v[k] = fmaf(fast_exp2(fmaf(a[k][j], ks[k], nm[j])), nm[TM + j], v[k]);
            }
        };
        auto store_weight = [&](const Item& w, int key, float v) {
            if (key >= w.sq.L) return;
            const int64_t row = (int64_t)w.sq.s * Hkv + w.h;
            if (PASS == kKeyWeights && splits > 1) {
                p.partial[((int64_t)w.z * p.num_seqs * Hkv + row) * p.max_context + key] = v;
            } else {
                float* dst = p.weights + row * p.weights_stride + key;
                *dst = key < w.sq.L - w.sq.n ? *dst + v : v;
            }
        };
        for (int it; run && (it = next_item(run)) >= 0;) {
            const Item w = item_at(it);
            if constexpr (PASS == kRowStats) {
                // a lone stationary tile is worked by all groups, every fourth
                // streamed tile each; else group hi, par works tile hi's
                const bool alone = NA == 2 && w.na == 1;
                const int x = alone ? 0 : hi;
                const int tok = (w.a0 + x) * TT + m / G, g = m % G;
                const bool valid = m < TT * G && tok < w.sq.rows;
                const int last = p.causal ? w.sq.L - w.sq.rows + tok : w.sq.L - 1;  // last key the row sees
                float m_used = -INFINITY, l = 0.f;
                for (int t = w.b0; t < w.b1; ++t, ++nx) {
                    if (!SC) {
                        if (((t - w.b0) & 1) != par || (alone && ((t - w.b0) >> 1 & 1) != hi)) continue;
                    } else {
                        if (((t - w.b0) & 1) != par) continue;
                    }
                    const float* ks = scale_s + nx % kScaleRing * TM;  // the tile's key scales (SC)
                    if constexpr (SC) {
                        const int sl_ = nx % kScaleRing;
                        if (!(run = mbar_wait_ns_warp(&s_full[sl_], (uint32_t)(nx / kScaleRing) & 1u, WAIT_NS))) break;
                        if (alone && ((t - w.b0) >> 1 & 1) != hi) {  // another group's; it is counted all the same
                            used(sl_);
                            continue;
                        }
                    }
                    if (!(run = __all_sync(0xffffffffu, acquire(hi)))) break;
                    // rows that hold no query are never stored; they take the
                    // unmasked path with their warp
                    const int vis = valid ? min(last - t * TM, TM - 1) : TM - 1;
                    const bool full = __all_sync(0xffffffffu, vis == TM - 1);
                    float sum = 0.f;
                    // Exponentials are taken against a maximum that the row
                    // keeps until a tile outgrows it by more than 2^8 (the sum
                    // of the exponentials, which bounds them, tells); only
                    // then, on the first tile and for a non-positive scale the
                    // tile's own maximum is taken first.
                    auto exp_pass = [&](float neg) {
                        sum = 0.f;
                        unsigned long long s2 = f32x2_pack(0.f, 0.f);
                        const unsigned long long sv = f32x2_pack(sl, sl), nv = f32x2_pack(neg, neg);
                        // (rolled, and the masked form apart: the four groups' loops
                        // otherwise wait for instructions, 575 against 521 us
                        // with both passes so, 8,192 tokens)
                        if (full) {
#pragma unroll 1
                            for (int q = 0; q < TM / 32; ++q) {
                                float a[32];
                                tmem_ld32(acc + 2 * TM * hi + 32 * q, a);
                                tmem_wait_ld();
#pragma unroll
                                for (int j = 0; j < 16; ++j) {
                                    const float2 k2 = SC ? *reinterpret_cast<const float2*>(ks + 32 * q + 2 * j) : make_float2(sl, sl);
                                    float x0, x1;
                                    f32x2_unpack(fma_f32x2(f32x2_pack(a[2 * j], a[2 * j + 1]), SC ? f32x2_pack(k2.x, k2.y) : sv, nv), x0, x1);
                                    s2 = add_f32x2(s2, f32x2_pack(fast_exp2(x0), fast_exp2(x1)));
                                }
                            }
                        } else {
#pragma unroll 1
                            for (int q = 0; q < TM / 32; ++q) {
                                float a[32];
                                tmem_ld32(acc + 2 * TM * hi + 32 * q, a);
                                tmem_wait_ld();
#pragma unroll
                                for (int j = 0; j < 32; ++j)
                                    sum += 32 * q + j <= vis ? fast_exp2(fmaf(a[j], SC ? ks[32 * q + j] : sl, neg)) : 0.f;
                            }
                        }
                        float s0, s1;
                        f32x2_unpack(s2, s0, s1);
                        sum += s0 + s1;
                    };
                    auto max_pass = [&]() -> float {
                        float mt = -INFINITY;
#pragma unroll 1
                        for (int q = 0; q < TM / 32; ++q) {
                            float a[32];
                            tmem_ld32(acc + 2 * TM * hi + 32 * q, a);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (32 * q + j <= vis) mt = fmaxf(mt, a[j] * (SC ? ks[32 * q + j] : sl));
                        }
                        return mt;
                    };
                    bool settled = !(sl > 0.f && __all_sync(0xffffffffu, m_used != -INFINITY));
                    float alpha = 1.f;
                    auto settle = [&](float mt) {
                        const float mn = fmaxf(m_used, mt);
                        if (m_used == -INFINITY || mn > m_used + 8.f) {
                            alpha = mn == -INFINITY ? 1.f : fast_exp2(m_used - mn);
                            m_used = mn;
                        }
                    };
                    if (settled) settle(max_pass());
#pragma unroll 1
                    for (;;) {
                        // a row that has seen only scores of -infinity (or no key) keeps a sum of 0
                        exp_pass(m_used == -INFINITY ? 0.f : -m_used);
                        if (settled || __all_sync(0xffffffffu, !(sum > 256.f))) break;
                        settled = true;
                        settle(max_pass());
                    }
                    l = fmaf(l, alpha, sum);
                    release(hi);
                    if constexpr (SC) used(nx % kScaleRing);
                }
                if (!run) break;
                // group 2 hi gets 2 hi + 1's; group 0 those of all others where the tile is alone
                const bool taker = alone ? wg == 0 : par == 0;
                if (!taker) {
                    run = give(wg - 1, make_float2(m_used, l));
                } else {
                    for (int g = wg; g < (alone ? Gm::NWG - 1 : wg + 1) && run; ++g) {
                        float2 o;
                        if (!(run = take(g, o))) break;
                        const float mn = fmaxf(m_used, o.x);
                        if (mn == -INFINITY) {
                            l += o.y;
                        } else {
                            l = l * exp2f(m_used - mn) + o.y * exp2f(o.x - mn);
                            m_used = mn;
                        }
                    }
                }
#pragma unroll
                for (int g = 0; g < 3; ++g) n_join[g] += alone || g != 1;
                if (!run) break;
                if (taker) {
                    if (splits == 1) {
                        float* st = p.tile_stats + stat_tile(w.sq, w.h, w.a0 + x) * 2 * TM;
                        const float2 v = valid ? row_stat(m_used, l) : make_float2(0.f, 0.f);
                        st[m] = v.x;
                        st[TM + m] = v.y;
                    } else if (valid) {
                        p.stats[(int64_t)w.z * part + (int64_t)(w.sq.stat0 + tok) * p.num_heads + w.h * G + g] =
                            make_float2(m_used, l);
                    }
                }
            } else if constexpr (PASS == kKeyWeights) {
                float total[2] = {0.f, 0.f}, ks[2] = {sl, sl};
                if constexpr (SC) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int key = (w.a0 + x) * TM + m;
                        ks[x] = key < w.sq.L ? __ldcg(p.key_scales + ((int64_t)w.sq.s * Hkv + w.h) * p.dense_stride + key) : 0.f;
                    }
                }
                for (int t = w.b0; t < w.b1; ++t, ++nx) {
                    if (((t - w.b0) & 1) != par) continue;
                    const int sl = nx % Gm::SRING;
                    const float* nm = stat_s + sl * 2 * TM + hi * HC;
                    bool ok = mbar_wait_ns(&s_full[sl], (uint32_t)(nx / Gm::SRING) & 1u, WAIT_NS);
                    ok = acquire(0) && ok;
                    if (w.na == 2) ok = acquire(NA - 1) && ok;
                    if (!(run = __all_sync(0xffffffffu, ok))) break;
                    // column c (query row) counts for key k where lo[k] <= c < end
                    const int end = min(TT, w.sq.rows - t * TT) * G;
                    int lo[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        lo[x] = p.causal ? ((w.a0 + x) * TM + m - (w.sq.L - w.sq.rows) - t * TT) * G : 0;
                    const bool full = __all_sync(0xffffffffu, max(lo[0], lo[NA - 1]) <= 0 && end == TT * G);
                    // summed tile by tile: a running sum over thousands of rows
                    // would round at its own size in every addition
                    float v[2] = {0.f, 0.f};
                    unsigned long long v2[2] = {f32x2_pack(0.f, 0.f), f32x2_pack(0.f, 0.f)};
                    using Both = std::integral_constant<int, NA>;
                    using One = std::integral_constant<int, 1>;
                    if (NA == 2 && full && w.na == 2 && TT * G == TM) {
#pragma unroll 2
                        for (int q = 0; q < HC / 16; ++q) {
                            float a[2][16];
                            tmem_ld16(acc + hi * HC + 16 * q, a[0]);
                            tmem_ld16(acc + 2 * TM + hi * HC + 16 * q, a[1]);
                            tmem_wait_ld();
                            if (q == HC / 16 - 1) {
                                release(0);
                                release(NA - 1);
                            }
                            add_whole(Both(), a, ks, nm + 16 * q, v2);
                        }
                    } else {
#pragma unroll 1
                    for (int q = 0; q < HC / 16; ++q) {
                        float a[2][16];
                        tmem_ld16(acc + hi * HC + 16 * q, a[0]);
                        if (NA == 2 && w.na == 2) tmem_ld16(acc + 2 * TM + hi * HC + 16 * q, a[1]);
                        tmem_wait_ld();
                        if (q == HC / 16 - 1) {
                            release(0);
                            if (w.na == 2) release(NA - 1);
                        }
                        if (w.na == 2) add_columns(Both(), a, ks, nm + 16 * q, hi * HC + 16 * q, full, lo, end, v, v2);
                        else add_columns(One(), a, ks, nm + 16 * q, hi * HC + 16 * q, full, lo, end, v, v2);
                    }
                    }
#pragma unroll
                    for (int x = 0; x < NA; ++x) {
                        float s0, s1;
                        f32x2_unpack(v2[x], s0, s1);
                        total[x] += v[x] + (s0 + s1);
                    }
                    used(sl);
                }
                if (!run) break;
                if (wg > 0) {
                    run = give(wg - 1, make_float2(total[0], total[1]));
                } else {
                    for (int g = 0; g < Gm::NWG - 1 && run; ++g) {
                        float2 o;
                        if (!(run = take(g, o))) break;
                        total[0] += o.x;
                        total[1] += o.y;
                    }
                }
#pragma unroll
                for (int g = 0; g < 3; ++g) ++n_join[g];
                if (!run) break;
                if (wg == 0) {
                    store_weight(w, w.a0 * TM + m, total[0]);
                    if (w.na == 2) store_weight(w, (w.a0 + 1) * TM + m, total[1]);
                }
            } else {
                if (w.b0 >= w.b1) continue;
                // few rows: the item's query tiles stay, their statistics with them
                if (!(run = meet())) break;  // the previous item's are used up
                if (wg < NA) {
                    const float* st = p.tile_stats + stat_tile(w.sq, w.h, wg) * 2 * TM;
                    stat_s[wg * 2 * TM + m] = wg < w.na ? __ldcg(st + m) : 0.f;
                    stat_s[wg * 2 * TM + TM + m] = wg < w.na ? __ldcg(st + TM + m) : 0.f;
                }
                if (!(run = meet())) break;
                for (int t = w.b0; t < w.b1; ++t, ++nx) {
                    if (((t - w.b0) & 1) != par) continue;
                    const int key = t * TM + m;
                    float v = 0.f, ks[2] = {sl, 0.f};
                    if constexpr (SC) {
                        const int sl_ = nx % kScaleRing;
                        if (!(run = mbar_wait_ns_warp(&s_full[sl_], (uint32_t)(nx / kScaleRing) & 1u, WAIT_NS))) break;
                        ks[0] = scale_s[sl_ * TM + m];
                        used(sl_);
                    }
                    const int turn = NA == 2 && w.na == 1 ? (t - w.b0) >> 1 & 1 : 0;  // a lone tile's accumulators rotate
#pragma unroll
                    for (int x = 0; x < NA; ++x) {
                        if (x >= w.na) break;
                        const int ax = x + turn;
                        if (!(run = __all_sync(0xffffffffu, acquire(ax)))) break;
                        const int end = min(TT, w.sq.rows - x * TT) * G;
                        const int lo[2] = {p.causal ? (key - (w.sq.L - w.sq.rows) - x * TT) * G : 0, 0};
                        const bool full = __all_sync(0xffffffffu, lo[0] <= 0 && end == TT * G);
                        float vx[2] = {0.f, 0.f};
                        unsigned long long v2[2] = {f32x2_pack(0.f, 0.f), 0};
                        const float* nm = stat_s + x * 2 * TM + hi * HC;
                        if (full && TT * G == TM) {
#pragma unroll 1
                            for (int q = 0; q < HC / 16; ++q) {
                                float a[2][16];
                                tmem_ld16(acc + 2 * TM * ax + hi * HC + 16 * q, a[0]);
                                tmem_wait_ld();
                                if (q == HC / 16 - 1) release(ax);
                                add_whole(std::integral_constant<int, 1>(), a, ks, nm + 16 * q, v2);
                            }
                        } else {
#pragma unroll 1
                            for (int q = 0; q < HC / 16; ++q) {
                                float a[2][16];
                                tmem_ld16(acc + 2 * TM * ax + hi * HC + 16 * q, a[0]);
                                tmem_wait_ld();
                                if (q == HC / 16 - 1) release(ax);
                                add_columns(std::integral_constant<int, 1>(), a, ks, nm + 16 * q,
                                            hi * HC + 16 * q, full, lo, end, vx, v2);
                            }
                        }
                        float s0, s1;
                        f32x2_unpack(v2[0], s0, s1);
                        v += vx[0] + (s0 + s1);
                    }
                    if (!run) break;
                    if (NA == 2) {  // the other half of the columns
                        float2 o = make_float2(v, 0.f);
                        if (!(run = hi == 1 ? give(par, o) : take(par, o))) break;
                        ++(par ? n_join[1] : n_join[0]);
                        if (hi == 1) continue;
                        v += o.x;
                    }
                    store_weight(w, key, v);
                }
            }
        }
        if (!run && lane == 0) fail();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == Gm::W_MMA) tmem_dealloc(tmem, Gm::TMEM_COLS);
}

// Lays a batch's keys out densely, request s's token t at row s * dense_stride
// + t: codes become their exact values in T and their scales, times the
// score's, a row per (request, KV head); 16-bit keys are copied.  A CTA takes
// 16 tokens at a time, a thread 16 bytes of pool, four in flight.  Bound: HBM
// (4 x 32,768 code keys of 8 heads: 403 MB in 77 us, 5.2 TB/s; with one load
// in flight 95 us).
constexpr int kDenseTokens = 16;
template <typename T, bool FP8>
__global__ void __launch_bounds__(256) dense_keys_kernel(const WeightArgs p, T* __restrict__ keys, float* __restrict__ scales) {
    constexpr int E = FP8 ? 16 : 8, U = 4;  // elements per 16 bytes
    pdl_wait_primary();
    pdl_launch_dependents();
    const int row = p.num_kv_heads * p.head_dim, chunks = row / E, bs = p.block_size;
    for (int s = blockIdx.y; s < p.num_seqs; s += gridDim.y) {
        const WeightSeq sq = weight_seq(p, s);
        if (sq.rows == 0) continue;
        const int32_t* table = p.block_tables + (int64_t)s * p.max_blocks;
        for (int t0 = blockIdx.x * kDenseTokens; t0 < sq.L; t0 += gridDim.x * kDenseTokens) {
            const int n = min(kDenseTokens, sq.L - t0) * chunks;
            for (int e0 = threadIdx.x; e0 < n; e0 += 256 * U) {
                uint4 v[U];
                float sc[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int e = e0 + 256 * u;
                    if (e >= n) break;
                    const int r = e / chunks, c = e - r * chunks, b = (t0 + r) / bs, off = t0 + r - b * bs;
                    const int64_t blk = table[b];
                    v[u] = __ldcg(reinterpret_cast<const uint4*>(p.k_cache) + (blk * bs + off) * chunks + c);
                    if (FP8 && c < p.num_kv_heads) sc[u] = __ldcg(p.k_scales + (blk * p.num_kv_heads + c) * bs + off);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int e = e0 + 256 * u;
                    if (e >= n) break;
                    const int r = e / chunks, c = e - r * chunks, t = t0 + r;
                    uint4* dst = reinterpret_cast<uint4*>(keys + ((int64_t)s * p.dense_stride + t) * row + c * E);
                    if constexpr (FP8) {
                        const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
                        uint32_t o[8];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t lo, hi;
                            e4m3x4_to_f16x2x2(w[k], lo, hi);
                            if constexpr (std::is_same<T, __half>::value) {
                                o[2 * k] = lo;
                                o[2 * k + 1] = hi;
                            } else {  // every code is a bf16 value as well
                                const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
                                const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
                                o[2 * k] = pack2<T>(a.x, a.y);
                                o[2 * k + 1] = pack2<T>(b.x, b.y);
                            }
                        }
                        dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
                        dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
                        if (c < p.num_kv_heads)
                            scales[((int64_t)s * p.num_kv_heads + c) * p.dense_stride + t] = p.scale_log2 * sc[u];
                    } else {
                        *dst = v[u];
                    }
                }
            }
        }
    }
}

// Joins pass 1's key splits into the statistics that pass 2 streams: a thread
// per row of a (request, KV head, query tile).
__global__ void __launch_bounds__(TM) stats_join_kernel(const WeightArgs p) {
    extern __shared__ int32_t prefix[];
    pdl_wait_primary();
    pdl_launch_dependents();
    const int G = p.num_heads / p.num_kv_heads, TT = TM / G, m = threadIdx.x;
    work_prefix(p, prefix, [&](const WeightSeq& sq) { return (sq.rows + TT - 1) / TT; });
    const int64_t items = (int64_t)prefix[p.num_seqs] * p.num_kv_heads;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        int s, h, tile;
        locate_work(prefix, p.num_seqs, p.num_kv_heads, it, s, h, tile);
        const WeightSeq sq = weight_seq(p, s);
        const int tok = tile * TT + m / G;
        const bool row = m < TT * G && tok < sq.rows;
        const float2 v = row ? joined_stat(p, (int64_t)(sq.stat0 + tok) * p.num_heads + h * G + m % G) : make_float2(0.f, 0.f);
        float* st = p.tile_stats + ((int64_t)h * p.stat_tiles + sq.stat0 / TT + s + tile) * 2 * TM;
        st[m] = v.x;
        st[TM + m] = v.y;
    }
}

// The row splits' partial weights, added in order into the weights.
__global__ void __launch_bounds__(256) weights_join_kernel(const WeightArgs p) {
    pdl_wait_primary();
    pdl_launch_dependents();
    const int64_t rows = (int64_t)p.num_seqs * p.num_kv_heads;
    for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
        const WeightSeq sq = weight_seq(p, (int)(row / p.num_kv_heads));
        const int key = blockIdx.x * 256 + threadIdx.x;
        if (key >= sq.L || sq.rows == 0) continue;
        float v = 0.f;
        for (int z = 0; z < p.row_splits; ++z) v += __ldcg(p.partial + ((int64_t)z * rows + row) * p.max_context + key);
        float* dst = p.weights + row * p.weights_stride + key;
        *dst = key < sq.L - sq.n ? *dst + v : v;
    }
}

// ---------------------------------------------------------------- host side

bool encode_map(CUtensorMap* m, const void* ptr, int dtype, const cuuint64_t (&dims)[3], const cuuint64_t (&strides)[2],
                const cuuint32_t (&box)[3], std::string* err) {
    return encode_tiled_3d(m, dtype == 1 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, ptr, dims,
                           strides, box, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, err);
}

template <typename T, int HD, bool SC>
cudaError_t launch_umma(const WeightArgs& args, int32_t num_blocks, std::string* err, cudaStream_t stream) {
    WeightArgs a = args;
    const int G = a.num_heads / a.num_kv_heads, TT = TM / G;
    const int64_t sms = sm_count();
    cudaError_t e = cudaMemsetAsync(a.next_item, 0, 2 * sizeof(uint32_t), stream);
    if (e != cudaSuccess) return e;
    int64_t k_rows = (int64_t)num_blocks * a.block_size;
    if (a.dense_stride) {
        T* keys = static_cast<T*>(a.dense_keys);
        const int64_t per = (a.max_context + kDenseTokens - 1) / kDenseTokens;
        const dim3 grid((unsigned)std::max<int64_t>(1, std::min<int64_t>(per, std::max<int64_t>(1, 8 * sms / a.num_seqs))),
                        (unsigned)a.num_seqs);
        e = launch_pdl(dense_keys_kernel<T, SC>, grid, dim3(256), stream, a, keys, a.key_scales);
        if (e != cudaSuccess) return e;
        a.k_cache = keys;
        k_rows = (int64_t)a.num_seqs * a.dense_stride;
    }
    CUtensorMap tmQ, tmK;
    {
        cuuint64_t dims[3] = {(cuuint64_t)HD, (cuuint64_t)a.num_heads, (cuuint64_t)a.total_q};
        cuuint64_t strides[2] = {(cuuint64_t)HD * 2, (cuuint64_t)a.num_heads * HD * 2};
        cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)TT};
        if (!encode_map(&tmQ, a.q, a.dtype, dims, strides, box, err)) return cudaErrorInvalidValue;
    }
    {
        cuuint64_t dims[3] = {64, (cuuint64_t)a.num_kv_heads * (HD / 64), (cuuint64_t)k_rows};
        cuuint64_t strides[2] = {128, (cuuint64_t)a.num_kv_heads * HD * 2};
        cuuint32_t box[3] = {64, 1, (cuuint32_t)(!a.dense_stride && a.block_size == 8 ? 8 : GRP)};
        if (!encode_map(&tmK, a.k_cache, a.dtype, dims, strides, box, err)) return cudaErrorInvalidValue;
    }
    const size_t smem = weights_smem<HD>(a.num_seqs);
    const dim3 block(WGeo<HD>::NTHREADS);
    auto k1 = weights_umma_kernel<T, HD, kRowStats, SC>;
    auto k2 = a.few_rows ? weights_umma_kernel<T, HD, kFewRows, SC> : weights_umma_kernel<T, HD, kKeyWeights, SC>;
    constexpr int kMost = kWeightMaxSeqsPerLaunch;
    e = allow_smem(reinterpret_cast<const void*>(k1), weights_smem<HD>(kMost));
    if (e == cudaSuccess) e = allow_smem(reinterpret_cast<const void*>(k2), weights_smem<HD>(kMost));
    if (e != cudaSuccess) return e;
    constexpr int NA = WGeo<HD>::NA;
    const int64_t rows = a.window > 0 ? std::min<int64_t>(a.total_q, (int64_t)a.num_seqs * a.window) : a.total_q;
    const int64_t q_items = (rows / (NA * TT) + a.num_seqs) * a.num_kv_heads;
    const int64_t k_items = a.few_rows ? (int64_t)a.num_seqs * a.num_kv_heads
                                       : (int64_t)a.num_seqs * a.num_kv_heads * ((a.max_context + NA * TM - 1) / (NA * TM));
    // one CTA fits an SM, and draws its share of the items
    auto ctas = [&](int64_t n) { return (unsigned)std::max<int64_t>(1, std::min<int64_t>(n, sms)); };
    e = launch_pdl_smem(k1, dim3(ctas(q_items * a.key_splits)), block, smem, stream, tmQ, tmK, a);
    if (e != cudaSuccess) return e;
    if (a.key_splits > 1) {
        const int64_t tiles = (rows / TT + a.num_seqs) * a.num_kv_heads;
        e = launch_pdl_smem(stats_join_kernel, dim3((unsigned)std::min<int64_t>(tiles, sms * 8)), dim3(TM),
                            (size_t)(a.num_seqs + 1) * sizeof(int32_t), stream, a);
        if (e != cudaSuccess) return e;
    }
    e = launch_pdl_smem(k2, dim3(ctas(k_items * a.row_splits)), block, smem, stream, tmQ, tmK, a);
    if (e != cudaSuccess || a.few_rows || a.row_splits == 1) return e;
    const int64_t wrows = (int64_t)a.num_seqs * a.num_kv_heads;
    return launch_pdl(weights_join_kernel,
                      dim3((unsigned)((a.max_context + 255) / 256), (unsigned)std::min<int64_t>(wrows, 65535)), dim3(256),
                      stream, a);
}

template <typename T, bool SC>
cudaError_t launch_hd(const WeightArgs& a, int32_t num_blocks, std::string* err, cudaStream_t stream) {
    return a.head_dim == 64    ? launch_umma<T, 64, SC>(a, num_blocks, err, stream)
           : a.head_dim == 128 ? launch_umma<T, 128, SC>(a, num_blocks, err, stream)
                               : launch_umma<T, 256, SC>(a, num_blocks, err, stream);
}

}  // namespace

bool weights_umma_supported(int dtype, int head_dim, int group) {
    return (dtype == 1 || dtype == 2) && (head_dim == 64 || head_dim == 128 || head_dim == 256) && group >= 1 &&
           group <= TM;
}

// How the work is cut: pieces of the streamed axis, where there are few
// stationary tiles.  Pieces of fewer than 16 tiles spend much of their time
// starting (2,048-token prompt: 1.2 x the time with pieces of 4 or more).
// Items of unequal length (causal tiles) are cut so that there are two per SM
// for the scheduling to even out (8,192 tokens: 1 % slower with four per SM,
// 12 % with eight); few rows over long contexts are equal pieces, as many as
// make three whole rounds over the SMs.
WeightPlan weights_umma_plan(int32_t num_seqs, int32_t total_q, int32_t max_q, int32_t num_heads,
                             int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t max_context,
                             int32_t window, bool kv_fp8) {
    constexpr int64_t kMinTiles = 16;
    const int G = num_heads / num_kv_heads, TT = TM / G, NA = head_dim <= 128 ? 2 : 1;
    auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    auto round = [](size_t b) { return (b + 255) / 256 * 256; };
    WeightPlan w;
    const int32_t row_max = window > 0 ? std::min(max_q, window) : max_q;  // of one request
    const int64_t k_tiles = up(max_context, TM), q_tiles = up(row_max, TT);
    // pools that no box fits, and code pools, are laid out densely first, of as
    // many requests at a time as the scratch space takes
    const bool dense = kv_fp8 || !(block_size == 8 || (block_size % GRP == 0 && block_size <= 256));
    const int64_t stride = k_tiles * TM, key_bytes = (int64_t)num_kv_heads * head_dim * 2;
    const int64_t scale_bytes = kv_fp8 ? num_kv_heads * (int64_t)sizeof(float) : 0;
    w.seqs = seqs_per_launch(num_seqs, dense ? (double)stride * (key_bytes + scale_bytes) : 0, kWeightMaxSeqsPerLaunch);
    if (dense) {
        // (several requests' tokens fit in int32 because their bytes fit in
        // the scratch space, at 128 each or more)
        w.dense_stride = stride <= (1 << 29) ? (int)stride : -1;  // (refused)
        w.dense_bytes = (size_t)w.seqs * stride * key_bytes;
        w.scale_bytes = (size_t)w.seqs * stride * scale_bytes;
    }
    const int64_t rows = window > 0 ? std::min<int64_t>(total_q, (int64_t)w.seqs * window) : total_q;
    w.few_rows = q_tiles <= NA;
    auto pieces = [&](int64_t items, int64_t tiles, int64_t most) {
        const int64_t want = w.few_rows ? 3 * kSms / items : up(2 * kSms, items);
        return (int)std::max<int64_t>(1, std::min({want, tiles / kMinTiles, most}));
    };
    const int64_t units = (int64_t)w.seqs * num_kv_heads;
    w.key_splits = pieces(w.few_rows ? units : std::max<int64_t>(1, up(rows, NA * TT)) * num_kv_heads, k_tiles, 64);
    w.row_splits = w.few_rows ? pieces(units, k_tiles, 256) : pieces(units * up(k_tiles, NA), q_tiles, 8);
    // partial statistics (several key splits), and the statistics by query
    // tile that pass 2 reads
    const int64_t stat_rows = weight_stat_rows(w.seqs, total_q, window).rows;
    if (w.key_splits > 1) w.stats_bytes = round((size_t)w.key_splits * stat_rows * num_heads * sizeof(float2));
    w.stat_tiles = (int)(stat_rows / TT) + w.seqs + 1;
    w.tile_stats_bytes = (size_t)w.stat_tiles * num_kv_heads * 2 * TM * sizeof(float);
    if (!w.few_rows && w.row_splits > 1)
        w.partial_bytes = (size_t)w.row_splits * units * max_context * sizeof(float);
    return w;
}

cudaError_t launch_weights_umma(const WeightArgs& a, int32_t num_blocks, std::string* err, cudaStream_t stream) {
    if (a.dtype == 1)
        return a.kv_fp8 ? launch_hd<__nv_bfloat16, true>(a, num_blocks, err, stream)
                        : launch_hd<__nv_bfloat16, false>(a, num_blocks, err, stream);
    return a.kv_fp8 ? launch_hd<__half, true>(a, num_blocks, err, stream)
                    : launch_hd<__half, false>(a, num_blocks, err, stream);
}

uint32_t weights_umma_status(bool clear) {
    unsigned int v = 0;
    cudaMemcpyFromSymbol(&v, g_weights_status, sizeof(v));
    if (clear) {
        const unsigned int z = 0;
        cudaMemcpyToSymbol(g_weights_status, &z, sizeof(z));
    }
    return v;
}

}  // namespace pa
