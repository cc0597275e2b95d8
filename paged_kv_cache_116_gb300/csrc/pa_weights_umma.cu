// pa_weights_umma.cu -- attention weights of a request's cached tokens on the
// 5th-generation tensor cores (tcgen05.mma, accumulators in tensor memory):
// bf16/f16, head_dim 64, 128 or 256, block_size 8 or a multiple of 16 up to
// 256.  The definition stands at the head of pa_weights_simt.cu; the two
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
// In both the reduction runs along the columns of the accumulator, that is
// within one thread's tensor-memory lane: no shuffle, no atomics, a fixed
// order.  A query tile is T = floor(128 / G) consecutive new tokens with the G
// query heads of a KV head (row t G + g).
//
// Where there are few query tiles (a short window over long contexts) pass 1
// is split over the keys, gridDim.y pieces whose (maximum, sum) pass 2 joins
// as it reads them.
//
// Roles (192 threads): warps 0-3 work the accumulator tiles (one row or key
// per thread), warp 4 loads tiles by TMA (128-byte swizzle; keys through the
// block table, one 16-token group per box), one lane of warp 5 issues the
// MMAs.  Two 128-column accumulators alternate, so the MMAs of the next tile
// run under the exponentials of this one; at head_dim up to 128 two CTAs share
// an SM, which hides each other's start and end.  Every wait is bounded; on
// expiry the CTA sets a status bit, abandons its work, waits (bounded) for
// its loads in flight and frees its tensor memory.
//
// Bound: the exponentials.  A 128 x 128 tile is 16,384 of them, 1,024 cycles
// of an SM's 16 per cycle, against 512 cycles or so of MMA at head_dim 128;
// both passes take every exponential.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <mutex>
#include <string>
#include <type_traits>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_launch.cuh"
#include "pa_weights.cuh"

namespace pa {
namespace {

__device__ unsigned int g_weights_status;

constexpr int TM = 128;                       // rows of A (query rows or keys) and columns of B
constexpr int GRP = 16;                       // keys per TMA box (two boxes of 8 with 8-token blocks)
constexpr int NGRP = TM / GRP;
constexpr int W_PROD = 4, W_MMA = 5, NTHREADS = 192;
constexpr uint32_t TMEM_COLS = 2 * TM;        // two accumulators
constexpr uint64_t WAIT_NS = 2000000000ull;   // 2 s
constexpr int RING = 2;                       // streamed tiles in flight
constexpr int kMaxCtas = 1 << 14;             // beyond this a CTA takes several items

template <int HD>
struct WGeo {
    static constexpr int CH = HD / 64;        // 128-byte chunks of a row
    static constexpr int CHB = TM * 128;      // bytes of one chunk of a tile
    static constexpr int TILE = CH * CHB;
    static constexpr int RING_OFF = TILE;     // after the stationary tile
    static constexpr int STAT_OFF = RING_OFF + RING * TILE;  // pass 2: [2][128] -M, [2][128] 1 / l
    static constexpr int BAR_OFF = STAT_OFF + 4 * TM * 4;
    // a_full, a_empty, b_full[RING], b_empty[RING], d_full[2], d_empty[2],
    // s_full[2] (pass 2: a query tile's statistics are in shared memory)
    static constexpr int NBAR = 2 + 2 * RING + 6;
    static constexpr int ADDR_OFF = BAR_OFF + NBAR * 8;
    static constexpr int PREF_OFF = ADDR_OFF + 16;
    static constexpr int MINB = HD <= 128 ? 2 : 1;
};
template <int HD>
size_t weights_smem(int num_seqs) { return 1024 + WGeo<HD>::PREF_OFF + (size_t)(num_seqs + 1) * 4; }

// One work item, as every role sees it.
struct Item {
    WeightSeq sq;
    int h;
    int a_row;   // pass 1: first new token (within the counted ones) of the query tile; pass 2: first key
    int b0, b1;  // streamed tiles
};

// PASS 1 or 2; T: the element type of q and the pool.
template <typename T, int HD, int PASS>
__global__ void __launch_bounds__(NTHREADS, WGeo<HD>::MINB)
    weights_umma_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const WeightArgs p, const int splits) {
    using Gm = WGeo<HD>;
    constexpr bool kBF16 = std::is_same<T, __nv_bfloat16>::value;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(base + Gm::BAR_OFF);
    uint64_t* a_full = bars;
    uint64_t* a_empty = bars + 1;
    uint64_t* b_full = bars + 2;
    uint64_t* b_empty = b_full + RING;
    uint64_t* d_full = b_empty + RING;
    uint64_t* d_empty = d_full + 2;
    uint64_t* s_full = d_empty + 2;
    float* neg_m = reinterpret_cast<float*>(base + Gm::STAT_OFF);  // [2][TM]
    float* inv_l = neg_m + 2 * TM;                                 // [2][TM]
    volatile uint32_t* taddr_slot = reinterpret_cast<volatile uint32_t*>(base + Gm::ADDR_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(base + Gm::ADDR_OFF + 4);
    int32_t* prefix = reinterpret_cast<int32_t*>(base + Gm::PREF_OFF);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = p.num_heads / p.num_kv_heads, Hkv = p.num_kv_heads, TT = TM / G;

    if (threadIdx.x == 32 * W_PROD) {
        prefetch_tmap(&tmQ);
        prefetch_tmap(&tmK);
    }
    if (threadIdx.x == 0) {
        // d_empty: one arrival per accumulator warp, s_full: one per thread of them
        for (int i = 0; i < Gm::NBAR; ++i) mbar_init(&bars[i], i >= Gm::NBAR - 2 ? 128u : i >= Gm::NBAR - 4 ? 4u : 1u);
        *abort_flag = 0;
        mbar_fence_init();
    }
    // tensor memory is taken after the previous grid is done: its CTAs may
    // still be waiting for theirs on this SM
    pdl_wait_primary();
    pdl_launch_dependents();
    work_prefix(p, prefix, [&](const WeightSeq& sq) {
        if (PASS == 1) return (sq.rows + TT - 1) / TT;
        return sq.rows ? (sq.L + TM - 1) / TM : 0;
    });
    const int64_t items = (int64_t)prefix[p.num_seqs] * Hkv;
    if (blockIdx.x >= items) return;  // uniform for the CTA
    if (warp == W_MMA) {
        tmem_alloc(const_cast<uint32_t*>(taddr_slot), TMEM_COLS);
        tmem_relinquish();
    }
    if (PASS == 2 && TT * G < TM) {
        // rows of a streamed query tile past its T G (token, head) pairs get
        // no TMA data: zeros, so that their columns are finite and weigh 0
        const int pad = TM - TT * G, per = Gm::CH * pad * 8;
        for (int e = threadIdx.x; e < RING * per; e += NTHREADS) {
            const int slot = e / per, r0 = e - slot * per, c = r0 / (pad * 8), r = r0 - c * pad * 8;
            *reinterpret_cast<uint4*>(base + Gm::RING_OFF + slot * Gm::TILE + c * Gm::CHB + (TT * G + r / 8) * 128 +
                                      (r & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *taddr_slot;

    auto item_at = [&](int64_t it) -> Item {
        Item w;
        int s, tile;
        locate_work(prefix, p.num_seqs, Hkv, it, s, w.h, tile);
        w.sq = weight_seq(p, s);
        if (PASS == 1) {
            // late tiles see the most keys under a causal mask: they go first
            tile = (w.sq.rows + TT - 1) / TT - 1 - tile;
            w.a_row = tile * TT;
            const int last = min(w.sq.rows, w.a_row + TT);
            const int seen = p.causal ? w.sq.L - w.sq.rows + last : w.sq.L;
            const int n = (max(seen, 0) + TM - 1) / TM;
            w.b0 = (int)((int64_t)n * blockIdx.y / splits);
            w.b1 = (int)((int64_t)n * (blockIdx.y + 1) / splits);
        } else {
            w.a_row = tile * TM;
            w.b0 = p.causal ? max(0, w.a_row - (w.sq.L - w.sq.rows)) / TT : 0;
            w.b1 = (w.sq.rows + TT - 1) / TT;
        }
        return w;
    };
    auto fail = [&]() {
        *abort_flag = 1;
        atomicOr(&g_weights_status, kStatusTimeout);
    };

    if (warp == W_PROD) {
        // ---------------- producer
        const uint64_t pol = l2_policy_evict_last();  // keys are read twice, query tiles by every key tile
        const int bsz = p.block_size, halves = bsz == 8 ? 2 : 1;
        const int rows_per = TM / GRP * halves;  // boxes along the keys of a tile
        int na = 0, nb = 0;
        bool run = true;
        // pool row of box `lane` of key tile kt (the last valid one where the
        // second half of a group holds no context; never read past it)
        auto key_row = [&](const Item& w, int kt) -> int32_t {
            if (lane >= rows_per) return 0;
            const int32_t* table = p.block_tables + (int64_t)w.sq.s * p.max_blocks;
            int tok = kt * TM + lane * (GRP / halves);
            if (halves == 2 && (lane & 1) && tok >= w.sq.L) tok -= 8;
            if (tok >= w.sq.L) return 0;
            return table[tok / bsz] * bsz + tok % bsz;
        };
        auto load_keys = [&](const Item& w, int kt, int32_t row, uint8_t* dst, uint64_t* bar) {
            const int groups = min(NGRP, (w.sq.L - kt * TM + GRP - 1) / GRP);
            if (lane == 0) {
                fence_proxy_async_smem();
                mbar_arrive_expect_tx(bar, (uint32_t)(groups * GRP * 128 * Gm::CH));
            }
            __syncwarp();
            const int boxes = groups * halves * Gm::CH;
            for (int e0 = 0; e0 < boxes; e0 += 32) {
                const int e = e0 + lane, b = e / Gm::CH, c = e - b * Gm::CH;  // box along the keys, chunk
                const int32_t r = __shfl_sync(0xffffffffu, row, min(b, 31));
                if (e < boxes)
                    tma_load_3d(dst + c * Gm::CHB + b * (GRP / halves) * 128, &tmK, bar, 0, w.h * Gm::CH + c, r, pol);
            }
        };
        auto load_queries = [&](const Item& w, int row, uint8_t* dst, uint64_t* bar) {
            if (lane == 0) {
                fence_proxy_async_smem();
                mbar_arrive_expect_tx(bar, (uint32_t)(Gm::CH * 128 * G * TT));
            }
            __syncwarp();
            if (lane < Gm::CH) tma_load_3d(dst + lane * Gm::CHB, &tmQ, bar, 64 * lane, w.h * G, w.sq.row0 + row, pol);
        };
        auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
            int ok = 0;
            if (lane == 0) {
                ok = mbar_wait_ns(bar, parity, WAIT_NS) && !*abort_flag;
                if (!ok) fail();
            }
            return __shfl_sync(0xffffffffu, ok, 0) != 0;
        };
        for (int64_t it = blockIdx.x; it < items && run; it += gridDim.x) {
            const Item w = item_at(it);
            if (w.b0 >= w.b1) continue;
            int32_t row = key_row(w, PASS == 1 ? w.b0 : w.a_row / TM);
            if (!(run = wait(a_empty, (uint32_t)(na & 1) ^ 1u))) break;
            if (PASS == 1) load_queries(w, w.a_row, base, a_full);
            else load_keys(w, w.a_row / TM, row, base, a_full);
            ++na;
            for (int t = w.b0; t < w.b1; ++t, ++nb) {
                const int slot = nb % RING;
                uint8_t* dst = base + Gm::RING_OFF + slot * Gm::TILE;
                if (!(run = wait(&b_empty[slot], (uint32_t)(nb / RING & 1) ^ 1u))) break;
                if (PASS == 1) {
                    load_keys(w, t, row, dst, &b_full[slot]);
                    if (t + 1 < w.b1) row = key_row(w, t + 1);
                } else {
                    load_queries(w, t * TT, dst, &b_full[slot]);
                }
            }
        }
        if (!run) {  // copies in flight land before the CTA's shared memory is given up
            if (na) mbar_wait_ns(a_full, (uint32_t)(na - 1) & 1u, WAIT_NS);
            for (int j = max(0, nb - RING); j < nb; ++j)
                mbar_wait_ns(&b_full[j % RING], (uint32_t)(j / RING) & 1u, WAIT_NS);
        }
    } else if (warp == W_MMA) {
        // ---------------- MMA issuer
        if (lane == 0) {
            const uint32_t idesc = umma_idesc_f16(TM, TM, kBF16, false);
            const uint32_t a_s = smem_u32(base);
            int na = 0, nb = 0;
            bool run = true;
            for (int64_t it = blockIdx.x; it < items && run; it += gridDim.x) {
                const Item w = item_at(it);
                if (w.b0 >= w.b1) continue;
                if (!(run = mbar_wait_ns(a_full, (uint32_t)na & 1u, WAIT_NS) && !*abort_flag)) break;
                ++na;
                for (int t = w.b0; t < w.b1; ++t, ++nb) {
                    const int slot = nb % RING, buf = nb & 1;
                    run = mbar_wait_ns(&d_empty[buf], ((uint32_t)(nb >> 1) & 1u) ^ 1u, WAIT_NS) &&
                          mbar_wait_ns(&b_full[slot], (uint32_t)(nb / RING) & 1u, WAIT_NS) && !*abort_flag;
                    if (!run) break;
                    tc_fence_after();
                    const uint32_t b_s = a_s + Gm::RING_OFF + slot * Gm::TILE;
#pragma unroll
                    for (int kk = 0; kk < HD / 16; ++kk) {
                        const int c = kk >> 2, ko = (kk & 3) * 32;
                        umma_f16(tmem + buf * TM, umma_sdesc_sw128(a_s + c * Gm::CHB + ko, 16, 1024),
                                 umma_sdesc_sw128(b_s + c * Gm::CHB + ko, 16, 1024), idesc, kk > 0 ? 1u : 0u);
                    }
                    umma_commit(&b_empty[slot]);
                    if (t == w.b1 - 1) umma_commit(a_empty);
                    umma_commit(&d_full[buf]);
                }
            }
            if (!run) {
                fail();
                if (nb) mbar_wait_ns(&d_full[(nb - 1) & 1], (uint32_t)((nb - 1) >> 1) & 1u, WAIT_NS);  // MMAs in flight
            }
        }
    } else {
        // ---------------- accumulator tiles: one row (pass 1) or key (pass 2) per thread
        const int m = threadIdx.x;
        const uint32_t t_lane = tmem + ((uint32_t)(warp * 32) << 16);
        const float sl = p.scale_log2;
        const int64_t part = (int64_t)p.total_q * p.num_heads;  // rows of one split's statistics
        int nb = 0;
        bool run = true;
        auto release = [&](int buf) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&d_empty[buf]);
        };
        auto acquire = [&](int buf) -> bool {
            const bool ok = !*abort_flag && mbar_wait_ns(&d_full[buf], (uint32_t)(nb >> 1) & 1u, WAIT_NS);
            tc_fence_after();
            return ok;
        };
        for (int64_t it = blockIdx.x; it < items && run; it += gridDim.x) {
            const Item w = item_at(it);
            if constexpr (PASS == 1) {
                const int tok = w.a_row + m / G, g = m % G;
                const bool valid = m < TT * G && tok < w.sq.rows;
                const int last = p.causal ? w.sq.L - w.sq.rows + tok : w.sq.L - 1;  // last key the row sees
                float m_used = -INFINITY, l = 0.f;
                for (int t = w.b0; t < w.b1; ++t, ++nb) {
                    const int buf = nb & 1;
                    if (!(run = acquire(buf))) break;
                    const uint32_t d = t_lane + buf * TM;
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
#pragma unroll
                        for (int q = 0; q < TM / 32; ++q) {
                            float a[32];
                            tmem_ld32(d + 32 * q, a);
                            tmem_wait_ld();
                            if (full) {
#pragma unroll
                                for (int j = 0; j < 16; ++j) {
                                    float x0, x1;
                                    f32x2_unpack(fma_f32x2(f32x2_pack(a[2 * j], a[2 * j + 1]), sv, nv), x0, x1);
                                    s2 = add_f32x2(s2, f32x2_pack(fast_exp2(x0), fast_exp2(x1)));
                                }
                            } else {
#pragma unroll
                                for (int j = 0; j < 32; ++j)
                                    sum += 32 * q + j <= vis ? fast_exp2(fmaf(a[j], sl, neg)) : 0.f;
                            }
                        }
                        float s0, s1;
                        f32x2_unpack(s2, s0, s1);
                        sum += s0 + s1;
                    };
                    auto max_pass = [&]() -> float {
                        float mt = -INFINITY;
#pragma unroll
                        for (int q = 0; q < TM / 32; ++q) {
                            float a[32];
                            tmem_ld32(d + 32 * q, a);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (32 * q + j <= vis) mt = fmaxf(mt, a[j] * sl);
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
                    release(buf);
                }
                if (run && valid)
                    p.stats[(int64_t)blockIdx.y * part + (int64_t)(w.sq.row0 + tok) * p.num_heads + w.h * G + g] =
                        make_float2(m_used, l);
            } else {
                const int key = w.a_row + m;
                // statistics of query tile t's row m, joined over the splits
                auto row_stat = [&](int t) -> float2 {
                    const int tok = t * TT + m / G;
                    if (m >= TT * G || tok >= w.sq.rows) return make_float2(0.f, 0.f);
                    const float2* st = p.stats + (int64_t)(w.sq.row0 + tok) * p.num_heads + w.h * G + m % G;
                    float2 s = __ldcg(st);
                    for (int z = 1; z < splits; ++z) {
                        const float2 o = __ldcg(st + z * part);
                        const float mn = fmaxf(s.x, o.x);
                        if (mn == -INFINITY) {  // no key, or none with a number for a score
                            s.y += o.y;
                            continue;
                        }
                        s.y = s.y * exp2f(s.x - mn) + o.y * exp2f(o.x - mn);
                        s.x = mn;
                    }
                    return make_float2(s.x == -INFINITY ? 0.f : -s.x, 1.f / s.y);
                };
                float total = 0.f;
                float2 st = w.b0 < w.b1 ? row_stat(w.b0) : make_float2(0.f, 0.f);
                for (int t = w.b0; t < w.b1; ++t, ++nb) {
                    const int buf = nb & 1;
                    float* nm = neg_m + buf * TM;
                    float* il = inv_l + buf * TM;
                    nm[m] = st.x;
                    il[m] = st.y;
                    // (a buffer written two tiles ago is free: every thread
                    // has been through the barrier of the tile between)
                    mbar_arrive(&s_full[buf]);
                    if (t + 1 < w.b1) st = row_stat(t + 1);
                    if (!(run = mbar_wait_ns(&s_full[buf], (uint32_t)(nb >> 1) & 1u, WAIT_NS) && acquire(buf))) break;
                    const uint32_t d = t_lane + buf * TM;
                    // columns [c0, c1) are rows of this request that see the key
                    const int c1 = min(TT, w.sq.rows - t * TT) * G;
                    const int c0 = p.causal ? max(0, key - (w.sq.L - w.sq.rows) - t * TT) * G : 0;
                    const bool full = __all_sync(0xffffffffu, c0 == 0 && c1 == TT * G);
                    // summed tile by tile: a running sum over thousands of
                    // rows would round at its own size in every addition
                    unsigned long long acc2 = f32x2_pack(0.f, 0.f);
                    float acc = 0.f;
#pragma unroll
                    for (int q = 0; q < TM / 32; ++q) {
                        float a[32];
                        tmem_ld32(d + 32 * q, a);
                        tmem_wait_ld();
                        if (full) {
                            const unsigned long long sv = f32x2_pack(sl, sl);
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const float4 n4 = *reinterpret_cast<const float4*>(nm + 32 * q + 4 * j);
                                const float4 i4 = *reinterpret_cast<const float4*>(il + 32 * q + 4 * j);
                                float x0, x1, x2, x3;
                                f32x2_unpack(fma_f32x2(f32x2_pack(a[4 * j], a[4 * j + 1]), sv, f32x2_pack(n4.x, n4.y)), x0, x1);
                                f32x2_unpack(fma_f32x2(f32x2_pack(a[4 * j + 2], a[4 * j + 3]), sv, f32x2_pack(n4.z, n4.w)), x2, x3);
                                acc2 = fma_f32x2(f32x2_pack(fast_exp2(x0), fast_exp2(x1)), f32x2_pack(i4.x, i4.y), acc2);
                                acc2 = fma_f32x2(f32x2_pack(fast_exp2(x2), fast_exp2(x3)), f32x2_pack(i4.z, i4.w), acc2);
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < 32; ++j) {
                                const int c = 32 * q + j;
                                if (c >= c0 && c < c1) acc = fmaf(fast_exp2(fmaf(a[j], sl, nm[c])), il[c], acc);
                            }
                        }
                    }
                    release(buf);
                    float s0, s1;
                    f32x2_unpack(acc2, s0, s1);
                    total += acc + (s0 + s1);
                }
                if (run && key < w.sq.L) {
                    float* dst = p.weights + ((int64_t)w.sq.s * Hkv + w.h) * p.weights_stride + key;
                    *dst = key < w.sq.L - w.sq.n ? *dst + total : total;
                }
            }
        }
        if (!run && lane == 0) fail();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == W_MMA) tmem_dealloc(tmem, TMEM_COLS);
}

// ---------------------------------------------------------------- host side

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    return fn;
}

bool encode_map(CUtensorMap* m, const void* ptr, int dtype, const cuuint64_t (&dims)[3], const cuuint64_t (&strides)[2],
                const cuuint32_t (&box)[3], std::string* err) {
    auto fn = encode_fn();
    if (!fn) {
        *err = "cuTensorMapEncodeTiled is not available from the driver";
        return false;
    }
    cuuint32_t estr[3] = {1, 1, 1};
    const CUtensorMapDataType ty = dtype == 1 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    CUresult r = fn(m, ty, 3, const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        *err = "cuTensorMapEncodeTiled failed with CUresult " + std::to_string((int)r);
        return false;
    }
    return true;
}

template <typename T, int HD>
cudaError_t launch_umma(const WeightArgs& a, int32_t num_blocks, int splits, std::string* err, cudaStream_t stream) {
    const int G = a.num_heads / a.num_kv_heads, TT = TM / G;
    CUtensorMap tmQ, tmK;
    {
        cuuint64_t dims[3] = {(cuuint64_t)HD, (cuuint64_t)a.num_heads, (cuuint64_t)a.total_q};
        cuuint64_t strides[2] = {(cuuint64_t)HD * 2, (cuuint64_t)a.num_heads * HD * 2};
        cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)TT};
        if (!encode_map(&tmQ, a.q, a.dtype, dims, strides, box, err)) return cudaErrorInvalidValue;
    }
    {
        cuuint64_t dims[3] = {64, (cuuint64_t)a.num_kv_heads * (HD / 64), (cuuint64_t)num_blocks * a.block_size};
        cuuint64_t strides[2] = {128, (cuuint64_t)a.num_kv_heads * HD * 2};
        cuuint32_t box[3] = {64, 1, (cuuint32_t)(a.block_size == 8 ? 8 : GRP)};
        if (!encode_map(&tmK, a.k_cache, a.dtype, dims, strides, box, err)) return cudaErrorInvalidValue;
    }
    const size_t smem = weights_smem<HD>(a.num_seqs);
    auto k1 = weights_umma_kernel<T, HD, 1>;
    auto k2 = weights_umma_kernel<T, HD, 2>;
    cudaError_t e = cudaFuncSetAttribute(k1, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k2, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int64_t rows = a.window > 0 ? std::min<int64_t>(a.total_q, (int64_t)a.num_seqs * a.window) : a.total_q;
    const int64_t q_items = (rows / TT + a.num_seqs) * a.num_kv_heads;
    const int64_t k_items = (int64_t)a.num_seqs * a.num_kv_heads * ((a.max_context + TM - 1) / TM);
    auto ctas = [](int64_t n) { return (unsigned)std::max<int64_t>(1, std::min<int64_t>(n, kMaxCtas)); };
    e = launch_pdl_smem(k1, dim3(ctas(q_items), (unsigned)splits), dim3(NTHREADS), smem, stream, tmQ, tmK, a, splits);
    if (e != cudaSuccess) return e;
    return launch_pdl_smem(k2, dim3(ctas(k_items)), dim3(NTHREADS), smem, stream, tmQ, tmK, a, splits);
}

}  // namespace

bool weights_umma_supported(int dtype, int head_dim, int block_size, int group, bool kv_fp8) {
    return !kv_fp8 && (dtype == 1 || dtype == 2) && (head_dim == 64 || head_dim == 128 || head_dim == 256) &&
           (block_size == 8 || (block_size % GRP == 0 && block_size <= 256)) && group >= 1 && group <= TM;
}

// Pieces of the key axis in pass 1: as many as give every SM two CTAs when
// there are few query tiles, each at least four key tiles long.
int weights_umma_splits(int32_t num_seqs, int32_t total_q, int32_t num_kv_heads, int32_t group, int32_t max_context,
                        int32_t window) {
    const int TT = TM / group;
    const int64_t rows = window > 0 ? std::min<int64_t>(total_q, (int64_t)num_seqs * window) : total_q;
    const int64_t items = std::max<int64_t>(1, (rows + TT - 1) / TT) * num_kv_heads;
    const int64_t want = (2 * 152 + items - 1) / items, most = (max_context + 4 * TM - 1) / (4 * TM);
    return (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(want, most), 32));
}

cudaError_t launch_weights_umma(const WeightArgs& a, int32_t num_blocks, int splits, std::string* err,
                                cudaStream_t stream) {
    if (a.dtype == 1)
        return a.head_dim == 64    ? launch_umma<__nv_bfloat16, 64>(a, num_blocks, splits, err, stream)
               : a.head_dim == 128 ? launch_umma<__nv_bfloat16, 128>(a, num_blocks, splits, err, stream)
                                   : launch_umma<__nv_bfloat16, 256>(a, num_blocks, splits, err, stream);
    return a.head_dim == 64    ? launch_umma<__half, 64>(a, num_blocks, splits, err, stream)
           : a.head_dim == 128 ? launch_umma<__half, 128>(a, num_blocks, splits, err, stream)
                               : launch_umma<__half, 256>(a, num_blocks, splits, err, stream);
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
