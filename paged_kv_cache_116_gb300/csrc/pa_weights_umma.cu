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
// tile feeds two MMAs.  With one (and two CTAs per SM) the streamed tiles
// crossed from L2 at 9.3 TB/s, which bounded the kernel (8,192-token prompt,
// 32 / 8 heads: 0.93 ms).
//
// Where there are few stationary tiles the streamed axis is split over
// gridDim.y: in pass 1 pass 2 joins the pieces' (maximum, sum) as it reads
// them, in pass 2 the pieces' partial weights are added by a third kernel.
//
// Roles: per (stationary tile x, parity of the streamed tile) a group of four
// warps that works the accumulator tile, one row or key per thread; then one
// warp that loads tiles by TMA (128-byte swizzle; keys through the block
// table, one 16-token group per box) and one whose first lane issues the MMAs.
// Every group has its own 128-column accumulator, so MMAs run under the other
// groups' exponentials.  Every wait is bounded; on expiry the CTA sets a status
// bit, abandons its work, waits (bounded) for its loads in flight and frees
// its tensor memory.
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

constexpr int TM = 128;                       // rows of A and columns of B
constexpr int GRP = 16;                       // keys per TMA box (two boxes of 8 with 8-token blocks)
constexpr int NGRP = TM / GRP;
constexpr uint64_t WAIT_NS = 2000000000ull;   // 2 s
constexpr int kMaxCtas = 1 << 14;             // beyond this a CTA takes several items

template <int HD>
struct WGeo {
    static constexpr int NA = HD <= 128 ? 2 : 1;    // stationary tiles
    static constexpr int RING = HD == 64 ? 6 : HD == 128 ? 4 : 2;  // streamed tiles in flight
    static constexpr int NWG = 2 * NA;              // accumulators and their warp groups
    static constexpr int W_PROD = 4 * NWG, W_MMA = W_PROD + 1, NTHREADS = 32 * (W_MMA + 1);
    static constexpr uint32_t TMEM_COLS = NWG * TM;
    static constexpr int CH = HD / 64;        // 128-byte chunks of a row
    static constexpr int CHB = TM * 128;      // bytes of one chunk of a tile
    static constexpr int TILE = CH * CHB;
    static constexpr int RING_OFF = NA * TILE;
    // per group two buffers of -M[128] and 1 / l[128]
    static constexpr int STAT_OFF = RING_OFF + RING * TILE;
    static constexpr int JOIN_OFF = STAT_OFF + NWG * 4 * TM * 4;  // results handed over, float2[2][128]
    static constexpr int BAR_OFF = JOIN_OFF + 2 * TM * 8;
    // a_full, a_empty, b_full[RING], b_empty[RING], d_full[NWG],
    // d_empty[NWG], s_full[NWG] (statistics are in shared memory), j_full[2],
    // j_empty[2] (results handed over)
    static constexpr int NBAR = 2 + 2 * RING + 3 * NWG + 4;
    static constexpr int ADDR_OFF = BAR_OFF + NBAR * 8;
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
};

enum Pass { kRowStats = 1, kKeyWeights = 2, kFewRows = 3 };

// T: the element type of q and the pool.
template <typename T, int HD, int PASS>
__global__ void __launch_bounds__(WGeo<HD>::NTHREADS, 1)
    weights_umma_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const WeightArgs p) {
    using Gm = WGeo<HD>;
    constexpr int NA = Gm::NA, RING = Gm::RING;
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
    uint64_t* d_empty = d_full + Gm::NWG;
    uint64_t* s_full = d_empty + Gm::NWG;
    uint64_t* j_full = s_full + Gm::NWG;
    uint64_t* j_empty = j_full + 2;
    float* stat_s = reinterpret_cast<float*>(base + Gm::STAT_OFF);  // [NWG][2][2][TM]
    float2* join_s = reinterpret_cast<float2*>(base + Gm::JOIN_OFF);
    volatile uint32_t* taddr_slot = reinterpret_cast<volatile uint32_t*>(base + Gm::ADDR_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(base + Gm::ADDR_OFF + 4);
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
            // d_empty: one arrival per warp of a group; s_full and j_*: one per thread of it
            mbar_init(bars + i, b >= s_full ? 128u : b >= d_empty ? 4u : 1u);
        }
        *abort_flag = 0;
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
    const int64_t items = (int64_t)prefix[p.num_seqs] * Hkv;
    if (blockIdx.x >= items) return;  // uniform for the CTA
    if (warp == Gm::W_MMA) {
        tmem_alloc(const_cast<uint32_t*>(taddr_slot), Gm::TMEM_COLS);
        tmem_relinquish();
    }
    if (PASS != kRowStats && TT * G < TM) {
        // rows of a query tile past its T G (token, head) pairs get no TMA
        // data: zeros, so that their columns are finite and weigh 0
        const int pad = TM - TT * G, per = Gm::CH * pad * 8;
        const int first = PASS == kFewRows ? 0 : NA, count = PASS == kFewRows ? NA : RING;
        for (int e = threadIdx.x; e < count * per; e += Gm::NTHREADS) {
            const int tile = first + e / per, r0 = e % per, c = r0 / (pad * 8), r = r0 - c * pad * 8;
            *reinterpret_cast<uint4*>(base + tile * Gm::TILE + c * Gm::CHB + (TT * G + r / 8) * 128 + (r & 7) * 16) =
                make_uint4(0, 0, 0, 0);
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
        w.b1 = w.b0 + (int)((int64_t)n * (blockIdx.y + 1) / gridDim.y);
        w.b0 += (int)((int64_t)n * blockIdx.y / gridDim.y);
        return w;
    };
    auto fail = [&]() {
        *abort_flag = 1;
        atomicOr(&g_weights_status, kStatusTimeout);
    };

    if (warp == Gm::W_PROD) {
        // ---------------- producer
        const uint64_t pol = l2_policy_evict_last();  // keys are read twice, query tiles by every key tile
        const int bsz = p.block_size, halves = bsz == 8 ? 2 : 1;
        const int nbox = NGRP * halves;  // boxes along the keys of a tile
        int na = 0, nb = 0;
        bool run = true;
        // pool row of box `lane` of key tile kt (where the second half of a
        // group holds no context, the first half's; never read past it)
        auto key_row = [&](const Item& w, int kt) -> int32_t {
            if (lane >= nbox) return 0;
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
                ok = mbar_wait_ns(bar, parity, WAIT_NS) && !*abort_flag;
                if (!ok) fail();
            }
            return __shfl_sync(0xffffffffu, ok, 0) != 0;
        };
        for (int64_t it = blockIdx.x; it < items && run; it += gridDim.x) {
            const Item w = item_at(it);
            if (w.b0 >= w.b1) continue;
            int32_t row = kKeysStream ? key_row(w, w.b0) : 0;
            if (!(run = wait(a_empty, (uint32_t)(na & 1) ^ 1u))) break;
            if (kKeysStream) {
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
                const int slot = nb % RING;
                uint8_t* dst = base + Gm::RING_OFF + slot * Gm::TILE;
                if (!(run = wait(&b_empty[slot], (uint32_t)(nb / RING & 1) ^ 1u))) break;
                if (kKeysStream) {
                    expect(&b_full[slot], key_groups(w, t) * group_bytes);
                    load_keys(w, t, row, dst, &b_full[slot]);
                    if (t + 1 < w.b1) row = key_row(w, t + 1);
                } else {
                    expect(&b_full[slot], query_bytes);
                    load_queries(w, t, dst, &b_full[slot]);
                }
            }
        }
        if (!run) {  // copies in flight land before the CTA's shared memory is given up
            if (na) mbar_wait_ns(a_full, (uint32_t)(na - 1) & 1u, WAIT_NS);
            for (int j = max(0, nb - RING); j < nb; ++j)
                mbar_wait_ns(&b_full[j % RING], (uint32_t)(j / RING) & 1u, WAIT_NS);
        }
    } else if (warp == Gm::W_MMA) {
        // ---------------- MMA issuer
        if (lane == 0) {
            const uint32_t idesc = umma_idesc_f16(TM, TM, kBF16, false);
            const uint32_t s_base = smem_u32(base);
            int na = 0, nb = 0, nx[2] = {0, 0}, last = -1;
            bool run = true;
            for (int64_t it = blockIdx.x; it < items && run; it += gridDim.x) {
                const Item w = item_at(it);
                if (w.b0 >= w.b1) continue;
                if (!(run = mbar_wait_ns(a_full, (uint32_t)na & 1u, WAIT_NS) && !*abort_flag)) break;
                ++na;
                for (int t = w.b0; t < w.b1 && run; ++t, ++nb) {
                    const int slot = nb % RING;
                    run = mbar_wait_ns(&b_full[slot], (uint32_t)(nb / RING) & 1u, WAIT_NS);
                    const uint32_t b_s = s_base + Gm::RING_OFF + slot * Gm::TILE;
#pragma unroll
                    for (int x = 0; x < NA; ++x) {
                        if (x >= w.na || !run) break;
                        const int d = 2 * x + (nx[x] & 1);
                        run = mbar_wait_ns(&d_empty[d], ((uint32_t)(nx[x] >> 1) & 1u) ^ 1u, WAIT_NS) && !*abort_flag;
                        if (!run) break;
                        ++nx[x];
                        tc_fence_after();
                        const uint32_t a_s = s_base + x * Gm::TILE;
                        // the accumulator's lanes are query rows, or keys
                        const uint32_t l_s = PASS == kFewRows ? b_s : a_s, c_s = PASS == kFewRows ? a_s : b_s;
#pragma unroll
                        for (int kk = 0; kk < HD / 16; ++kk) {
                            const int c = kk >> 2, ko = (kk & 3) * 32;
                            umma_f16(tmem + d * TM, umma_sdesc_sw128(l_s + c * Gm::CHB + ko, 16, 1024),
                                     umma_sdesc_sw128(c_s + c * Gm::CHB + ko, 16, 1024), idesc, kk > 0 ? 1u : 0u);
                        }
                        if (x == w.na - 1) {
                            umma_commit(&b_empty[slot]);
                            if (t == w.b1 - 1) umma_commit(a_empty);
                        }
                        umma_commit(&d_full[d]);
                        last = d;
                    }
                }
            }
            if (!run) {
                fail();
                if (last >= 0)  // MMAs in flight
                    mbar_wait_ns(&d_full[last], (uint32_t)((nx[last >> 1] - 1) >> 1) & 1u, WAIT_NS);
            }
        }
    } else {
        // ---------------- accumulator tiles: one row or key per thread
        const int wg = warp >> 2, x = wg >> 1, par = wg & 1, m = threadIdx.x & 127;
        const uint32_t d = tmem + ((uint32_t)((warp & 3) * 32) << 16) + wg * TM;
        const float sl = p.scale_log2;
        const int64_t part = (int64_t)p.total_q * p.num_heads;  // rows of one split's statistics
        int nx = 0, n_stat = 0, n_join = 0;  // streamed tiles of x; this group's statistics and handovers
        bool run = true;
        auto release = [&]() {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&d_empty[wg]);
        };
        auto acquire = [&]() -> bool {
            const bool ok = !*abort_flag && mbar_wait_ns(&d_full[wg], (uint32_t)(nx >> 1) & 1u, WAIT_NS);
            tc_fence_after();
            return ok;
        };
        // a giving group hands its values to the receiving one through buffer j
        auto hand_over = [&](int j, bool give, float2& v) -> bool {
            const uint32_t ph = (uint32_t)n_join++ & 1u;
            if (give) {
                if (*abort_flag || !mbar_wait_ns(&j_empty[j], ph ^ 1u, WAIT_NS)) return false;
                join_s[j * TM + m] = v;
                mbar_arrive(&j_full[j]);
            } else {
                if (*abort_flag || !mbar_wait_ns(&j_full[j], ph, WAIT_NS)) return false;
                v = join_s[j * TM + m];
                mbar_arrive(&j_empty[j]);
            }
            return true;
        };
        // statistics of query tile t's row m, joined over pass 1's splits: (-M, 1 / l)
        auto row_stat = [&](const Item& w, int t) -> float2 {
            const int tok = t * TT + m / G;
            if (m >= TT * G || tok >= w.sq.rows) return make_float2(0.f, 0.f);
            const float2* st = p.stats + (int64_t)(w.sq.row0 + tok) * p.num_heads + w.h * G + m % G;
            float2 s = __ldcg(st);
            for (int z = 1; z < p.key_splits; ++z) {
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
        // this thread's statistics into the group's next buffer; false if the wait ran out
        auto share_stat = [&](float2 st, float*& nm) -> bool {
            const uint32_t ph = (uint32_t)n_stat++ & 1u;
            nm = stat_s + (2 * wg + ph) * 2 * TM;
            nm[m] = st.x;
            nm[TM + m] = st.y;
            // (a buffer written two turns ago is free: every thread has been
            // through the barrier of the turn between)
            mbar_arrive(&s_full[wg]);
            return true;
        };
        auto stat_ready = [&]() -> bool {
            return !*abort_flag && mbar_wait_ns(&s_full[wg], (uint32_t)(n_stat - 1) & 1u, WAIT_NS);
        };
        // sum over the columns [c0, c1) of exp2(x - M) / l for this thread's key
        auto key_sum = [&](const float* nm, int c0, int c1) -> float {
            const float* il = nm + TM;
            const bool full = __all_sync(0xffffffffu, c0 <= 0 && c1 == TT * G);
            // summed tile by tile: a running sum over thousands of rows would
            // round at its own size in every addition
            unsigned long long acc2 = f32x2_pack(0.f, 0.f);
            float acc = 0.f;
            const unsigned long long sv = f32x2_pack(sl, sl);
#pragma unroll
            for (int q = 0; q < TM / 32; ++q) {
                float a[32];
                tmem_ld32(d + 32 * q, a);
                tmem_wait_ld();
                if (full) {
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
            float s0, s1;
            f32x2_unpack(acc2, s0, s1);
            return acc + (s0 + s1);
        };
        auto store_weight = [&](const Item& w, int key, float v) {
            if (key >= w.sq.L) return;
            const int64_t row = (int64_t)w.sq.s * Hkv + w.h;
            if (PASS == kKeyWeights && gridDim.y > 1) {
                p.partial[((int64_t)blockIdx.y * p.num_seqs * Hkv + row) * p.max_context + key] = v;
            } else {
                float* dst = p.weights + row * p.weights_stride + key;
                *dst = key < w.sq.L - w.sq.n ? *dst + v : v;
            }
        };
        for (int64_t it = blockIdx.x; it < items && run; it += gridDim.x) {
            const Item w = item_at(it);
            if (x >= w.na) continue;
            if constexpr (PASS == kRowStats) {
                const int tok = (w.a0 + x) * TT + m / G, g = m % G;
                const bool valid = m < TT * G && tok < w.sq.rows;
                const int last = p.causal ? w.sq.L - w.sq.rows + tok : w.sq.L - 1;  // last key the row sees
                float m_used = -INFINITY, l = 0.f;
                for (int t = w.b0; t < w.b1; ++t, ++nx) {
                    if ((nx & 1) != par) continue;
                    if (!(run = acquire())) break;
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
                    release();
                }
                float2 o = make_float2(m_used, l);
                if (run) run = hand_over(x, par == 1, o);
                if (run && par == 0) {
                    const float mn = fmaxf(m_used, o.x);
                    if (mn == -INFINITY) {
                        l += o.y;
                    } else {
                        l = l * exp2f(m_used - mn) + o.y * exp2f(o.x - mn);
                        m_used = mn;
                    }
                    if (valid)
                        p.stats[(int64_t)blockIdx.y * part + (int64_t)(w.sq.row0 + tok) * p.num_heads + w.h * G + g] =
                            make_float2(m_used, l);
                }
            } else if constexpr (PASS == kKeyWeights) {
                const int key = (w.a0 + x) * TM + m;
                const int mine = w.b0 + ((nx ^ par) & 1);  // this group's first tile
                float2 st = mine < w.b1 ? row_stat(w, mine) : make_float2(0.f, 0.f);
                float total = 0.f;
                for (int t = w.b0; t < w.b1; ++t, ++nx) {
                    if ((nx & 1) != par) continue;
                    float* nm;
                    share_stat(st, nm);
                    if (t + 2 < w.b1) st = row_stat(w, t + 2);
                    if (!(run = stat_ready() && acquire())) break;
                    // columns [c0, c1) are rows of this request that see the key
                    const int c1 = min(TT, w.sq.rows - t * TT) * G;
                    const int c0 = p.causal ? (key - (w.sq.L - w.sq.rows) - t * TT) * G : 0;
                    total += key_sum(nm, c0, c1);
                    release();
                }
                float2 o = make_float2(total, 0.f);
                if (run) run = hand_over(x, par == 1, o);
                if (run && par == 0) store_weight(w, key, total + o.x);
            } else {
                // few rows: the item's query tile x stays, its statistics with it
                float* nm;
                if (w.b0 < w.b1) {
                    share_stat(row_stat(w, x), nm);
                    run = stat_ready();
                }
                const int c1 = min(TT, w.sq.rows - x * TT) * G;
                for (int t = w.b0; t < w.b1 && run; ++t, ++nx) {
                    if ((nx & 1) != par) continue;
                    if (!(run = acquire())) break;
                    const int key = t * TM + m;
                    const int c0 = p.causal ? (key - (w.sq.L - w.sq.rows) - x * TT) * G : 0;
                    float v = key_sum(nm, c0, c1);
                    release();
                    if (w.na == 2) {  // tile 1's part of the same keys
                        float2 o = make_float2(v, 0.f);
                        if (!(run = hand_over(par, x == 1, o))) break;
                        v += o.x;
                    }
                    if (x == 0) store_weight(w, key, v);
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
cudaError_t launch_umma(const WeightArgs& a, int32_t num_blocks, std::string* err, cudaStream_t stream) {
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
    const dim3 block(WGeo<HD>::NTHREADS);
    auto k1 = weights_umma_kernel<T, HD, kRowStats>;
    auto k2 = a.few_rows ? weights_umma_kernel<T, HD, kFewRows> : weights_umma_kernel<T, HD, kKeyWeights>;
    cudaError_t e = cudaFuncSetAttribute(k1, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k2, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    constexpr int NA = WGeo<HD>::NA;
    const int64_t rows = a.window > 0 ? std::min<int64_t>(a.total_q, (int64_t)a.num_seqs * a.window) : a.total_q;
    const int64_t q_items = (rows / (NA * TT) + a.num_seqs) * a.num_kv_heads;
    const int64_t k_items = a.few_rows ? (int64_t)a.num_seqs * a.num_kv_heads
                                       : (int64_t)a.num_seqs * a.num_kv_heads * ((a.max_context + NA * TM - 1) / (NA * TM));
    auto ctas = [](int64_t n) { return (unsigned)std::max<int64_t>(1, std::min<int64_t>(n, kMaxCtas)); };
    e = launch_pdl_smem(k1, dim3(ctas(q_items), (unsigned)a.key_splits), block, smem, stream, tmQ, tmK, a);
    if (e != cudaSuccess) return e;
    e = launch_pdl_smem(k2, dim3(ctas(k_items), (unsigned)a.row_splits), block, smem, stream, tmQ, tmK, a);
    if (e != cudaSuccess || a.few_rows || a.row_splits == 1) return e;
    const int64_t wrows = (int64_t)a.num_seqs * a.num_kv_heads;
    return launch_pdl(weights_join_kernel,
                      dim3((unsigned)((a.max_context + 255) / 256), (unsigned)std::min<int64_t>(wrows, 65535)), dim3(256),
                      stream, a);
}

}  // namespace

bool weights_umma_supported(int dtype, int head_dim, int block_size, int group, bool kv_fp8) {
    return !kv_fp8 && (dtype == 1 || dtype == 2) && (head_dim == 64 || head_dim == 128 || head_dim == 256) &&
           (block_size == 8 || (block_size % GRP == 0 && block_size <= 256)) && group >= 1 && group <= TM;
}

// How the work is cut.  A CTA holds an SM; where there are fewer items than
// two per SM the streamed axis is split, into pieces of at least four tiles.
WeightPlan weights_umma_plan(int32_t num_seqs, int32_t total_q, int32_t max_q, int32_t num_heads,
                             int32_t num_kv_heads, int32_t head_dim, int32_t max_context, int32_t window) {
    constexpr int64_t kWant = 2 * 152, kMinTiles = 4;
    const int G = num_heads / num_kv_heads, TT = TM / G, NA = head_dim <= 128 ? 2 : 1;
    auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    auto pieces = [&](int64_t items, int64_t tiles, int64_t most) {
        return (int)std::max<int64_t>(1, std::min({up(kWant, items), tiles / kMinTiles, most}));
    };
    WeightPlan w;
    const int64_t rows = window > 0 ? std::min<int64_t>(total_q, (int64_t)num_seqs * window) : total_q;
    const int32_t row_max = window > 0 ? std::min(max_q, window) : max_q;  // of one request
    const int64_t k_tiles = up(max_context, TM), q_tiles = up(row_max, TT);
    w.key_splits = pieces(std::max<int64_t>(1, up(rows, NA * TT)) * num_kv_heads, k_tiles, 32);
    w.few_rows = q_tiles <= NA;
    if (w.few_rows) {
        w.row_splits = pieces((int64_t)num_seqs * num_kv_heads, k_tiles, 256);
    } else {
        w.row_splits = pieces((int64_t)num_seqs * num_kv_heads * up(k_tiles, NA), q_tiles, 8);
    }
    w.stats_bytes = ((size_t)w.key_splits * total_q * num_heads * sizeof(float2) + 255) / 256 * 256;
    w.partial_bytes = !w.few_rows && w.row_splits > 1
                          ? (size_t)w.row_splits * std::min(num_seqs, kWeightMaxSeqsPerLaunch) * num_kv_heads *
                                max_context * sizeof(float)
                          : 0;
    return w;
}

cudaError_t launch_weights_umma(const WeightArgs& a, int32_t num_blocks, std::string* err, cudaStream_t stream) {
    if (a.dtype == 1)
        return a.head_dim == 64    ? launch_umma<__nv_bfloat16, 64>(a, num_blocks, err, stream)
               : a.head_dim == 128 ? launch_umma<__nv_bfloat16, 128>(a, num_blocks, err, stream)
                                   : launch_umma<__nv_bfloat16, 256>(a, num_blocks, err, stream);
    return a.head_dim == 64    ? launch_umma<__half, 64>(a, num_blocks, err, stream)
           : a.head_dim == 128 ? launch_umma<__half, 128>(a, num_blocks, err, stream)
                               : launch_umma<__half, 256>(a, num_blocks, err, stream);
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
