// pa_prefix_umma.cu -- attention of many sequences' single queries over a
// prefix that they share, on the 5th-generation tensor cores (tcgen05);
// bf16/f16, head_dim 64, 128 or 256, block_size 8 or a multiple of 16.
//
// For the members s of a group and query head h of KV head kv, over the P
// tokens whose blocks the members share:
//   m = max x_t, l = sum 2^(x_t - m), o = sum 2^(x_t - m) v_t,
//   x_t = scale * log2 e * q[s, h] . k_t,
// which pa_decode_shared.cu joins with the rest of each context.  The G query
// heads of floor(128 / G) members are the 128 rows of a tile: K and V cross
// from memory once for all of them, where a decode reads them once a member.
//
// Roles of a CTA (320 threads): warps 0-3 softmax, a row a thread, P (16 bits)
// to tensor memory as the A operand of P V, taken against the row's reference
// as it stands (a sum of at most 2^9 proves that no score is more than 9 above
// it; otherwise, and on a unit's first tile, the reference moves to the tile's
// maximum and O is rescaled); warps 4-5 and 6-7 load 16 KB stages of K (64
// elements of 128 keys) and V (all elements of 8,192 / head_dim keys) through
// the group's first block-table row; warps 8 and 9 issue S = Q K^T and
// O += P V.  Tensor memory: O, then two buffers of S (one at head_dim 256) and
// two of P.
//
// Bound: with 64 members of 4 heads per KV head a tile of 128 keys takes 1,750
// cycles where its products need 1,040 and shared memory 1,250 (64 KB loaded,
// 96 KB read by the products), but a CTA has seven of them behind 16,000 cycles
// of start (its first loads) and before 5,000 of records: 21 us for 8,192 keys,
// most of the start hidden behind the end of the decode before it.  With few
// members the prefix's bytes (5 x 13 members, 40 KV heads: 210 MB in 47 us).
//
// Every wait is bounded in time; on expiry the kernel sets a status bit, the
// roles leave their loops and the CTA still frees its tensor memory.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <string>
#include <type_traits>

#include "pa_cluster.cuh"
#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_launch.cuh"
#include "pa_shared.cuh"
#include "pa_tmap.cuh"

namespace pa {
namespace {

__device__ unsigned int g_prefix_status;

constexpr int TM = 128, BK = kPrefixKeys;
constexpr int STAGE = BK * 128;  // bytes
constexpr int NP = 2;            // loading warps of each ring
constexpr int W_LOAD = 4, W_S = W_LOAD + 2 * NP, W_O = W_S + 1;
constexpr int NTHREADS = 32 * (W_O + 1);
constexpr uint32_t TMEM_COLS = 512;
constexpr uint64_t WAIT_NS = 2000000000ull;

template <int HD>
struct Geo {
    static constexpr int CH = HD / 64;      // 128-byte chunks of a row; K stages (and V stages) per tile
    static constexpr int VK = 8192 / HD;    // keys of a V stage
    static constexpr int NK = HD == 64 ? 6 : HD == 128 ? 5 : 4, NV = HD == 256 ? 4 : 5, NST = NK + NV;
    static constexpr int NS = HD == 256 ? 1 : 2;  // S buffers
    static constexpr uint32_t O_COL = 0, S_COL = HD, P_COL = HD + NS * 128;
    static constexpr int Q_OFF = 0;
    static constexpr int OUT_OFF = TM * HD * 2;  // 4 KB a softmax warp
    static constexpr int ST_OFF = OUT_OFF + 4 * 4096;
    static constexpr int BAR_OFF = ST_OFF + NST * STAGE;
    // full[NST], empty[NST], s_full[2], s_empty[2], p_full[2], p_empty[2], q_full, q_empty, o_empty
    static constexpr int NBAR = 2 * NST + 8 + 3;
    static constexpr int MISC_OFF = BAR_OFF + NBAR * 8;
    static constexpr int PREFIX_OFF = MISC_OFF + 16;
    static_assert(P_COL + 128 <= TMEM_COLS, "fits in tensor memory");
};
template <int HD>
constexpr size_t smem_bytes(int groups) {
    return 1024 + Geo<HD>::PREFIX_OFF + (size_t)(groups + 1) * 4;
}
static_assert(smem_bytes<64>(kDecodeMaxSeqsPerLaunch) <= 232448 && smem_bytes<128>(kDecodeMaxSeqsPerLaunch) <= 232448 &&
                  smem_bytes<256>(kDecodeMaxSeqsPerLaunch) <= 232448,
              "fits in shared memory");

struct Params {
    SharedGroups g;
    const int32_t* block_tables;
    int32_t max_blocks;
    int32_t num_heads;
    int32_t group;  // query heads per KV head
    int32_t box_rows;
    float scale_log2;
};

// A unit and its key tiles [k0, k1) of nk within the run [f0, f1).
struct Segment {
    int g, kv, t;  // group, KV head, tile of members
    int P, nk, k0, k1;
    int64_t u0;
    __device__ __forceinline__ int64_t end() const { return u0 + kPrefixUnit + nk; }
    __device__ __forceinline__ void cut(int64_t f0, int64_t f1) {
        k0 = (int)max(f0 - u0 - kPrefixUnit, (int64_t)0);
        k1 = (int)max(min((int64_t)nk, f1 - u0 - kPrefixUnit), (int64_t)0);
    }
    __device__ __forceinline__ void of_group(const Params& p, int group) {
        g = group;
        P = shared_tokens(p.g, g);
        nk = (P + BK - 1) / BK;
    }
    // to the unit after this one (before the list's end)
    __device__ __forceinline__ void next(const Params& p, int64_t f0, int64_t f1) {
        u0 = end();
        if (++t == shared_row_tiles(p.g, g)) {
            t = 0;
            if (++kv == p.g.num_kv_heads) {
                kv = 0;
                do of_group(p, g + 1);
                while (nk == 0);
            }
        }
        cut(f0, f1);
    }
};
__device__ __forceinline__ Segment locate(const Params& p, const int32_t* prefix, int64_t f0, int64_t f1) {
    int lo = 0, hi = p.g.groups - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= f0) lo = mid;
        else hi = mid - 1;
    }
    Segment s;
    s.of_group(p, lo);
    const int unit = (int)(f0 - prefix[lo]) / (s.nk + kPrefixUnit), tiles = shared_row_tiles(p.g, lo);
    s.kv = unit / tiles;
    s.t = unit - s.kv * tiles;
    s.u0 = prefix[lo] + (int64_t)unit * (s.nk + kPrefixUnit);
    s.cut(f0, f1);
    return s;
}

__device__ __forceinline__ uint32_t lane0(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
// Shared-memory matrix descriptor of a 128-byte-swizzled operand from its low
// word (address >> 4 | leading byte offset >> 4 << 16): stride 1024 bytes.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t lo) {
    return (uint64_t)((1024u >> 4) | (1u << 14) | (2u << 29)) << 32 | lo;
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

template <typename T, int HD>
__global__ void __launch_bounds__(NTHREADS, 1)
    prefix_umma_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const Params p) {
    using Gm = Geo<HD>;
    constexpr int CH = Gm::CH, VK = Gm::VK, NST = Gm::NST, NS = Gm::NS, REC = HD + 4;
    constexpr bool kBF16 = std::is_same<T, __nv_bfloat16>::value;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(base + Gm::BAR_OFF);
    uint64_t* empty = full + NST;
    uint64_t* s_full = empty + NST;
    uint64_t* s_empty = s_full + 2;
    uint64_t* p_full = s_empty + 2;
    uint64_t* p_empty = p_full + 2;
    uint64_t* q_full = p_empty + 2;
    uint64_t* q_empty = q_full + 1;
    uint64_t* o_empty = q_empty + 1;
    volatile uint32_t* taddr_slot = reinterpret_cast<volatile uint32_t*>(base + Gm::MISC_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(base + Gm::MISC_OFF + 4);
    int32_t* prefix = reinterpret_cast<int32_t*>(base + Gm::PREFIX_OFF);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = p.group;

    if (threadIdx.x == 32 * W_LOAD) {
        prefetch_tmap(&tmQ);
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
    }
    // Launched behind the decode of the rests, whose output this kernel does not
    // read: it starts on each SM as the decode leaves it.  Its inputs are older
    // than that grid, which waited for the grids before it.  The join behind
    // waits for this grid only, so one CTA waits for the decode at its end.
    pdl_launch_dependents();
    shared_prefix(p.g, prefix);
    const int64_t W = prefix[p.g.groups], C = shared_ctas(W, gridDim.x);
    const int64_t f0 = blockIdx.x * W / C, f1 = (blockIdx.x + 1) * W / C;
    if (blockIdx.x >= C || f0 == f1) {
        if (blockIdx.x == 0) pdl_wait_primary();
        return;
    }
    const Segment first = locate(p, prefix, f0, f1);

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2 * NST; ++i) mbar_init(&full[i], 1u);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1u);
            mbar_init(&s_empty[i], 4u);
            mbar_init(&p_full[i], 4u);
            mbar_init(&p_empty[i], 1u);
        }
        mbar_init(q_full, NP);
        mbar_init(q_empty, 1u);
        mbar_init(o_empty, 4u);
        *abort_flag = 0;
        mbar_fence_init();
    }
    if (warp == W_S) {
        tmem_alloc(const_cast<uint32_t*>(taddr_slot), TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *taddr_slot;
    const uint32_t sb = smem_u32(base);

    auto fail = [&]() {
        *abort_flag = 1;
        atomicOr(&g_prefix_status, kStatusTimeout);
    };
    // A whole warp's bounded wait, with one answer for all lanes.  `ready`: what
    // an earlier look told this lane.
    auto wait_after = [&](uint64_t* bar, uint32_t parity, bool ready) -> bool {
        if (__all_sync(0xffffffffu, ready)) return true;
        const uint64_t t0 = global_ns();
        bool ok = true;
        for (int i = 0; !__all_sync(0xffffffffu, mbar_try_wait(bar, parity)); ++i)
            if ((i & 15) == 15 && __any_sync(0xffffffffu, *abort_flag != 0 || global_ns() - t0 > WAIT_NS)) {
                ok = false;
                break;
            }
        if (!ok && lane == 0) fail();
        return ok;
    };
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool { return wait_after(bar, parity, mbar_test(bar, parity)); };

    // A role's place in its ring: slots [first, first + n) of the stages.
    struct Ring {
        int first, n, slot;
        uint32_t phase;
        __device__ __forceinline__ void next() {
            if (++slot == first + n) slot = first, phase ^= 1;
        }
    };

    if (warp >= W_LOAD && warp < W_S) {
        // ---------------- loads: the stages of a ring go to its NP warps in turn
        const int w = (warp - W_LOAD) % NP;
        const bool values = warp >= W_LOAD + NP;
        const int br = p.box_rows, gpt = BK / br, gpv = VK / br;
        Ring ring = values ? Ring{Gm::NK, Gm::NV, Gm::NK, 0} : Ring{0, Gm::NK, 0, 0};
        int seg = 0, turn = 0;
        bool run = true;
        auto skip = [&]() -> bool {
            const bool other = turn != w;
            if (++turn == NP) turn = 0;
            if (other) ring.next();
            return other;
        };
        for (Segment s = first; run; s.next(p, f0, f1)) {
            if (s.k1 <= s.k0) break;
            const int s0 = p.g.starts[s.g];
            const int32_t* table = p.block_tables + (int64_t)s0 * p.max_blocks;
            // pool row of this lane's box of tile k
            auto box_row = [&](int k) -> int32_t {
                const int tok = k * BK + lane * br, bs = p.g.block_size;
                return lane < gpt && k < s.k1 && tok < s.P ? table[tok / bs] * bs + tok % bs : 0;
            };
            int32_t cur = box_row(s.k0);
            if (!values) {
                // the members' queries: chunks w, w + NP, ..
                if (!(run = wait(q_empty, (seg & 1) ^ 1))) break;
                const int chunks = w < CH ? (CH - w + NP - 1) / NP : 0;
                if (lane == 0) {
                    if (chunks) mbar_arrive_expect_tx(q_full, (uint32_t)(chunks * 128 * G * p.g.tokens));
                    else mbar_arrive(q_full);
                }
                __syncwarp();
                if (lane < chunks) {
                    const int c = w + NP * lane;
                    tma_load_3d(base + Gm::Q_OFF + c * TM * 128, &tmQ, q_full, 64 * c, s.kv * G,
                                s0 + s.t * p.g.tokens, l2_policy_evict_last());
                }
            }
            for (int k = s.k0; k < s.k1 && run; ++k) {
                const int32_t nxt = box_row(k + 1);
                const int valid = min(s.P - k * BK, BK);
                const int n = values ? (valid + VK - 1) / VK : CH;
                for (int j = 0; j < n; ++j) {
                    if (skip()) continue;
                    if (!(run = wait(&empty[ring.slot], ring.phase ^ 1))) break;
                    uint8_t* st = base + Gm::ST_OFF + ring.slot * STAGE;
                    uint64_t* bar = &full[ring.slot];
                    if (!values) {  // chunk j of the tile's keys
                        const int boxes = (valid + br - 1) / br;
                        if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(boxes * br * 128));
                        __syncwarp();
                        if (lane < boxes)
                            tma_load_3d(st + lane * br * 128, &tmK, bar, 0, s.kv * CH + j, cur, l2_policy_evict_last());
                    } else {  // all chunks of VK keys
                        const int boxes = (min(valid - j * VK, VK) + br - 1) / br;
                        const int b = lane % gpv, c = lane / gpv;
                        const int32_t row = __shfl_sync(0xffffffffu, cur, j * gpv + b);
                        if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(boxes * CH * br * 128));
                        __syncwarp();
                        if (c < CH && b < boxes)
                            tma_load_3d(st + c * VK * 128 + b * br * 128, &tmV, bar, 0, s.kv * CH + c, row,
                                        l2_policy_evict_last());
                    }
                    ring.next();
                }
                cur = nxt;
            }
            ++seg;
            if (s.end() >= f1) break;
        }
        // every stage handed back, and the last queries read
        for (int i = 0; i < ring.n && run; ++i) {
            run = wait(&empty[ring.slot], ring.phase ^ 1);
            ring.next();
        }
        if (run && !values) run = wait(q_empty, (seg & 1) ^ 1);
        if (!run) {  // a wait ran out: the copies in flight get time to land
            const uint64_t t0 = global_ns();
            while (global_ns() - t0 < 1000000ull) {}
        }
    } else if (warp == W_S) {
        // ---------------- S = Q K^T
        constexpr uint32_t idS = umma_idesc_f16(128, BK, kBF16, false);
        Ring ring{0, Gm::NK, 0, 0};
        int seg = 0, it = 0;
        bool run = true;
        const uint32_t tm0 = lane0(tmem), q_lo = lane0(((sb + Gm::Q_OFF) & 0x3ffffu) >> 4 | 1u << 16);
        const uint32_t st_lo = lane0(((sb + Gm::ST_OFF) & 0x3ffffu) >> 4 | 1u << 16);
        for (Segment s = first; run; s.next(p, f0, f1)) {
            if (s.k1 <= s.k0) break;
            if (!(run = wait(q_full, seg & 1))) break;
            bool ready = mbar_test(&full[ring.slot], ring.phase);
            for (int k = s.k0; k < s.k1 && run; ++k, ++it) {
                const int buf = NS == 2 ? it & 1 : 0, use = NS == 2 ? it >> 1 : it;
                const uint32_t d = lane0(tm0 + Gm::S_COL + 128 * buf);
                if (!(run = wait(&s_empty[buf], (use & 1) ^ 1))) break;
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < CH; ++c) {
                    if (!(run = wait_after(&full[ring.slot], ring.phase, ready))) break;
                    const uint32_t a = lane0(q_lo + c * (TM * 128 / 16)), b = lane0(st_lo + ring.slot * (STAGE / 16));
                    const uint32_t old = lane0(c ? 1u : 0u);
                    uint64_t* done = &empty[ring.slot];
                    ring.next();
                    ready = mbar_test(&full[ring.slot], ring.phase);
                    if (elect_lane()) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_f16(d, sw128_desc(a + 2 * kk), sw128_desc(b + 2 * kk), idS, kk ? 1u : old);
                        umma_commit(done);
                        if (c == CH - 1) {
                            umma_commit(&s_full[buf]);
                            if (k == s.k1 - 1) umma_commit(q_empty);
                        }
                    }
                    __syncwarp();
                }
            }
            ++seg;
            if (s.end() >= f1) break;
        }
    } else if (warp == W_O) {
        // ---------------- O += P V
        constexpr uint32_t idO = umma_idesc_f16(128, HD, kBF16, true);
        Ring ring{Gm::NK, Gm::NV, Gm::NK, 0};
        int seg = 0, it = 0;
        bool run = true;
        const uint32_t tm0 = lane0(tmem);
        const uint32_t st_lo = lane0(((sb + Gm::ST_OFF) & 0x3ffffu) >> 4 | (uint32_t)(VK * 128 / 16) << 16);
        for (Segment s = first; run; s.next(p, f0, f1)) {
            if (s.k1 <= s.k0) break;
            if (!(run = wait(o_empty, (seg & 1) ^ 1))) break;
            for (int k = s.k0; k < s.k1 && run; ++k, ++it) {
                const int buf = it & 1;
                bool ready = mbar_test(&full[ring.slot], ring.phase);
                if (!(run = wait(&p_full[buf], (it >> 1) & 1))) break;
                tc_fence_after();
                const int valid = min(s.P - k * BK, BK), steps = valid / 16, n = (valid + VK - 1) / VK;
#pragma unroll 1
                for (int j = 0; j < n; ++j) {
                    if (!(run = wait_after(&full[ring.slot], ring.phase, ready))) break;
                    const uint32_t a = lane0(tm0 + Gm::P_COL + 64 * buf + j * (VK / 2));
                    const uint32_t b = lane0(st_lo + ring.slot * (STAGE / 16));
                    const uint32_t old = lane0(k > s.k0 || j ? 1u : 0u);
                    uint64_t* done = &empty[ring.slot];
                    ring.next();
                    ready = mbar_test(&full[ring.slot], ring.phase);
                    if (elect_lane()) {
#pragma unroll
                        for (int kk = 0; kk < VK / 16; ++kk) {
                            if (j * (VK / 16) + kk >= steps) break;
                            umma_f16_ts(tm0 + Gm::O_COL, a + 8 * kk, sw128_desc(b + kk * 128), idO, kk ? 1u : old);
                        }
                        umma_commit(done);
                        if (j == n - 1) umma_commit(&p_empty[buf]);
                    }
                    __syncwarp();
                }
            }
            ++seg;
            if (s.end() >= f1) break;
        }
    } else {
        // ---------------- softmax: thread r has row r
        const int r = threadIdx.x;
        const uint32_t t_lane = tmem + ((uint32_t)(warp * 32) << 16);
        const float scale = p.scale_log2 == 0.f ? 1e-38f : p.scale_log2;  // (0: every score counts alike)
        const float hidden = scale > 0.f ? -INFINITY : INFINITY;
        int it = 0;
        bool ok = true;
        for (Segment s = first; ok; s.next(p, f0, f1)) {
            if (s.k1 <= s.k0) break;
            const int s0 = p.g.starts[s.g] + s.t * p.g.tokens, members = min(p.g.starts[s.g + 1] - s0, p.g.tokens);
            const int rows = members * G;
            const bool mine = r < rows;
            float m = -INFINITY, l = 0.f;
            for (int k = s.k0; k < s.k1 && ok; ++k, ++it) {
                const int buf = it & 1, sbuf = NS == 2 ? buf : 0, suse = NS == 2 ? it >> 1 : it;
                if (!(ok = wait(&s_full[sbuf], suse & 1))) break;
                if (!(ok = wait(&p_empty[buf], ((it >> 1) & 1) ^ 1))) break;
                tc_fence_after();
                const int valid = s.P - k * BK;
                const uint32_t t_s = t_lane + Gm::S_COL + 128 * sbuf;
                auto scores = [&](int c, float (&x)[32]) {
                    tmem_ld32(t_s + 32 * c, x);
                    tmem_wait_ld();
                    if (valid < BK) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] = 32 * c + i < valid ? x[i] : hidden;
                    }
                };
                bool move = k == s.k0;
                float alpha = 1.f, sum = 0.f;
                while (warp * 32 < rows) {
                    if (move) {
                        float mx = -INFINITY;
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            float x[32];
                            scores(c, x);
#pragma unroll
                            for (int i = 0; i < 32; ++i) mx = fmaxf(mx, x[i] * scale);
                        }
                        if (mine && (mx > m + 9.f || (m == -INFINITY && mx > m))) {
                            alpha = fast_exp2(m - mx);
                            m = mx;
                        }
                    }
                    const float ms = m == -INFINITY ? 0.f : m;
                    const unsigned long long sc2 = f32x2_pack(scale, scale), off2 = f32x2_pack(-ms, -ms);
                    unsigned long long sum2 = 0ull;
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        float x[32];
                        uint32_t pk[16];
                        scores(c, x);
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            float a, b;
                            f32x2_unpack(fma_f32x2(f32x2_pack(x[i], x[i + 1]), sc2, off2), a, b);
                            a = fast_exp2(a);
                            b = fast_exp2(b);
                            sum2 = add_f32x2(sum2, f32x2_pack(a, b));
                            pk[i / 2] = pack2<T>(a, b);
                        }
                        tmem_st16(t_lane + Gm::P_COL + 64 * buf + 16 * c, pk);
                    }
                    float sa, sc;
                    f32x2_unpack(sum2, sa, sc);
                    sum = sa + sc;
                    if (move || !__any_sync(0xffffffffu, mine && !(sum <= 512.f && m != -INFINITY))) break;
                    move = true;
                }
                l = fmaf(l, alpha, sum);
                tmem_wait_st();
                if (k > s.k0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                    // O holds the tiles before this one
                    if (!(ok = wait(&p_empty[buf ^ 1], ((it - 1) >> 1) & 1))) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < HD; c += 32) {
                        float o[32];
                        tmem_ld32(t_lane + Gm::O_COL + c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] *= alpha;
                        tmem_st32(t_lane + Gm::O_COL + c, o);
                    }
                    tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&s_empty[sbuf]);
                    mbar_arrive(&p_full[buf]);
                }
            }
            if (!ok || !(ok = wait(&p_empty[(it - 1) & 1], ((it - 1) >> 1) & 1))) break;
            tc_fence_after();
            // the rows' records, 32 columns at a time through shared memory
            uint8_t* stage = base + Gm::OUT_OFF + warp * 4096;
            const int first_row = warp * 32, n = min(max(rows - first_row, 0), 32);
            auto record = [&](int i) -> float* {  // of row first_row + i
                const int row = first_row + i, seq = row / G;
                return s.k0 ? p.g.cont + ((int64_t)blockIdx.x * TM + row) * REC
                            : p.g.rows + ((int64_t)(s0 + seq) * p.num_heads + s.kv * G + row - seq * G) * REC;
            };
            if (mine) {
                float* rec = record(lane);
                rec[HD] = m;
                rec[HD + 1] = l;
            }
            if (n > 0) {
                float* out[8];  // of rows lane / 8, + 4, ..
#pragma unroll
                for (int i = 0; i < 8; ++i) out[i] = record(min((lane >> 3) + 4 * i, n - 1)) + 4 * (lane & 7);
#pragma unroll 1
                for (int c = 0; c < HD; c += 32) {
                    float o[32];
                    tmem_ld32(t_lane + Gm::O_COL + c, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        *reinterpret_cast<float4*>(stage + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                            make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int row = (lane >> 3) + 4 * i;
                        if (row < n)
                            *reinterpret_cast<float4*>(out[i] + c) =
                                *reinterpret_cast<const float4*>(stage + row * 128 + (((lane & 7) ^ (row & 7)) << 4));
                    }
                    __syncwarp();
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_empty);
            if (s.end() >= f1) break;
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == W_S) tmem_dealloc(tmem, TMEM_COLS);
    if (blockIdx.x == 0) pdl_wait_primary();
}

// ---------------------------------------------------------------- host side

template <typename T, int HD>
cudaError_t launch_typed(const AttnArgs& a, const SharedGroups& g, int32_t num_blocks, int ctas, std::string* err,
                         cudaStream_t stream) {
    const int G = a.num_heads / a.num_kv_heads, ch = HD / 64, bs = a.block_size;
    const CUtensorMapDataType ty = a.dtype == 1 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    Params p;
    p.box_rows = bs == 8 ? 8 : bs % 64 == 0 && HD <= 128 ? 64 : bs % 32 == 0 ? 32 : 16;
    CUtensorMap tmQ, tmK, tmV;
    const cuuint64_t qdims[3] = {(cuuint64_t)HD, (cuuint64_t)a.num_heads, (cuuint64_t)a.num_seqs};
    const cuuint64_t qstr[2] = {(cuuint64_t)HD * 2, (cuuint64_t)a.num_heads * HD * 2};
    const cuuint32_t qbox[3] = {64, (cuuint32_t)G, (cuuint32_t)g.tokens};
    const cuuint64_t dims[3] = {64, (cuuint64_t)a.num_kv_heads * ch, (cuuint64_t)num_blocks * bs};
    const cuuint64_t str[2] = {128, (cuuint64_t)a.num_kv_heads * HD * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)p.box_rows};
    if (!encode_tiled_3d(&tmQ, ty, a.q, qdims, qstr, qbox, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, err) ||
        !encode_tiled_3d(&tmK, ty, a.k_cache, dims, str, box, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, err) ||
        !encode_tiled_3d(&tmV, ty, a.v_cache, dims, str, box, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, err))
        return cudaErrorInvalidValue;
    p.g = g;
    p.block_tables = a.block_tables;
    p.max_blocks = a.max_blocks;
    p.num_heads = a.num_heads;
    p.group = G;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(&prefix_umma_kernel<T, HD>),
                               smem_bytes<HD>(kDecodeMaxSeqsPerLaunch));
    if (e != cudaSuccess) return e;
    return launch_pdl_smem(prefix_umma_kernel<T, HD>, dim3((unsigned)ctas), dim3(NTHREADS), smem_bytes<HD>(g.groups),
                           stream, tmQ, tmK, tmV, p);
}

}  // namespace

cudaError_t launch_prefix_umma(const AttnArgs& a, const SharedGroups& g, int32_t num_blocks, int ctas,
                               std::string* err, cudaStream_t stream) {
    if (a.dtype == 1)
        return a.head_dim == 64    ? launch_typed<__nv_bfloat16, 64>(a, g, num_blocks, ctas, err, stream)
               : a.head_dim == 128 ? launch_typed<__nv_bfloat16, 128>(a, g, num_blocks, ctas, err, stream)
                                   : launch_typed<__nv_bfloat16, 256>(a, g, num_blocks, ctas, err, stream);
    return a.head_dim == 64    ? launch_typed<__half, 64>(a, g, num_blocks, ctas, err, stream)
           : a.head_dim == 128 ? launch_typed<__half, 128>(a, g, num_blocks, ctas, err, stream)
                               : launch_typed<__half, 256>(a, g, num_blocks, ctas, err, stream);
}

uint32_t prefix_umma_status(bool clear) {
    unsigned int v = 0;
    cudaMemcpyFromSymbol(&v, g_prefix_status, sizeof(v));
    if (clear) {
        const unsigned int z = 0;
        cudaMemcpyToSymbol(g_prefix_status, &z, sizeof(z));
    }
    return v;
}

}  // namespace pa
