// pa_latent_umma.cu -- attention over a latent cache on the 5th-generation
// tensor cores, two SMs per tile (cta_group::2); bf16/f16, rows of 512 latent
// and 64 rotated elements.
//
// Row t of the cache is [c_t | r_t].  For query row (token i, head h):
//   x_t = scale * q[i, h] . [c_t | r_t],  out[i, h] = softmax(x) C.
// All heads of a request share its rows, so a tile is 128 consecutive (token,
// head) rows of one request, whatever the number of heads: one row of 1,152
// bytes then feeds 128 x 1,088 products.  A single token of 128 heads is one
// tile, and at 16 heads a tile is an eighth full, which costs nothing while
// the cache's bytes are the bound (below).
//
// Why two SMs.  O is 128 rows x 512 columns of fp32: all of an SM's tensor
// memory, with no place for the scores.  A pair of SMs works the 128 rows as
// 64 + 64: each holds its rows' O in 256 columns (lanes 0-63 dims 0-255, lanes
// 64-127 dims 256-511) and two score buffers of 64 columns (lanes 0-63 keys
// 0-63 of the tile, lanes 64-127 keys 64-127).  For S = Q K^T each CTA brings
// 64 of the 128 keys (all 576 elements), for O += P C its half of the latent
// dims of all 128 keys.  One SM with half of the dims would compute every
// score twice (1.5 times the products).
//
// Roles of a CTA (320 threads):
//   warps 0-3   softmax: a thread has one row and half of a tile's keys;
//               partners (64 threads apart) swap their maxima through shared
//               memory; P goes to shared memory as the A operand.  O is
//               rescaled only when a row's maximum grows by more than 2^8.
//   warps 4-7   loads: 16 KB stages -- two 64-element chunks of the CTA's 64
//               keys in a ring of four or five (warps 4, 5), two chunks of its
//               dims of 64 keys in a ring of the other three or two (warps 6,
//               7), boxes issued by a
//               lane each; both CTAs' bytes are counted on the even CTA's
//               barrier.
//   warp 8, 9   (even CTA) issue the MMAs of S and of P C: two warps, because
//               a stage's wait, descriptors and commit take one warp longer
//               than its products take the tensor pipe.
//
// Work: all (request, row tile) units' key tiles form one list, cut into equal
// runs, one per pair; a unit cut between pairs leaves (m, l, o) records that
// latent_merge_kernel joins.  The cut depends on the lengths only.
//
// Bound: shared memory.  Per tile and SM the products read 147 KB (S: 4 KB per
// M 128 x N 128 instruction of a pair) and 98 KB (P C), the loads write 136 KB
// (each CTA's keys, and its dims of all keys once more) and P 16 KB: 3,100
// cycles at 128 bytes each, where the tensor pipe needs 2,180 and memory, for
// single tokens, 3,140.  A tile takes 2,700-3,000 cycles of 8,192 new tokens
// (1.35-1.4 PFLOP/s) and 3,700 from memory (8 x 32,768 tokens: 4.2 TB/s over the
// call).  A unit costs kUnit tiles more, and the first products of a launch
// come 10 us after its start: 152 SMs fill their rings at once.
//
// Every wait is bounded in time; on expiry the kernel sets a status bit, the
// roles leave their loops, and the pair still frees its tensor memory.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <string>
#include <type_traits>

#include "pa_cluster.cuh"
#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_launch.cuh"
#include "pa_tmap.cuh"

namespace pa {
namespace {

__device__ unsigned int g_latent_status;

constexpr int LAT = 512, ROT = 64, D = LAT + ROT;
constexpr int CH = D / 64;     // 128-byte chunks of a row
constexpr int TM = 128;        // query rows per tile, 64 per CTA
constexpr int BK = 128;        // keys per tile, 64 per CTA
constexpr int CHB = 64 * 128;  // bytes of a chunk of 64 rows
constexpr int STAGE = 2 * CHB;
constexpr int NST = 7;  // stages, of keys and of values
constexpr int W_LOAD = 4, NP = 2;  // NP loading warps for keys, NP for values
constexpr int W_S = W_LOAD + 2 * NP, W_O = W_S + 1;
constexpr int NTHREADS = 32 * (W_O + 1);
constexpr uint32_t TMEM_COLS = 512, O_COL = 0, S_COL = 256;  // S: two buffers of 64
constexpr uint64_t WAIT_NS = 2000000000ull;
constexpr int kMaxSeqs = 2000;    // requests per launch (their tile counts' prefix is in shared memory)
constexpr int REC = LAT + 4;      // floats of a record's row: o, m, l
constexpr int kPairs = kSms / 2;

constexpr int Q_OFF = 0;
constexpr int P_OFF = CH * CHB;
constexpr int ST_OFF = P_OFF + 2 * 2 * CHB;
constexpr int BAR_OFF = ST_OFF + NST * STAGE;
// full[NST], empty[NST], s_full[2], s_empty[2], p_full[2], p_empty[2], q_full, q_empty, o_empty, tail[NP]
// (full and empty: the keys' ring, then the values')
constexpr int NBAR = 2 * NST + 8 + 3 + NP;
constexpr int X_OFF = (BAR_OFF + NBAR * 8 + 15) / 16 * 16;  // float [2][128] swapped maxima (and sums)
constexpr int MISC_OFF = X_OFF + 2 * 128 * 4;               // tensor-memory address, abort flag
constexpr int PREFIX_OFF = MISC_OFF + 16;
constexpr size_t smem_bytes(int seqs) { return 1024 + PREFIX_OFF + (size_t)(seqs + 1) * 4; }
static_assert(smem_bytes(kMaxSeqs) <= 232448, "fits in shared memory");

struct Params {
    void* out;
    const int32_t* block_tables;
    int32_t max_blocks;
    const int32_t* seq_lens;
    const int32_t* cu;  // nullptr: one query per sequence
    int32_t num_seqs;
    int32_t num_heads;
    int32_t block_size;
    int32_t box_rows;  // rows of a box of the cache: a power of two, up to 64
    int32_t causal;
    float scale_log2;
    float* records;  // [2 pairs][rec_rows][REC]
    int32_t rec_rows;
    struct Cut* cuts;  // [pairs]
};
// The unit that a pair begins and others end, for the kernel that joins its
// records: its rows from row0 on (0 rows: there is none), the last pair of it,
// and the list's cost (pairs beyond it have no piece).
struct alignas(16) Cut {
    int32_t rows, last, cost, pad;
    int64_t row0, pad2;
};

// A request: its first (token, head) row, rows, tokens cached before the new
// ones, context; its row tiles, the key tiles of its context, and b (below).
struct Request {
    int64_t row0, b;
    int rows, before, L, tiles, whole;
};
__device__ __forceinline__ Request request(const Params& p, int s) {
    Request r;
    r.L = max(p.seq_lens[s], 0);
    int q0 = s, n = 1;
    if (p.cu) {
        q0 = p.cu[s];
        n = max(p.cu[s + 1] - q0, 0);
    }
    if (r.L == 0) n = 0;
    r.row0 = (int64_t)q0 * p.num_heads;
    r.rows = n * p.num_heads;
    r.before = max(r.L - n, 0);
    r.tiles = (r.rows + TM - 1) / TM;
    r.whole = (r.L + BK - 1) / BK;
    r.b = (127 + (int64_t)p.num_heads * (r.before + 128)) >> 7;
    return r;
}
// Key tiles of row tile t.  With causal masking tile t ends at row x = 128 t +
// 127, of token x / H, which sees before + x / H + 1 keys: ceil of that by 128
// is floor((t + b) / H) with b = floor((127 + H (before + 128)) / 128), so sums
// over t are closed forms.  The last tile sees the whole context.
__device__ __forceinline__ int key_tiles(const Params& p, const Request& r, int t) {
    if (!p.causal || t == r.tiles - 1) return r.whole;
    const uint64_t x = (uint64_t)(t + r.b);
    return x >> 32 ? (int)(x / (uint64_t)p.num_heads) : (int)((uint32_t)x / (uint32_t)p.num_heads);
}
// A unit (row tile of a request) costs its key tiles and kUnit more: what
// loading its queries, its first maxima and its output cost in tiles.
constexpr int kUnit = 3;
__device__ __forceinline__ int64_t floor_sum(int64_t x, int64_t h) {  // sum of floor(i / h), i < x
    const int64_t q = x / h;
    return h * (q * (q - 1) / 2) + (x - q * h) * q;
}
// Cost of a request's units before t.
__device__ __forceinline__ int64_t cost_before(const Params& p, const Request& r, int t) {
    if (t <= 0) return 0;
    if (!p.causal || r.tiles == 1) return (int64_t)t * (r.whole + kUnit);
    const int64_t u = min(t, r.tiles - 1);
    return floor_sum(r.b + u, p.num_heads) - floor_sum(r.b, p.num_heads) + (t == r.tiles ? r.whole : 0) +
           (int64_t)t * kUnit;
}

// Exclusive prefix of the requests' costs, in shared memory (every thread;
// ends with a block barrier).
__device__ __forceinline__ void cost_prefix(const Params& p, int32_t* prefix) {
    for (int s = threadIdx.x; s < p.num_seqs; s += blockDim.x) {
        const Request r = request(p, s);
        prefix[s + 1] = (int)cost_before(p, r, r.tiles);
    }
    if (threadIdx.x == 0) prefix[0] = 0;
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x, per = (p.num_seqs + 31) / 32;
        const int lo = 1 + lane * per, hi = min(p.num_seqs + 1, lo + per);
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

// The unit at a place of the flat list of costs, and its key tiles [k0, k1) of
// nk that lie in the run [f0, f1) of a pair: none where the run ends within the
// unit's own cost.  Walks the units of a run one after the other.
struct Segment {
    int req, t;      // request, row tile
    int k0, k1, nk;
    int64_t u0;      // the unit's place
    Request r;
    __device__ __forceinline__ int64_t end() const { return u0 + kUnit + nk; }
    // A continuation is its pair's first piece, any other piece that does not
    // end its unit the pair's last: a record each.
    __device__ __forceinline__ int slot() const { return k0 ? 0 : 1; }
    __device__ __forceinline__ void cut(const Params& p, int64_t f0, int64_t f1) {
        nk = key_tiles(p, r, t);
        k0 = (int)max(f0 - u0 - kUnit, (int64_t)0);
        k1 = (int)max(min((int64_t)nk, f1 - u0 - kUnit), (int64_t)0);
    }
    // to the unit after this one (before the list's end)
    __device__ __forceinline__ void next(const Params& p, int64_t f0, int64_t f1) {
        u0 = end();
        if (++t >= r.tiles) {
            t = 0;
            do r = request(p, ++req);
            while (r.tiles == 0);
        }
        cut(p, f0, f1);
    }
};
__device__ __forceinline__ Segment locate(const Params& p, const int32_t* prefix, int64_t f, int64_t f0, int64_t f1) {
    Segment s;
    int lo = 0, hi = p.num_seqs - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= f) lo = mid;
        else hi = mid - 1;
    }
    s.req = lo;
    s.r = request(p, lo);
    const int64_t rem = f - prefix[lo];
    int a = 0, b = s.r.tiles - 1;
    while (a < b) {
        const int mid = (a + b + 1) >> 1;
        if (cost_before(p, s.r, mid) <= rem) a = mid;
        else b = mid - 1;
    }
    s.t = a;
    s.u0 = prefix[lo] + cost_before(p, s.r, a);
    s.cut(p, f0, f1);
    return s;
}

__device__ __forceinline__ uint32_t lane0(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
// Shared-memory matrix descriptor of a 128-byte-swizzled operand from its low
// word (address >> 4 | leading byte offset >> 4 << 16): stride 1024 bytes.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t lo) {
    return (uint64_t)((1024u >> 4) | (1u << 14) | (2u << 29)) << 32 | lo;
}

// FINE: boxes of one or two rows (block sizes that are no multiple of 4), more
// than a box a lane and stage: 64 x 2,048 tokens of 16 heads in blocks of 6 take
// 109 us and in blocks of one 189 (on the CUDA cores 912, in blocks of 16 58).
// An instance of its own: as a branch it cost the other sizes 1 to 5 %.
// SINGLE: one token per request.  The keys come from memory, the values mostly
// from L2 behind them: five stages for the keys (8 x 32,768 tokens 88 -> 85 us,
// 64 x 16 heads 60 -> 56; four and three for prompts, whose rows stay in L2:
// 8,192 tokens 800 us against 884, 16 chunks 261 against 296).
template <typename T, bool SINGLE, bool FINE>
__global__ void __launch_bounds__(NTHREADS, 1)
    latent_umma_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmC,
                       const Params p) {
    constexpr bool kBF16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr int NK = SINGLE ? 5 : 4, NV = NST - NK;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(base + BAR_OFF);
    uint64_t* full = bars;  // even CTA: both CTAs' loads of a stage
    uint64_t* empty = full + NST;
    uint64_t* s_full = empty + NST;
    uint64_t* s_empty = s_full + 2;  // even CTA: both CTAs' softmax warps
    uint64_t* p_full = s_empty + 2;  // even CTA, the same
    uint64_t* p_empty = p_full + 2;
    uint64_t* q_full = p_empty + 2;  // even CTA
    uint64_t* q_empty = q_full + 1;
    uint64_t* o_empty = q_empty + 1;  // even CTA
    uint64_t* tail = o_empty + 1;
    float* xch = reinterpret_cast<float*>(base + X_OFF);
    volatile uint32_t* taddr_slot = reinterpret_cast<volatile uint32_t*>(base + MISC_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(base + MISC_OFF + 4);
    int32_t* prefix = reinterpret_cast<int32_t*>(base + PREFIX_OFF);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int H = p.num_heads;

    if (threadIdx.x == 32 * W_LOAD) {
        prefetch_tmap(&tmQ);
        prefetch_tmap(&tmC);
    }
    pdl_wait_primary();
    pdl_launch_dependents();
    cost_prefix(p, prefix);
    if (!p.cu) {  // no context: a zero row
        for (int s = blockIdx.x; s < p.num_seqs; s += gridDim.x) {
            if (prefix[s + 1] != prefix[s]) continue;
            uint4* o = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + (int64_t)s * H * LAT);
            for (int e = threadIdx.x; e < H * (LAT / 8); e += NTHREADS) o[e] = make_uint4(0, 0, 0, 0);
        }
    }
    const int64_t W = prefix[p.num_seqs], pairs = gridDim.x / 2, pair = blockIdx.x / 2;
    const int64_t f0 = pair * W / pairs, f1 = (pair + 1) * W / pairs;
    if (threadIdx.x == 0 && rank == 0) p.cuts[pair].rows = 0;  // (the same thread may write it again below)
    if (f0 == f1) return;  // (both CTAs of the pair)
    const Segment first = locate(p, prefix, f0, f0, f1);

    if (threadIdx.x == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(&full[i], 2u);
            mbar_init(&empty[i], 1u);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1u);
            mbar_init(&s_empty[i], 8u);
            mbar_init(&p_full[i], 8u);
            mbar_init(&p_empty[i], 1u);
        }
        mbar_init(q_full, 2u * NP);
        mbar_init(q_empty, 1u);
        mbar_init(o_empty, 8u);
        for (int i = 0; i < NP; ++i) mbar_init(&tail[i], 1u);
        *abort_flag = 0;
        mbar_fence_init();
    }
    if (warp == W_S) tmem_pair_alloc(const_cast<uint32_t*>(taddr_slot), TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *taddr_slot;
    const uint32_t sb = smem_u32(base);

    auto fail = [&]() {
        *abort_flag = 1;
        atomicOr(&g_latent_status, kStatusTimeout);
    };
    // A whole warp's bounded wait, with one answer for all lanes (every lane
    // polls: one lane's polls and a shuffle were slower).  `ready`: what an
    // earlier look told this lane.
    auto look = [&](uint64_t* bar, uint32_t parity) -> bool { return mbar_test(bar, parity); };
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
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool { return wait_after(bar, parity, look(bar, parity)); };

    // A role's place in its ring: slots [first, first + n) of the stages.
    struct Ring {
        int first, n, slot;
        uint32_t phase;  // of the current turn
        __device__ __forceinline__ void next() {
            if (++slot == first + n) slot = first, phase ^= 1;
        }
    };

    if (warp >= W_LOAD && warp < W_S) {
        // ---------------- loads: the stages of a ring go to its NP warps in turn
        const int w = (warp - W_LOAD) % NP;
        const bool values = warp >= W_LOAD + NP;
        const int br = p.box_rows, gpt = BK / br, gph = 64 / br;  // boxes per tile and chunk, per half tile
        // a lane has a box of a stage (b, of chunk c); FINE: boxes lane and
        // lane + 32 of both chunks
        const int b = lane % gph, c = lane / gph;
        const uint32_t full0 = smem_of(full, 0), tail_bar = smem_of(&tail[w], rank), q_bar = smem_of(q_full, 0);
        Ring ring = values ? Ring{NK, NV, NK, 0} : Ring{0, NK, 0, 0};
        int seg = 0, turn = 0, tail_turn = 0;
        bool run = true;
        // the next stage, and whether it is this warp's
        auto skip = [&]() -> bool {
            const bool other = turn != w;
            if (++turn == NP) turn = 0;
            if (other) ring.next();
            return other;
        };
        for (Segment s = first; run; s.next(p, f0, f1)) {
            if (s.k1 <= s.k0) break;
            const int32_t* table = p.block_tables + (int64_t)s.req * p.max_blocks;
            const int L = s.r.L;
            // pool rows of this lane's boxes of tile k: box `lane` of the
            // tile, or boxes lane and lane + 32 of each half
            auto box_rows_of = [&](int k, int32_t (&to)[4]) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    to[i] = 0;
                    if (i && !FINE) continue;
                    const int in = lane + 32 * (i & 1), tok = k * BK + 64 * (i >> 1) + in * br;
                    if (in < (FINE ? gph : gpt) && k < s.k1 && tok < L)
                        to[i] = table[tok / p.block_size] * p.block_size + tok % p.block_size;
                }
            };
            int32_t cur[4], nxt[4];
            box_rows_of(s.k0, cur);
            // boxes of half tile h, n chunks from `chunk` on, to a stage
            // (row: half_row(h))
            auto half_row = [&](int h) -> int32_t {
                return FINE ? 0 : __shfl_sync(0xffffffffu, cur[0], h * gph + b);
            };
            auto load = [&](uint8_t* st, uint32_t bar, int h, int32_t row, int boxes, int n, int chunk) {
                if (!FINE) {
                    if (c < n && b < boxes)
                        tma_load_3d_pair(st + c * CHB + b * br * 128, &tmC, bar, 0, chunk + c, row);
                    return;
                }
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (lane + 32 * e < boxes)
                        for (int i = 0; i < n; ++i)
                            tma_load_3d_pair(st + i * CHB + (lane + 32 * e) * br * 128, &tmC, bar, 0, chunk + i,
                                             h ? cur[2 + e] : cur[e]);
            };
            if (!values) {
                // the query rows of this CTA: chunks w, w + NP, ..
                if (!(run = wait(q_empty, (seg & 1) ^ 1))) break;
                const int row = s.t * TM + 64 * (int)rank, rows = min(max(s.r.rows - row, 0), 64);
                const int boxes = (rows + 15) / 16, chunks = (CH - w + NP - 1) / NP;
                if (lane == 0) {
                    if (boxes) mbar_arrive_expect_tx_at(q_bar, (uint32_t)(boxes * chunks * 16 * 128));
                    else mbar_arrive_at(q_bar);
                }
                __syncwarp();
                const int qc = w + NP * (lane / 4), g = lane % 4;
                if (qc < CH && g < boxes)
                    tma_load_3d_pair(base + Q_OFF + qc * CHB + g * 16 * 128, &tmQ, q_bar, 0, qc,
                                     (int)(s.r.row0 + row + 16 * g));
            }
            for (int k = s.k0; k < s.k1 && run; ++k) {
                box_rows_of(k + 1, nxt);
                if (!values) {
                    // this CTA's 64 keys, two chunks a stage
                    const int own = min(max(L - k * BK - 64 * (int)rank, 0), 64), boxes = (own + br - 1) / br;
                    const int32_t row = half_row((int)rank);
                    for (int c0 = 0; c0 < CH; c0 += 2) {
                        if (skip()) continue;
                        if (!(run = wait(&empty[ring.slot], ring.phase ^ 1))) break;
                        const int nc = min(2, CH - c0);
                        const uint32_t fb = full0 + 8 * ring.slot;
                        if (lane == 0) {
                            if (boxes) mbar_arrive_expect_tx_at(fb, (uint32_t)(boxes * nc * br * 128));
                            else mbar_arrive_at(fb);
                        }
                        __syncwarp();
                        load(base + ST_OFF + ring.slot * STAGE, fb, (int)rank, row, boxes, nc, c0);
                        ring.next();
                    }
                } else {
                    // this CTA's dims of all keys: (half tile, two chunks) a stage
                    const int valid = min(L - k * BK, BK), halves = valid > 64 ? 2 : 1;
                    const int rest = valid & 15;  // keys of the last, partial group of 16
                    for (int h = 0; h < halves && run; ++h) {
                        const int keys = min(valid - 64 * h, 64), boxes = (keys + br - 1) / br;
                        const bool ragged = rest != 0 && h == halves - 1;
                        const int32_t row = half_row(h);
                        for (int pc = 0; pc < 2; ++pc) {
                            if (skip()) continue;
                            if (!(run = wait(&empty[ring.slot], ring.phase ^ 1))) break;
                            const uint32_t fb = ragged ? tail_bar : full0 + 8 * ring.slot;
                            if (lane == 0) mbar_arrive_expect_tx_at(fb, (uint32_t)(boxes * 2 * br * 128));
                            __syncwarp();
                            uint8_t* st = base + ST_OFF + ring.slot * STAGE;
                            load(st, fb, h, row, boxes, 2, 4 * (int)rank + 2 * pc);
                            if (ragged) {
                                // rows past the context hold anything, and P
                                // is zero there: they are zeroed before the
                                // product reads them (only a unit's last tile
                                // has such)
                                if (!(run = wait(&tail[w], tail_turn & 1))) break;
                                ++tail_turn;
                                const int end = (keys + 15) / 16 * 16;
                                for (int i = lane; i < (end - keys) * 16; i += 32)
                                    *reinterpret_cast<uint4*>(st + ((i >> 3) & 1) * CHB + (keys + i / 16) * 128 +
                                                              (i & 7) * 16) = make_uint4(0, 0, 0, 0);
                                fence_proxy_async_smem();
                                __syncwarp();
                                if (lane == 0) mbar_arrive_at(full0 + 8 * ring.slot);
                            }
                            ring.next();
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) cur[i] = nxt[i];
            }
            ++seg;
            if (s.end() >= f1) break;
        }
        // every stage handed back, and the last queries read: no arrival is
        // still on its way to this CTA
        for (int i = 0; i < ring.n && run; ++i) {
            run = wait(&empty[ring.slot], ring.phase ^ 1);
            ring.next();
        }
        if (run && !values) run = wait(q_empty, (seg & 1) ^ 1);
    } else if (warp == W_S) {
        // ---------------- S = Q K^T (even CTA)
        if (rank == 0) {
            constexpr uint32_t idS = umma_idesc_f16(128, BK, kBF16, false);
            Ring ring{0, NK, 0, 0};
            int seg = 0, it = 0;
            bool run = true;
            // operands as lane 0 has them: in uniform registers
            const uint32_t tm0 = lane0(tmem), q_lo = lane0(((sb + Q_OFF) & 0x3ffffu) >> 4 | 1u << 16);
            const uint32_t st_lo = lane0(((sb + ST_OFF) & 0x3ffffu) >> 4 | 1u << 16);
            for (Segment s = first; run; s.next(p, f0, f1)) {
                if (s.k1 <= s.k0) break;
                if (!(run = wait(q_full, seg & 1))) break;
                bool ready = look(&full[ring.slot], ring.phase);
                for (int k = s.k0; k < s.k1 && run; ++k, ++it) {
                    const int buf = it & 1;
                    const uint32_t d = lane0(tm0 + S_COL + 64 * buf);
                    if (!(run = wait(&s_empty[buf], ((it >> 1) & 1) ^ 1))) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c0 = 0; c0 < CH; c0 += 2) {  // (short loops: instructions are fetched once)
                        if (!(run = wait_after(&full[ring.slot], ring.phase, ready))) break;
                        const uint32_t a = lane0(q_lo + c0 * (CHB / 16)), b = lane0(st_lo + ring.slot * (STAGE / 16));
                        const uint32_t old = lane0(c0 ? 1u : 0u);
                        const bool two = c0 + 2 <= CH;
                        uint64_t* done = &empty[ring.slot];
                        ring.next();
                        ready = look(&full[ring.slot], ring.phase);  // (looked at while the MMAs go out)
                        if (elect_lane()) {
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk) {
                                if (kk == 4 && !two) break;
                                const uint32_t off = ((kk >> 2) * CHB + (kk & 3) * 32) / 16;
                                umma_pair_f16(d, sw128_desc(a + off), sw128_desc(b + off), idS, kk ? 1u : old);
                            }
                            umma_pair_commit(done);
                            if (c0 + 2 >= CH) {
                                umma_pair_commit(&s_full[buf]);
                                if (k == s.k1 - 1) umma_pair_commit(q_empty);
                            }
                        }
                        __syncwarp();
                    }
                }
                ++seg;
                if (s.end() >= f1) break;
            }
        }
    } else if (warp == W_O) {
        // ---------------- O += P C (even CTA)
        if (rank == 0) {
            constexpr uint32_t idO = umma_idesc_f16(128, 256, kBF16, true);
            Ring ring{NK, NV, NK, 0};
            int seg = 0, it = 0;
            bool run = true;
            const uint32_t tm0 = lane0(tmem), p_lo = lane0(((sb + P_OFF) & 0x3ffffu) >> 4 | 1u << 16);
            const uint32_t st_lo = lane0(((sb + ST_OFF) & 0x3ffffu) >> 4 | (CHB / 16) << 16);
            for (Segment s = first; run; s.next(p, f0, f1)) {
                if (s.k1 <= s.k0) break;
                if (!(run = wait(o_empty, (seg & 1) ^ 1))) break;
                for (int k = s.k0; k < s.k1 && run; ++k, ++it) {
                    const int buf = it & 1;
                    bool ready = look(&full[ring.slot], ring.phase);
                    if (!(run = wait(&p_full[buf], (it >> 1) & 1))) break;
                    tc_fence_after();
                    const int valid = min(s.r.L - k * BK, BK), nks = (valid + 15) / 16;
                    const int halves = valid > 64 ? 2 : 1;
                    for (int h = 0; h < halves && run; ++h)
#pragma unroll 1
                        for (int pc = 0; pc < 2; ++pc) {
                            if (!(run = wait_after(&full[ring.slot], ring.phase, ready))) break;
                            const uint32_t a = lane0(p_lo + (2 * buf + h) * (CHB / 16)), d = lane0(tm0 + O_COL + 128 * pc);
                            const uint32_t b = lane0(st_lo + ring.slot * (STAGE / 16));
                            const uint32_t old = lane0(k > s.k0 || h ? 1u : 0u);
                            uint64_t* done = &empty[ring.slot];
                            ring.next();
                            ready = look(&full[ring.slot], ring.phase);
                            if (elect_lane()) {
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    if (4 * h + j >= nks) break;
                                    umma_pair_f16(d, sw128_desc(a + 2 * j), sw128_desc(b + j * 128), idO, j ? 1u : old);
                                }
                                umma_pair_commit(done);
                                if (h == halves - 1 && pc == 1) umma_pair_commit(&p_empty[buf]);
                            }
                            __syncwarp();
                        }
                }
                ++seg;
                if (s.end() >= f1) break;
            }
        }
    } else {
        // ---------------- softmax: row r of this CTA's 64, keys 64 hf .. of each tile
        const int tid = threadIdx.x, hf = warp >> 1, r = (warp & 1) * 32 + lane;
        const uint32_t t_lane = tmem + ((uint32_t)(warp * 32) << 16);
        const float scale = p.scale_log2 == 0.f ? 1e-38f : p.scale_log2;  // (0: every score counts alike)
        const float hidden = scale > 0.f ? -INFINITY : INFINITY;
        const uint32_t s_empty0 = smem_of(s_empty, 0), p_full0 = smem_of(p_full, 0), o_empty0 = smem_of(o_empty, 0);
        int it = 0, seg = 0;
        bool ok = true;
        for (Segment s = first;; s.next(p, f0, f1)) {
            if (s.k1 <= s.k0) break;
            const int row = s.t * TM + 64 * (int)rank + r;
            const bool mine = row < s.r.rows;
            const bool some = __any_sync(0xffffffffu, mine);  // (of these 32 rows: the partner warp's too)
            const int vis = p.causal ? min(s.r.L, s.r.before + min(row, s.r.rows - 1) / H + 1) : s.r.L;
            int vmin = vis;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) vmin = min(vmin, __shfl_xor_sync(0xffffffffu, vmin, o));
            float m = -INFINITY, l = 0.f;
            for (int k = s.k0; k < s.k1; ++k, ++it) {
                const int buf = it & 1;
                const uint32_t turn = (it >> 1) & 1;
                // the scores, and P of two tiles ago read
                if (ok) ok = wait(&s_full[buf], turn);
                if (ok) ok = wait(&p_empty[buf], turn ^ 1);
                if (ok) tc_fence_after();
                const int key0 = k * BK + 64 * hf;
                const bool masked = key0 + 64 > vmin;
                // this thread's scores 32 c ..; those it may not see end at -inf once scaled
                auto scores = [&](int c, float (&x)[32]) {
                    tmem_ld32(t_lane + S_COL + 64 * buf + 32 * c, x);
                    tmem_wait_ld();
                    if (masked) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] = key0 + 32 * c + i < vis ? x[i] : hidden;
                    }
                };
                // P is taken against the row's reference as it stands: a sum of
                // at most 2^8 proves that no score is more than 8 above it.
                // Otherwise (and on a segment's first tile) the partners swap
                // their maxima, the reference moves, and P is taken again.
                bool move = k == s.k0;
                float alpha = 1.f, sum = 0.f;
                while (true) {
                    if (move) {
                        float mx = -INFINITY;
                        if (ok && some) {
#pragma unroll 1
                            for (int c = 0; c < 2; ++c) {
                                float x[32];
                                scores(c, x);
#pragma unroll
                                for (int i = 0; i < 32; ++i) mx = fmaxf(mx, x[i] * scale);
                            }
                        }
                        xch[buf * 128 + tid] = mx;
                        ok = bar_all(1, 128, ok);  // all four warps go on, or none
                        if (!ok) break;
                        mx = fmaxf(mx, xch[buf * 128 + (tid ^ 64)]);
                        if (mine && (mx > m + 8.f || (m == -INFINITY && mx > m))) {
                            alpha = fast_exp2(m - mx);  // (0 where nothing was seen yet)
                            m = mx;
                        }
                    }
                    const float ms = m == -INFINITY ? 0.f : m;
                    if (ok && some) {
                        const unsigned long long sc2 = f32x2_pack(scale, scale), off2 = f32x2_pack(-ms, -ms);
                        unsigned long long sum2 = 0ull;
                        uint32_t dst = sb + P_OFF + (2 * buf + hf) * CHB + r * 128, piece = r & 7;
#pragma unroll 1
                        for (int c = 0; c < 2; ++c, piece ^= 4) {
                            float x[32];
                            scores(c, x);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                uint32_t pk[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    float a, b;
                                    const int i = 8 * j + 2 * e;
                                    f32x2_unpack(fma_f32x2(f32x2_pack(x[i], x[i + 1]), sc2, off2), a, b);
                                    a = fast_exp2(a);
                                    b = fast_exp2(b);
                                    sum2 = add_f32x2(sum2, f32x2_pack(a, b));
                                    pk[e] = pack2<T>(a, b);
                                }
                                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + ((piece ^ j) << 4)),
                                             "r"(pk[0]), "r"(pk[1]), "r"(pk[2]), "r"(pk[3])
                                             : "memory");
                            }
                        }
                        float sa, sb2;
                        f32x2_unpack(sum2, sa, sb2);
                        sum = sa + sb2;
                    }
                    if (move || bar_all(1, 128, ok && (!mine || (sum <= 256.f && m != -INFINITY)))) break;
                    move = true;
                }
                if (!ok) break;
                l = fmaf(l, alpha, sum);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_at(s_empty0 + 8 * buf);
                fence_proxy_async_smem();
                if (k > s.k0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                    // O holds the tiles before this one
                    ok = wait(&p_empty[buf ^ 1], ((it - 1) >> 1) & 1);
                    if (ok) {
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < 256; c += 32) {
                            float o[32];
                            tmem_ld32(t_lane + O_COL + c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] *= alpha;
                            tmem_st32(t_lane + O_COL + c, o);
                        }
                        tmem_wait_st();
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (ok && lane == 0) mbar_arrive_at(p_full0 + 8 * buf);
            }
            // the segment's last product
            if (ok) ok = wait(&p_empty[(it - 1) & 1], ((it - 1) >> 1) & 1);
            xch[(it & 1) * 128 + tid] = l;
            ok = bar_all(1, 128, ok);
            if (!ok) break;
            tc_fence_after();
            l += xch[(it & 1) * 128 + (tid ^ 64)];
            const bool whole = s.k0 == 0 && s.k1 == s.nk;
            const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
            // The rows go out through P's place, 8 KB a warp (P of this segment
            // is read, and the next segment's first tile has a barrier of the
            // four warps before P): written a row per lane, 16 of 16 bytes at a
            // time, they are stored 256 bytes of a row together.  Stored
            // straight from the lanes a tile took 9,500 cycles.
            const int row0 = row - lane, rows = min(max(s.r.rows - row0, 0), 32);  // of this warp
            uint8_t* stage = base + P_OFF + warp * CHB;
            const int half = lane >> 4, u = lane & 15;
            if (whole) {
                T* o0 = static_cast<T*>(p.out) + (s.r.row0 + row0) * LAT + 256 * hf;
#pragma unroll 1
                for (int c = 0; c < 256; c += 128) {
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        float o[32];
                        tmem_ld32(t_lane + O_COL + c + 32 * q, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            *reinterpret_cast<uint4*>(stage + lane * 256 + (((4 * q + j) ^ (lane & 7)) << 4)) =
                                make_uint4(pack2<T>(o[8 * j] * inv, o[8 * j + 1] * inv),
                                           pack2<T>(o[8 * j + 2] * inv, o[8 * j + 3] * inv),
                                           pack2<T>(o[8 * j + 4] * inv, o[8 * j + 5] * inv),
                                           pack2<T>(o[8 * j + 6] * inv, o[8 * j + 7] * inv));
                    }
                    __syncwarp();
#pragma unroll 4
                    for (int i = half; i < rows; i += 2)
                        *reinterpret_cast<uint4*>(o0 + (int64_t)i * LAT + c + 8 * u) =
                            *reinterpret_cast<const uint4*>(stage + i * 256 + ((u ^ (i & 7)) << 4));
                    __syncwarp();
                }
            } else {
                float* rec = p.records + ((2 * pair + s.slot()) * p.rec_rows + (row0 - s.t * TM)) * (int64_t)REC;
                if (threadIdx.x == 0 && rank == 0 && s.k0 == 0) {
                    Cut cut;
                    cut.rows = min(s.r.rows - s.t * TM, TM);
                    cut.last = (int)((s.end() * pairs + W - 1) / W) - 1;  // of the pair owning its last place
                    cut.cost = (int)W;
                    cut.row0 = s.r.row0 + s.t * TM;
                    p.cuts[pair] = cut;
                }
                if (mine && hf == 0) {
                    rec[(int64_t)lane * REC + LAT] = m;
                    rec[(int64_t)lane * REC + LAT + 1] = l;
                }
                rec += 256 * hf;
#pragma unroll 1
                for (int c = 0; c < 256; c += 64) {
#pragma unroll 1
                    for (int q = 0; q < 2; ++q) {
                        float o[32];
                        tmem_ld32(t_lane + O_COL + c + 32 * q, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            *reinterpret_cast<float4*>(stage + lane * 256 + (((8 * q + j) ^ (lane & 7)) << 4)) =
                                make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                    }
                    __syncwarp();
#pragma unroll 4
                    for (int i = half; i < rows; i += 2)
                        *reinterpret_cast<float4*>(rec + (int64_t)i * REC + c + 4 * u) =
                            *reinterpret_cast<const float4*>(stage + i * 256 + ((u ^ (i & 7)) << 4));
                    __syncwarp();
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_at(o_empty0);
            ++seg;
            if (s.end() >= f1) break;
        }
    }

    // After a wait that ran out: the copies in flight are given time to land
    // before the shared memory is let go.
    __syncwarp();
    if (*abort_flag && warp == W_S) {
        const uint64_t t0 = global_ns();
        while (global_ns() - t0 < 1000000ull) {}
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    if (warp == W_S) tmem_pair_dealloc(tmem, TMEM_COLS);
}

// Joins the records of the units cut between pairs: a warp folds every step-th
// record of a row (o: 16 of its dims, the warp's lanes beside each other), B of
// them in flight.
struct Joined {
    float M = -INFINITY, l = 0.f;
    float4 o[4] = {};
};
__device__ __forceinline__ Joined join_records(const Params& p, int pairs, int c, int row, const int4 cut, int from,
                                               int step) {
    constexpr int B = 4;
    const int lane = threadIdx.x & 31, last = cut.y;
    const int64_t W = cut.z;
    Joined j;
    for (int q0 = c + from; q0 <= last; q0 += B * step) {
        float m[B], lq[B];
        float4 a[B][4];
#pragma unroll
        for (int k = 0; k < B; ++k) {
            const int q = q0 + k * step;
            const bool there = q <= last && (W >= pairs || q * W / pairs != (q + 1) * W / pairs);  // (no empty run)
            const float* rec = p.records + ((2ll * q + (q == c ? 1 : 0)) * p.rec_rows + row) * REC;
            m[k] = there ? __ldcg(rec + LAT) : -INFINITY;
            lq[k] = there ? __ldcg(rec + LAT + 1) : 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                a[k][i] = there ? __ldcg(reinterpret_cast<const float4*>(rec) + 32 * i + lane)
                                : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float mn = j.M;
#pragma unroll
        for (int k = 0; k < B; ++k) mn = fmaxf(mn, m[k]);
        const float ms = mn == -INFINITY ? 0.f : mn, e0 = exp2f(j.M - ms);
        j.l *= e0;
#pragma unroll
        for (int i = 0; i < 4; ++i) j.o[i] = make_float4(j.o[i].x * e0, j.o[i].y * e0, j.o[i].z * e0, j.o[i].w * e0);
#pragma unroll
        for (int k = 0; k < B; ++k) {
            const float e = exp2f(m[k] - ms);
            j.l = fmaf(lq[k], e, j.l);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                j.o[i].x = fmaf(a[k][i].x, e, j.o[i].x);
                j.o[i].y = fmaf(a[k][i].y, e, j.o[i].y);
                j.o[i].z = fmaf(a[k][i].z, e, j.o[i].z);
                j.o[i].w = fmaf(a[k][i].w, e, j.o[i].w);
            }
        }
        j.M = mn;
    }
    return j;
}

// CTA (c, g): the unit that pair c begins, rows 4 g .. 4 g + 3, a warp each
// (small CTAs: they are resident beside the kernel whose end they wait for).
template <typename T>
__global__ void __launch_bounds__(128) latent_merge_kernel(const Params p, int pairs) {
    pdl_wait_primary();
    pdl_launch_dependents();
    const int c = blockIdx.x, row = blockIdx.y * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int4 cut = __ldcg(reinterpret_cast<const int4*>(p.cuts + c));
    if (row >= cut.x) return;
    const int64_t row0 = __ldcg(&p.cuts[c].row0);
    const Joined j = join_records(p, pairs, c, row, cut, 0, 1);
    const float inv = j.l == 0.f ? 0.f : 1.f / j.l;
    T* out = static_cast<T*>(p.out) + (row0 + row) * LAT;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint2*>(out + 128 * i + 4 * lane) =
            make_uint2(pack2<T>(j.o[i].x * inv, j.o[i].y * inv), pack2<T>(j.o[i].z * inv, j.o[i].w * inv));
}

// The same for units in many pieces: a CTA per row, whose eight warps fold every
// eighth record each and then their results in order (a row's warp reading 75
// records of 2 KB by itself took 18 us: 1 x 32,768 tokens of 16 heads 45.7 ->
// 33.4 us, 1 x 1,999 17.4 -> 15.9; 8 x 32,768, nine pieces each, 72 either way).
template <typename T>
__global__ void __launch_bounds__(256) latent_merge_many_kernel(const Params p, int pairs) {
    __shared__ float4 part[8][LAT / 4];
    __shared__ float2 ml[8];
    pdl_wait_primary();
    pdl_launch_dependents();
    const int c = blockIdx.x, row = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int4 cut = __ldcg(reinterpret_cast<const int4*>(p.cuts + c));
    if (row >= cut.x) return;
    const int64_t row0 = __ldcg(&p.cuts[c].row0);
    const Joined j = join_records(p, pairs, c, row, cut, warp, 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) part[warp][32 * i + lane] = j.o[i];
    if (lane == 0) ml[warp] = make_float2(j.M, j.l);
    __syncthreads();
    float M = -INFINITY, l = 0.f, x = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) M = fmaxf(M, ml[w].x);
    const float ms = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        const float e = exp2f(ml[w].x - ms);
        const float2 v = reinterpret_cast<const float2*>(part[w])[threadIdx.x];
        l = fmaf(ml[w].y, e, l);
        x = fmaf(v.x, e, x);
        y = fmaf(v.y, e, y);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    reinterpret_cast<uint32_t*>(static_cast<T*>(p.out) + (row0 + row) * LAT)[threadIdx.x] = pack2<T>(x * inv, y * inv);
}

// ---------------------------------------------------------------- host side

// Rows of a box: as many as lie together in every block, up to half a tile.
// (A box need not fill the eight rows of a swizzle pattern, which goes by the
// address.)
int box_rows(int block_size) {
    int n = 64;
    while (block_size % n) n /= 2;
    return n;
}

// Pairs of SMs that run at once.  Not every two SMs are a pair (a cluster lies
// within one part of the GPU): with a pair for every two of the 152 SMs a few
// ran after the others and the kernel took twice as long.  Asked once a device.
int resident_pairs(const void* kernel) {
    constexpr int kDevices = 64;
    static std::atomic<int> known[kDevices];
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < kDevices && known[dev].load(std::memory_order_relaxed)) return known[dev].load(std::memory_order_relaxed);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * kPairs);
    cfg.blockDim = dim3(NTHREADS);
    cfg.dynamicSmemBytes = smem_bytes(kMaxSeqs);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();
        return kPairs / 2;  // (asked again by the next call)
    }
    n = std::min(n, kPairs);
    if (dev < kDevices) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

template <typename T>
cudaError_t launch_typed(const LatentArgs& a, int32_t num_blocks, void* workspace, int rec_rows, std::string* err,
                         cudaStream_t stream) {
    const CUtensorMapDataType ty = a.dtype == 1 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const int64_t rows = (int64_t)a.total_q * a.num_heads;
    CUtensorMap tmQ, tmC;
    const cuuint64_t strides[2] = {128, D * 2};
    const cuuint64_t qdims[3] = {64, CH, (cuuint64_t)rows};
    const cuuint32_t qbox[3] = {64, 1, 16};
    const cuuint64_t cdims[3] = {64, CH, (cuuint64_t)num_blocks * a.block_size};
    const cuuint32_t cbox[3] = {64, 1, (cuuint32_t)box_rows(a.block_size)};
    if (!encode_tiled_3d(&tmQ, ty, a.q, qdims, strides, qbox, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, err) ||
        !encode_tiled_3d(&tmC, ty, a.cache, cdims, strides, cbox, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, err))
        return cudaErrorInvalidValue;
    Params p;
    p.out = a.out;
    p.block_tables = a.block_tables;
    p.max_blocks = a.max_blocks;
    p.seq_lens = a.seq_lens;
    p.cu = a.cu;
    p.num_seqs = a.num_seqs;
    p.num_heads = a.num_heads;
    p.block_size = a.block_size;
    p.box_rows = box_rows(a.block_size);
    p.causal = a.causal;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.records = static_cast<float*>(workspace);
    p.cuts = reinterpret_cast<Cut*>(p.records + (int64_t)2 * kPairs * rec_rows * REC);
    p.rec_rows = rec_rows;
    // every pair there is, fewer where even the longest contexts give them less
    // than one tile each
    const int64_t units = a.cu ? rows / TM + a.num_seqs : (int64_t)a.num_seqs * ((a.num_heads + TM - 1) / TM);
    const int64_t tiles = units * (((int64_t)a.max_context + BK - 1) / BK);
    const auto kernel = p.box_rows < 4 ? (a.cu ? latent_umma_kernel<T, false, true> : latent_umma_kernel<T, true, true>)
                                       : (a.cu ? latent_umma_kernel<T, false, false> : latent_umma_kernel<T, true, false>);
    const void* kfn = reinterpret_cast<const void*>(kernel);
    cudaError_t e = allow_smem(kfn, smem_bytes(kMaxSeqs));
    if (e != cudaSuccess) return e;
    const int pairs = (int)std::max<int64_t>(1, std::min<int64_t>(resident_pairs(kfn), tiles));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * pairs));
    cfg.blockDim = dim3(NTHREADS);
    cfg.dynamicSmemBytes = smem_bytes(a.num_seqs);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, kernel, tmQ, tmC, p);
    if (e != cudaSuccess || pairs == 1) return e;
    // units in more than eight pieces on average: a CTA a row (see there)
    if (pairs > 8 * units)
        return launch_pdl(latent_merge_many_kernel<T>, dim3((unsigned)(pairs - 1), (unsigned)rec_rows), dim3(256),
                          stream, p, pairs);
    return launch_pdl(latent_merge_kernel<T>, dim3((unsigned)(pairs - 1), (unsigned)((rec_rows + 3) / 4)), dim3(128),
                      stream, p, pairs);
}

}  // namespace

bool latent_umma_supported(int dtype, int32_t latent_dim, int32_t rope_dim, int32_t block_size) {
    return (dtype == 1 || dtype == 2) && latent_dim == LAT && rope_dim == ROT &&
           block_size > 0;
}

size_t latent_umma_workspace(int64_t rows) {
    return (size_t)2 * kPairs * (size_t)std::min<int64_t>(rows, TM) * REC * sizeof(float) + kPairs * sizeof(Cut);
}

cudaError_t launch_latent_umma(const LatentArgs& a, int32_t num_blocks, void* workspace, std::string* err,
                               cudaStream_t stream) {
    if (a.total_q == 0 || a.num_seqs == 0) return cudaSuccess;
    // rows of a tile (of one token in a decode)
    const int rec_rows = (int)std::min<int64_t>((int64_t)(a.cu ? a.total_q : 1) * a.num_heads, TM);
    for (int32_t s0 = 0; s0 < a.num_seqs; s0 += kMaxSeqs) {
        LatentArgs c = a;
        c.num_seqs = std::min(a.num_seqs - s0, kMaxSeqs);
        c.seq_lens = a.seq_lens + s0;
        c.block_tables = a.block_tables + (int64_t)s0 * a.max_blocks;
        if (a.cu) {  // query rows keep their numbers
            c.cu = a.cu + s0;
        } else {
            c.total_q = c.num_seqs;
            c.q = static_cast<const uint8_t*>(a.q) + (int64_t)s0 * a.num_heads * D * 2;
            c.out = static_cast<uint8_t*>(a.out) + (int64_t)s0 * a.num_heads * LAT * 2;
        }
        cudaError_t e = a.dtype == 1 ? launch_typed<__nv_bfloat16>(c, num_blocks, workspace, rec_rows, err, stream)
                                     : launch_typed<__half>(c, num_blocks, workspace, rec_rows, err, stream);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

uint32_t latent_umma_status(bool clear) {
    unsigned int v = 0;
    cudaMemcpyFromSymbol(&v, g_latent_status, sizeof(v));
    if (clear) {
        const unsigned int z = 0;
        cudaMemcpyToSymbol(g_latent_status, &z, sizeof(z));
    }
    return v;
}

}  // namespace pa
