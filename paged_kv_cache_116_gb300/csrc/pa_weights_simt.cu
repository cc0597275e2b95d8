// pa_weights_simt.cu -- attention weights of a request's cached tokens on the
// CUDA cores: any element type, head_dim up to 256, any block size, 16-bit or
// fp32 pools and E4M3 code pools.
//
// For request s the last `window` of its n new tokens (all n where window is
// 0) are the query rows; row (i, g) of KV head h is query head h G + g of new
// token i, at position L - n + i, and sees the keys up to it (causal) or all
// L.  With p the row's softmax over the keys it sees, token j of the request
// gets
//   w(j) = sum over rows (i, g) of p(j),
// added to weights[s, h, j] for a token that was cached before this call
// (j < L - n) and stored there for a new one.
//
// The row normalisers have to be known before any weight can be summed, so
// the work is two passes over Q K^T, each a product of 64-row by 64-key tiles
// in fp32 (64 x 64 x 32 steps, 4 x 4 accumulators per thread):
//   pass 1  one CTA per (request, KV head, 64 rows) walks the keys with an
//           online maximum and sum and stores (max, 1 / sum) per row;
//   pass 2  one CTA per (request, KV head, 64 keys) walks the rows that see
//           them and sums exp2(x - max) / sum per key in fp32.
// Each weight has one owner and a fixed order of summation: no atomics, and
// the same bits from every run.  The subtraction x - max comes before the
// division by the sum (rather than one exponent x - log-sum-exp) because a
// log-sum-exp rounded to fp32 would cost |lse| 2^-24 relative in every
// weight.
// Bound: fp32 FMA issue, with both operands from shared memory.
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_launch.cuh"
#include "pa_weights.cuh"

namespace pa {
namespace {

constexpr int TR = 64, TK = 64, KC = 32, NTH = 256;

template <typename T, bool FP8> struct PoolElt {
    using S = T;
    static __device__ __forceinline__ float to_f(S x) { return Elt<T>::to_f(x); }
};
template <typename T> struct PoolElt<T, true> {
    using S = uint8_t;
    static __device__ __forceinline__ float to_f(S x) {
        return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)x, __NV_E4M3)));
    }
};

struct Tile {
    float q[TR][KC + 1];
    float k[TK][KC + 1];
};

// x[i][j] = log2(e) * scale * (row ty + 16 i) . (key tx + 16 j)
template <typename T, bool FP8>
__device__ __forceinline__ void scores(const WeightArgs& a, const WeightSeq& sq, int h, int r0, int k0, Tile& tl,
                                       float (&x)[4][4]) {
    using P = PoolElt<T, FP8>;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, hd = a.head_dim;
    const int G = a.num_heads / a.num_kv_heads;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][j] = 0.f;
    const int32_t* table = a.block_tables + (int64_t)sq.s * a.max_blocks;
    for (int d0 = 0; d0 < hd; d0 += KC) {
        __syncthreads();
        for (int e = threadIdx.x; e < TR * KC; e += NTH) {
            const int r = e / KC, d = d0 + e % KC, row = r0 + r;
            float v = 0.f;
            if (row < sq.rows * G && d < hd)
                v = Elt<T>::to_f(static_cast<const T*>(a.q)[((int64_t)(sq.row0 + row / G) * a.num_heads + h * G +
                                                             row % G) * hd + d]);
            tl.q[r][e % KC] = v;
        }
        for (int e = threadIdx.x; e < TK * KC; e += NTH) {
            const int c = e / KC, d = d0 + e % KC, t = k0 + c;
            float v = 0.f;
            if (t < sq.L && d < hd) {
                const int64_t slot = (int64_t)table[t / a.block_size] * a.block_size + t % a.block_size;
                v = P::to_f(static_cast<const typename P::S*>(a.k_cache)[(slot * a.num_kv_heads + h) * hd + d]);
            }
            tl.k[c][e % KC] = v;
        }
        __syncthreads();
#pragma unroll 8
        for (int d = 0; d < KC; ++d) {
            float qv[4], kv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) qv[i] = tl.q[ty + 16 * i][d];
#pragma unroll
            for (int j = 0; j < 4; ++j) kv[j] = tl.k[tx + 16 * j][d];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) x[i][j] = fmaf(qv[i], kv[j], x[i][j]);
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float m = a.scale_log2;
        if constexpr (FP8) {
            const int t = min(k0 + tx + 16 * j, sq.L - 1);
            m *= a.k_scales[((int64_t)table[t / a.block_size] * a.num_kv_heads + h) * a.block_size + t % a.block_size];
        }
        // rounded here: contracted with a subtraction of the maximum in one pass
        // and not in the other, a row's weights would be off by half a unit of
        // its scores (1e-4 at scores of 4,000)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i][j] = __fmul_rn(x[i][j], m);
    }
}

// The keys that flat row r (token r / G) of the request sees.
__device__ __forceinline__ int visible(const WeightArgs& a, const WeightSeq& sq, int r, int G) {
    if (r >= sq.rows * G) return 0;
    return a.causal ? sq.L - sq.rows + r / G + 1 : sq.L;
}

template <typename T, bool FP8>
__global__ void __launch_bounds__(NTH) row_stats_kernel(const WeightArgs a) {
    __shared__ Tile tl;
    extern __shared__ int32_t prefix[];
    pdl_wait_primary();
    pdl_launch_dependents();
    const int G = a.num_heads / a.num_kv_heads, Hkv = a.num_kv_heads;
    work_prefix(a, prefix, [&](const WeightSeq& sq) { return (sq.rows * G + TR - 1) / TR; });
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int64_t items = (int64_t)prefix[a.num_seqs] * Hkv;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        int s, h, tile;
        locate_work(prefix, a.num_seqs, Hkv, it, s, h, tile);
        const WeightSeq sq = weight_seq(a, s);
        const int r0 = tile * TR;
        int vis[4], top = 0;
        float m[4], l[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            vis[i] = visible(a, sq, r0 + ty + 16 * i, G);
            m[i] = -INFINITY;
            l[i] = 0.f;
        }
        top = visible(a, sq, min(r0 + TR, sq.rows * G) - 1, G);
        for (int k0 = 0; k0 < top; k0 += TK) {
            float x[4][4];
            scores<T, FP8>(a, sq, h, r0, k0, tl, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float mx = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (k0 + tx + 16 * j >= vis[i]) x[i][j] = -INFINITY;
                    mx = fmaxf(mx, x[i][j]);
                }
#pragma unroll
                for (int o = 1; o < 16; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                const float mn = fmaxf(m[i], mx), ms = mn == -INFINITY ? 0.f : mn;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) sum += exp2f(x[i][j] - ms);
                l[i] = l[i] * exp2f(m[i] - ms) + sum;
                m[i] = mn;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
            const int r = r0 + ty + 16 * i;
            if (tx == 0 && r < sq.rows * G)
                a.stats[(int64_t)(sq.stat0 + r / G) * a.num_heads + h * G + r % G] =
                    make_float2(m[i] == -INFINITY ? 0.f : m[i], 1.f / l[i]);
        }
    }
}

template <typename T, bool FP8>
__global__ void __launch_bounds__(NTH) key_weights_kernel(const WeightArgs a) {
    __shared__ Tile tl;
    __shared__ float part[16][TK];
    extern __shared__ int32_t prefix[];
    pdl_wait_primary();
    pdl_launch_dependents();
    const int G = a.num_heads / a.num_kv_heads, Hkv = a.num_kv_heads;
    work_prefix(a, prefix, [&](const WeightSeq& sq) { return sq.rows ? (sq.L + TK - 1) / TK : 0; });
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int64_t items = (int64_t)prefix[a.num_seqs] * Hkv;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        int s, h, tile;
        locate_work(prefix, a.num_seqs, Hkv, it, s, h, tile);
        const WeightSeq sq = weight_seq(a, s);
        const int k0 = tile * TK;
        // the first row that sees key k0
        const int first = a.causal ? max(0, k0 - (sq.L - sq.rows)) * G : 0;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        for (int r0 = first / TR * TR; r0 < sq.rows * G; r0 += TR) {
            float x[4][4];
            scores<T, FP8>(a, sq, h, r0, k0, tl, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = r0 + ty + 16 * i, vis = visible(a, sq, r, G);
                if (vis <= k0) continue;
                const float2 st = a.stats[(int64_t)(sq.stat0 + r / G) * a.num_heads + h * G + r % G];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (k0 + tx + 16 * j < vis) sum[j] = fmaf(exp2f(x[i][j] - st.x), st.y, sum[j]);
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j) part[ty][tx + 16 * j] = sum[j];
        __syncthreads();
        if (threadIdx.x < TK && k0 + threadIdx.x < sq.L) {
            float w = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) w += part[i][threadIdx.x];
            const int t = k0 + threadIdx.x;
            float* dst = a.weights + ((int64_t)s * Hkv + h) * a.weights_stride + t;
            *dst = t < sq.L - sq.n ? *dst + w : w;
        }
    }
}

template <typename T, bool FP8>
cudaError_t launch_weights_typed(const WeightArgs& a, cudaStream_t stream) {
    const int sms = sm_count();
    const int G = a.num_heads / a.num_kv_heads;
    const int64_t row_items = std::min<int64_t>(
        ((int64_t)a.total_q * G + TR - 1) / TR + a.num_seqs, (int64_t)1 << 20) * a.num_kv_heads;
    const int64_t key_items = (int64_t)a.num_seqs * a.num_kv_heads * ((a.max_context + TK - 1) / TK);
    const size_t smem = (size_t)(a.num_seqs + 1) * sizeof(int32_t);
    auto grid = [&](int64_t items) { return dim3((unsigned)std::max<int64_t>(1, std::min<int64_t>(items, sms * 8))); };
    cudaError_t e = launch_pdl_smem(row_stats_kernel<T, FP8>, grid(row_items), dim3(NTH), smem, stream, a);
    if (e != cudaSuccess) return e;
    return launch_pdl_smem(key_weights_kernel<T, FP8>, grid(key_items), dim3(NTH), smem, stream, a);
}

}  // namespace

cudaError_t launch_weights_simt(const WeightArgs& a, cudaStream_t stream) {
    switch (a.dtype) {
        case 0: return a.kv_fp8 ? launch_weights_typed<float, true>(a, stream) : launch_weights_typed<float, false>(a, stream);
        case 1: return a.kv_fp8 ? launch_weights_typed<__nv_bfloat16, true>(a, stream)
                                : launch_weights_typed<__nv_bfloat16, false>(a, stream);
        default: return a.kv_fp8 ? launch_weights_typed<__half, true>(a, stream)
                                 : launch_weights_typed<__half, false>(a, stream);
    }
}

}  // namespace pa
