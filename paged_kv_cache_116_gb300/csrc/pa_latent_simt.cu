// pa_latent_simt.cu -- CUDA-core attention over a latent cache, for every
// element type and rows of up to 576 elements: the path of fp32 (whose bound
// rules out 16-bit operands) and of shapes the tensor-core kernel does not
// take.
//
// Row t of the cache is [c_t | r_t] (latent_dim and rope_dim elements).  For
// query row i of head h:
//   x_t = scale * q[i, h] . [c_t | r_t],  p = softmax(x),  out[i, h] = sum p_t c_t
// over the keys the row sees: every head's key is the whole row and its value
// the row's latent part, so a row is read once for all the CTA's heads and for
// both products.
//
// One CTA of four warps per (query row, 16 heads), and per piece of the keys
// where there are too few rows to fill the GPU: the rows of eight keys at a time
// go through shared memory, three stages ahead (cp.async; element by element
// where rows are no multiple of 16 bytes), and are read there by every warp, each
// with four heads of its own: lanes split the row's elements, two keys are worked
// at once.  With eight heads or fewer the warps share out the keys instead and
// their states are joined at the end, in order; pieces leave (o, m, l) records
// that latent_simt_join_kernel joins in order.  Bound: the issue of instructions
// with two warps a scheduler (180 registers hold four heads' queries and sums).
// 64 x 2,048 fp32 tokens of 16 heads 245 us (409 with a row at a time straight
// from memory for four heads a CTA, 289 with every lane taking all weights), 1 x
// 32,768 107 (255); bf16, 256 + 32 elements, 64 x 2,048: 183 (348).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_launch.cuh"

namespace pa {
namespace {

// Two neighbouring elements of shared memory.
__device__ __forceinline__ unsigned long long pair_of(const float* x) {
    const float2 v = *reinterpret_cast<const float2*>(x);
    return f32x2_pack(v.x, v.y);
}
__device__ __forceinline__ unsigned long long pair_of(const __nv_bfloat16* x) {
    const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(x));
    return f32x2_pack(v.x, v.y);
}
__device__ __forceinline__ unsigned long long pair_of(const __half* x) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(x));
    return f32x2_pack(v.x, v.y);
}

constexpr int kWarps = 4;
constexpr int GH = 4;                // heads per warp
constexpr int HEADS = GH * kWarps;   // heads per CTA
constexpr int KEYS = 8, STAGES = 4;  // keys per stage
constexpr int kMaxSplits = kSms; // pieces of a row

// DPL: elements of a row per lane, in pairs (2 lane + 64 j).
// splits pieces of each row's keys; records (splits > 1): [rows][heads][splits]
// of latent_dim + 2 floats.
template <typename T, int DPL>
__global__ void __launch_bounds__(kWarps * 32, 2) latent_simt_kernel(const LatentArgs a, int splits, float* records) {
    constexpr int PITCH = DPL * 32;  // elements of a row in shared memory
    extern __shared__ __align__(16) uint8_t smem[];  // [STAGES][KEYS][PITCH] of T; at the end [HEADS][PITCH] floats
    __shared__ float sm_m[kWarps][GH], sm_l[kWarps][GH];
    static_assert(STAGES * KEYS * sizeof(T) >= HEADS * sizeof(float), "the sums fit in the stages");
    pdl_wait_primary();
    pdl_launch_dependents();
    const int row = blockIdx.x, h0 = blockIdx.y * HEADS, nh = min(HEADS, a.num_heads - h0), piece = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int req = row, num_new = 1, j = 0;
    if (a.cu != nullptr) {
        if (row >= a.cu[a.num_seqs]) return;  // behind the last request
        int lo = 0, hi = a.num_seqs - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (a.cu[mid] <= row) lo = mid;
            else hi = mid - 1;
        }
        req = lo;
        num_new = a.cu[req + 1] - a.cu[req];
        j = row - a.cu[req];
    }
    const int L = a.seq_lens[req];
    const int seen = a.causal ? min(L, L - num_new + j + 1) : L;  // keys this row sees, and this piece of them
    const int from = (int)((int64_t)max(seen, 0) * piece / splits);
    const int visible = (int)((int64_t)max(seen, 0) * (piece + 1) / splits);
    const int lat = a.latent_dim, D = lat + a.rope_dim;
    const T* cache = static_cast<const T*>(a.cache);
    const int32_t* table = a.block_tables + (int64_t)req * a.max_blocks;
    const float scale_log2 = a.scale * 1.4426950408889634f;
    // this warp's heads, and its share of the keys
    const int groups = nh <= GH ? 1 : nh <= 2 * GH ? 2 : 4, shares = kWarps / groups;
    const int group = warp % groups, share = warp / groups, mine = min(GH, nh - GH * group);

    unsigned long long qv[GH][DPL / 2], acc[GH][DPL / 2];
    // of head lane / 4 % 4; l: of the first (lanes 0 ..) and second keys of the pairs
    float m = -INFINITY, l = 0.f;
    const T* q = static_cast<const T*>(a.q) + ((int64_t)row * a.num_heads + h0 + GH * group) * D;
#pragma unroll
    for (int h = 0; h < GH; ++h) {
#pragma unroll
        for (int k = 0; k < DPL / 2; ++k) {
            const int d = 2 * lane + 64 * k;
            qv[h][k] = f32x2_pack(h < mine && d < D ? Elt<T>::to_f(q[(int64_t)h * D + d]) : 0.f,
                                  h < mine && d + 1 < D ? Elt<T>::to_f(q[(int64_t)h * D + d + 1]) : 0.f);
            acc[h][k] = 0ull;
        }
    }
    T* const stages = reinterpret_cast<T*>(smem);
    if (D < PITCH) {  // what no row fills is zero
        for (int i = threadIdx.x; i < STAGES * KEYS * PITCH * (int)sizeof(T) / 16; i += kWarps * 32)
            reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
    }
    // loads: keys warp and warp + 4 of a tile
    const int bytes = D * (int)sizeof(T), tiles = (visible - from + KEYS - 1) / KEYS;
    const bool vec = bytes % 16 == 0;
    const T* ahead[2];  // the rows of the tile to load next
    auto rows_of = [&](int tile) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = from + tile * KEYS + warp + kWarps * i;
            ahead[i] = t < visible ? cache + ((int64_t)table[t / a.block_size] * a.block_size + t % a.block_size) * D
                                   : nullptr;
        }
    };
    auto load = [&](int tile) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            T* to = stages + (tile % STAGES * KEYS + warp + kWarps * i) * PITCH;
            if (ahead[i] == nullptr) {  // zero beside the last key
                for (int d = lane; d < D; d += 32) to[d] = Elt<T>::from_f(0.f);
            } else if (vec) {
                const uint8_t* src = reinterpret_cast<const uint8_t*>(ahead[i]);
                const uint32_t dst = (uint32_t)__cvta_generic_to_shared(to);
                for (int c = 16 * lane; c < bytes; c += 512)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + c), "l"(src + c) : "memory");
            } else {
                for (int d = lane; d < D; d += 32) to[d] = ahead[i][d];
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        rows_of(tile + 1);
    };
    rows_of(0);
    for (int i = 0; i < STAGES - 1; ++i) load(i);
    for (int tile = 0; tile < tiles; ++tile) {
        asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
        __syncthreads();  // this tile is there, and the one before it read
        load(tile + STAGES - 1);
        const int keys = min(KEYS, visible - from - tile * KEYS);
        if (mine <= 0) continue;
        for (int t = 2 * share; t < keys; t += 2 * shares) {
            const T* x0 = stages + (tile % STAGES * KEYS + t) * PITCH + 2 * lane;
            unsigned long long x[2][DPL / 2];
#pragma unroll
            for (int k = 0; k < DPL / 2; ++k) {
                x[0][k] = pair_of(x0 + 64 * k);
                x[1][k] = pair_of(x0 + PITCH + 64 * k);  // (zero where there is none)
            }
            float dot[2 * GH];  // of key 0, then of key 1
#pragma unroll
            for (int h = 0; h < GH; ++h)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    unsigned long long d2 = 0ull;
#pragma unroll
                    for (int k = 0; k < DPL / 2; ++k) d2 = fma_f32x2(qv[h][k], x[e][k], d2);
                    float u, v;
                    f32x2_unpack(d2, u, v);
                    dot[GH * e + h] = u + v;
                }
            // the eight sums over the lanes: each exchange halves what a lane
            // keeps, so nine shuffles instead of forty; lanes 4 i .. 4 i + 3
            // end with sum i and take its weight for all
            static_assert(GH == 4, "three exchanges leave one sum a lane");
            float z[4], y[2], s1;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool up = lane & 16;
                z[i] = (up ? dot[4 + i] : dot[i]) + __shfl_xor_sync(0xffffffffu, up ? dot[i] : dot[4 + i], 16);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const bool up = lane & 8;
                y[i] = (up ? z[2 + i] : z[i]) + __shfl_xor_sync(0xffffffffu, up ? z[i] : z[2 + i], 8);
            }
            s1 = (lane & 4 ? y[1] : y[0]) + __shfl_xor_sync(0xffffffffu, lane & 4 ? y[0] : y[1], 4);
            s1 += __shfl_xor_sync(0xffffffffu, s1, 2);
            s1 += __shfl_xor_sync(0xffffffffu, s1, 1);
            const float x2 = lane < 16 || t + 1 < keys ? s1 * scale_log2 : -INFINITY;
            const float mx = fmaxf(x2, __shfl_xor_sync(0xffffffffu, x2, 16));
            if (__any_sync(0xffffffffu, mx > m)) {  // (ever more seldom)
                const float mn = fmaxf(m, mx), c = mn == -INFINITY ? 1.f : exp2f(m - mn);
                m = mn;
                l *= c;
#pragma unroll
                for (int h = 0; h < GH; ++h) {
                    const float ch = __shfl_sync(0xffffffffu, c, 4 * h);
                    if (ch == 1.f) continue;
                    const unsigned long long c2 = f32x2_pack(ch, ch);
#pragma unroll
                    for (int k = 0; k < DPL / 2; ++k) acc[h][k] = fma_f32x2(acc[h][k], c2, 0ull);
                }
            }
            const float w = exp2f(x2 - (m == -INFINITY ? 0.f : m));
            l += w;
#pragma unroll
            for (int h = 0; h < GH; ++h) {
                const float wa = __shfl_sync(0xffffffffu, w, 4 * h), wb = __shfl_sync(0xffffffffu, w, 16 + 4 * h);
                const unsigned long long wa2 = f32x2_pack(wa, wa), wb2 = f32x2_pack(wb, wb);
#pragma unroll
                for (int k = 0; k < DPL / 2; ++k)
                    acc[h][k] = fma_f32x2(wb2, x[1][k], fma_f32x2(wa2, x[0][k], acc[h][k]));
            }
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    l += __shfl_xor_sync(0xffffffffu, l, 16);
    if (lane < 16 && lane % 4 == 0) sm_m[warp][lane / 4] = m, sm_l[warp][lane / 4] = l;
    // a head's sums, one share after the other (a fixed order)
    float* const sums = reinterpret_cast<float*>(smem);
    for (int w = 0; w < shares; ++w) {
        __syncthreads();
        if (share != w) continue;
#pragma unroll
        for (int h = 0; h < GH; ++h) {
            float M = -INFINITY;
            for (int v = group; v < kWarps; v += groups) M = fmaxf(M, sm_m[v][h]);
            const float f = exp2f(sm_m[warp][h] - (M == -INFINITY ? 0.f : M));
#pragma unroll
            for (int k = 0; k < DPL / 2; ++k) {
                float2* s = reinterpret_cast<float2*>(sums + (GH * group + h) * PITCH + 2 * lane + 64 * k);
                float u, v;
                f32x2_unpack(acc[h][k], u, v);
                const float2 old = w ? *s : make_float2(0.f, 0.f);
                *s = make_float2(old.x + f * u, old.y + f * v);
            }
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < nh * lat; e += blockDim.x) {
        const int h = e / lat, d = e - h * lat, g = h / GH;
        float M = -INFINITY, sum = 0.f;
        for (int v = g; v < kWarps; v += groups) M = fmaxf(M, sm_m[v][h % GH]);
        for (int v = g; v < kWarps; v += groups)
            sum += exp2f(sm_m[v][h % GH] - (M == -INFINITY ? 0.f : M)) * sm_l[v][h % GH];
        const float o = sums[h * PITCH + d];
        if (splits > 1) {
            float* rec = records + (((int64_t)row * a.num_heads + h0 + h) * splits + piece) * (lat + 2);
            rec[d] = o;
            if (d == 0) {
                rec[lat] = M;
                rec[lat + 1] = sum;
            }
            continue;
        }
        // (a row that sees nothing is zero; a NaN sum stays NaN)
        static_cast<T*>(a.out)[((int64_t)row * a.num_heads + h0 + h) * lat + d] =
            Elt<T>::from_f(visible > 0 ? o / sum : 0.f);
    }
}

// Joins the pieces of a (row, head), in order: 128 dims a CTA.
template <typename T>
__global__ void __launch_bounds__(128) latent_simt_join_kernel(const LatentArgs a, int splits, const float* records) {
    pdl_wait_primary();
    pdl_launch_dependents();
    const int lat = a.latent_dim;
    const int64_t rh = (int64_t)blockIdx.x * a.num_heads + blockIdx.y;
    if (a.cu && (int)blockIdx.x >= a.cu[a.num_seqs]) return;  // behind the last request
    const float* rec = records + rh * splits * (lat + 2);
    __shared__ float weight[kMaxSplits], top[4], total[4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float M = -INFINITY, sum = 0.f;
    for (int i = threadIdx.x; i < splits; i += 128) M = fmaxf(M, weight[i] = rec[(int64_t)i * (lat + 2) + lat]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (lane == 0) top[warp] = M;
    __syncthreads();
    M = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    const float ms = M == -INFINITY ? 0.f : M;
    for (int i = threadIdx.x; i < splits; i += 128)
        sum = fmaf(weight[i] = exp2f(weight[i] - ms), rec[(int64_t)i * (lat + 2) + lat + 1], sum);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) total[warp] = sum;
    __syncthreads();
    sum = (total[0] + total[1]) + (total[2] + total[3]);
    if (const int d = blockIdx.z * 128 + threadIdx.x; d < lat) {
        float o = 0.f;
#pragma unroll 16
        for (int i = 0; i < splits; ++i) o = fmaf(weight[i], rec[(int64_t)i * (lat + 2) + d], o);
        static_cast<T*>(a.out)[rh * lat + d] = Elt<T>::from_f(sum == 0.f ? 0.f : o / sum);
    }
}

// Pieces of each row's keys: four CTAs for every SM (two run at once) or a few
// less, of 64 keys at least (1 x 32,768 fp32 tokens of 16 heads are one CTA
// otherwise).
int simt_splits(int64_t total_q, int32_t num_heads, int32_t max_context) {
    const int64_t ctas = total_q * ((num_heads + HEADS - 1) / HEADS);
    const int64_t want = ctas <= kSms ? 4 * kSms / ctas : (4 * kSms + ctas - 1) / ctas;
    const int64_t most = ((int64_t)max_context + 63) / 64;
    return (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(want, kMaxSplits), most));
}

template <typename T, int DPL>
cudaError_t launch_rows(const LatentArgs& a, int splits, float* records, cudaStream_t stream) {
    const dim3 grid((unsigned)a.total_q, (unsigned)((a.num_heads + HEADS - 1) / HEADS), (unsigned)splits);
    const size_t smem = (size_t)STAGES * KEYS * DPL * 32 * sizeof(T);
    const auto kernel = latent_simt_kernel<T, DPL>;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), smem);
    if (e != cudaSuccess) return e;
    return launch_pdl_smem(kernel, grid, dim3(kWarps * 32), smem, stream, a, splits, records);
}

template <typename T>
cudaError_t launch_typed(const LatentArgs& a, float* records, cudaStream_t stream) {
    const int D = a.latent_dim + a.rope_dim, splits = simt_splits(a.total_q, a.num_heads, a.max_context);
    cudaError_t e = D <= 128   ? launch_rows<T, 4>(a, splits, records, stream)
                    : D <= 320 ? launch_rows<T, 10>(a, splits, records, stream)
                               : launch_rows<T, 18>(a, splits, records, stream);
    if (e != cudaSuccess || splits == 1) return e;
    return launch_pdl(latent_simt_join_kernel<T>, dim3((unsigned)a.total_q, (unsigned)a.num_heads, (unsigned)((a.latent_dim + 127) / 128)),
                      dim3(128), stream, a, splits, (const float*)records);
}

}  // namespace

bool latent_simt_supported(int dtype, int32_t row_dim) { return dtype >= 0 && dtype <= 2 && row_dim <= 576; }

size_t latent_simt_workspace(int64_t total_q, int32_t num_heads, int32_t latent_dim, int32_t max_context) {
    const int splits = simt_splits(total_q, num_heads, max_context);
    return splits == 1 ? 0 : (size_t)total_q * num_heads * splits * (latent_dim + 2) * sizeof(float);
}

cudaError_t launch_latent_simt(const LatentArgs& a, void* workspace, cudaStream_t stream) {
    float* records = static_cast<float*>(workspace);
    if (a.total_q == 0 || a.num_seqs == 0) return cudaSuccess;
    switch (a.dtype) {
        case 0: return launch_typed<float>(a, records, stream);
        case 1: return launch_typed<__nv_bfloat16>(a, records, stream);
        default: return launch_typed<__half>(a, records, stream);
    }
}

}  // namespace pa
