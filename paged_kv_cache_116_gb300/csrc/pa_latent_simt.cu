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
// One CTA of four warps per (query row, four heads): lanes split the row's
// elements, each warp keeps one online softmax per head over an interleaved
// share of the keys, and the warps' states are joined at the end.  Bound: the
// shuffles of the scores' sums (five per head and key).  Two keys per warp in
// flight hide the table's and the row's round trips.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_launch.cuh"

namespace pa {
namespace {

constexpr int kWarps = 4;
constexpr int GH = 4;  // heads per CTA

// DPL: elements of a row per lane.
template <typename T, int DPL>
__global__ void __launch_bounds__(kWarps * 32) latent_simt_kernel(const LatentArgs a) {
    __shared__ float sm_m[kWarps][GH], sm_l[kWarps][GH];
    __shared__ float sm_acc[GH][DPL * 32];
    pdl_wait_primary();
    pdl_launch_dependents();
    const int row = blockIdx.x, h0 = blockIdx.y * GH, nh = min(GH, a.num_heads - h0);
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
    const int visible = a.causal ? min(L, L - num_new + j + 1) : L;
    const int lat = a.latent_dim, D = lat + a.rope_dim;
    const T* q = static_cast<const T*>(a.q) + ((int64_t)row * a.num_heads + h0) * D;
    const T* cache = static_cast<const T*>(a.cache);
    const int32_t* table = a.block_tables + (int64_t)req * a.max_blocks;
    const float scale_log2 = a.scale * 1.4426950408889634f;

    float qv[GH][DPL], acc[GH][DPL], m[GH], l[GH];
#pragma unroll
    for (int h = 0; h < GH; ++h) {
        m[h] = -INFINITY;
        l[h] = 0.f;
#pragma unroll
        for (int k = 0; k < DPL; ++k) {
            const int d = lane + 32 * k;
            qv[h][k] = h < nh && d < D ? Elt<T>::to_f(q[(int64_t)h * D + d]) : 0.f;
            acc[h][k] = 0.f;
        }
    }
    constexpr int U = DPL <= 9 ? 2 : 1;
    for (int t0 = warp; t0 < visible; t0 += U * kWarps) {
        float x[U][DPL];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = min(t0 + u * kWarps, visible - 1);
            const T* r = cache + ((int64_t)table[t / a.block_size] * a.block_size + t % a.block_size) * D;
#pragma unroll
            for (int k = 0; k < DPL; ++k) {
                const int d = lane + 32 * k;
                x[u][k] = d < D ? Elt<T>::to_f(r[d]) : 0.f;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (t0 + u * kWarps >= visible) break;  // (the whole warp)
            float dot[GH];
#pragma unroll
            for (int h = 0; h < GH; ++h) {
                dot[h] = 0.f;
#pragma unroll
                for (int k = 0; k < DPL; ++k) dot[h] = fmaf(qv[h][k], x[u][k], dot[h]);
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1)
#pragma unroll
                for (int h = 0; h < GH; ++h) dot[h] += __shfl_xor_sync(0xffffffffu, dot[h], off);
#pragma unroll
            for (int h = 0; h < GH; ++h) {
                const float s = dot[h] * scale_log2, m_new = fmaxf(m[h], s);
                const float c = exp2f(m[h] - m_new), p = exp2f(s - m_new);
                l[h] = l[h] * c + p;
#pragma unroll
                for (int k = 0; k < DPL; ++k) acc[h][k] = fmaf(p, x[u][k], acc[h][k] * c);
                m[h] = m_new;
            }
        }
    }
    if (lane == 0) {
#pragma unroll
        for (int h = 0; h < GH; ++h) {
            sm_m[warp][h] = m[h];
            sm_l[warp][h] = l[h];
        }
    }
    // the warps' sums, one warp after the other (a fixed order)
    for (int w = 0; w < kWarps; ++w) {
        __syncthreads();
        if (warp != w) continue;
#pragma unroll
        for (int h = 0; h < GH; ++h) {
            float M = -INFINITY;
            for (int v = 0; v < kWarps; ++v) M = fmaxf(M, sm_m[v][h]);
            const float f = m[h] == -INFINITY ? 0.f : exp2f(m[h] - M);
#pragma unroll
            for (int k = 0; k < DPL; ++k) {
                float* s = &sm_acc[h][lane + 32 * k];
                *s = (w ? *s : 0.f) + f * acc[h][k];
            }
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < nh * lat; e += blockDim.x) {
        const int h = e / lat, d = e - h * lat;
        float M = -INFINITY, sum = 0.f;
#pragma unroll
        for (int v = 0; v < kWarps; ++v) M = fmaxf(M, sm_m[v][h]);
#pragma unroll
        for (int v = 0; v < kWarps; ++v) sum += sm_m[v][h] == -INFINITY ? 0.f : exp2f(sm_m[v][h] - M) * sm_l[v][h];
        // (a row that sees nothing is zero; a NaN sum stays NaN)
        static_cast<T*>(a.out)[((int64_t)row * a.num_heads + h0 + h) * lat + d] =
            Elt<T>::from_f(visible > 0 ? sm_acc[h][d] / sum : 0.f);
    }
}

template <typename T>
cudaError_t launch_typed(const LatentArgs& a, cudaStream_t stream) {
    const int D = a.latent_dim + a.rope_dim;
    const dim3 grid((unsigned)a.total_q, (unsigned)((a.num_heads + GH - 1) / GH)), block(kWarps * 32);
    if (D <= 128) return launch_pdl(latent_simt_kernel<T, 4>, grid, block, stream, a);
    if (D <= 288) return launch_pdl(latent_simt_kernel<T, 9>, grid, block, stream, a);
    return launch_pdl(latent_simt_kernel<T, 18>, grid, block, stream, a);
}

}  // namespace

bool latent_simt_supported(int dtype, int32_t row_dim) { return dtype >= 0 && dtype <= 2 && row_dim <= 576; }

cudaError_t launch_latent_simt(const LatentArgs& a, cudaStream_t stream) {
    if (a.total_q == 0 || a.num_seqs == 0) return cudaSuccess;
    switch (a.dtype) {
        case 0: return launch_typed<float>(a, stream);
        case 1: return launch_typed<__nv_bfloat16>(a, stream);
        default: return launch_typed<__half>(a, stream);
    }
}

}  // namespace pa
