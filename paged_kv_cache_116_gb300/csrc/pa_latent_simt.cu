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
// One CTA of four warps per (query row, four heads), and per piece of the keys
// where there are too few rows to fill the GPU: lanes split the row's elements,
// each warp keeps one online softmax per head over an interleaved share of the
// keys, and the warps' states are joined at the end; pieces leave (o, m, l)
// records that latent_simt_join_kernel joins in order.  Bound: instructions (per
// key and four heads 144 products of a lane's elements and ten shuffles).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_launch.cuh"

namespace pa {
namespace {

constexpr int kWarps = 4;
constexpr int GH = 4;  // heads per CTA

// DPL: elements of a row per lane.
// splits pieces of each row's keys; records (splits > 1): [rows][heads][splits]
// of latent_dim + 2 floats.
template <typename T, int DPL>
__global__ void __launch_bounds__(kWarps * 32) latent_simt_kernel(const LatentArgs a, int splits, float* records) {
    __shared__ float sm_m[kWarps][GH], sm_l[kWarps][GH];
    __shared__ float sm_acc[GH][DPL * 32];
    pdl_wait_primary();
    pdl_launch_dependents();
    const int row = blockIdx.x, h0 = blockIdx.y * GH, nh = min(GH, a.num_heads - h0), piece = blockIdx.z;
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
    // the next key's row is on its way while one is worked, and the table entry
    // of the one after it
    auto row_of = [&](int t) -> const T* {
        t = min(t, visible - 1);
        return cache + ((int64_t)table[t / a.block_size] * a.block_size + t % a.block_size) * D;
    };
    auto fetch = [&](const T* r, float (&x)[DPL]) {
#pragma unroll
        for (int k = 0; k < DPL; ++k) {
            const int d = lane + 32 * k;
            x[k] = d < D ? Elt<T>::to_f(r[d]) : 0.f;
        }
    };
    int t = from + warp;
    float x[DPL], ahead[DPL];
    const T* next = nullptr;
    if (t < visible) {
        fetch(row_of(t), x);
        next = row_of(t + kWarps);
    }
    for (; t < visible; t += kWarps) {
        fetch(next, ahead);
        next = row_of(t + 2 * kWarps);
        float dot[GH];
#pragma unroll
        for (int h = 0; h < GH; ++h) {
            dot[h] = 0.f;
#pragma unroll
            for (int k = 0; k < DPL; ++k) dot[h] = fmaf(qv[h][k], x[k], dot[h]);
        }
        // the four sums over the lanes: each exchange halves what a lane
        // keeps, so ten shuffles instead of twenty
        static_assert(GH == 4, "two exchanges leave one head a lane");
        const bool upper = lane & 16, odd = lane & 8;
        float a0 = upper ? dot[2] : dot[0], a1 = upper ? dot[3] : dot[1];
        a0 += __shfl_xor_sync(0xffffffffu, upper ? dot[0] : dot[2], 16);
        a1 += __shfl_xor_sync(0xffffffffu, upper ? dot[1] : dot[3], 16);
        float z = odd ? a1 : a0;
        z += __shfl_xor_sync(0xffffffffu, odd ? a0 : a1, 8);
#pragma unroll
        for (int off = 4; off > 0; off >>= 1) z += __shfl_xor_sync(0xffffffffu, z, off);
#pragma unroll
        for (int h = 0; h < GH; ++h) {
            const float s = __shfl_sync(0xffffffffu, z, 8 * h) * scale_log2;
            if (s > m[h]) {  // (the whole warp, and ever more seldom)
                const float c = exp2f(m[h] - s);
                l[h] *= c;
#pragma unroll
                for (int k = 0; k < DPL; ++k) acc[h][k] *= c;
                m[h] = s;
            }
            const float p = exp2f(s - (m[h] == -INFINITY ? 0.f : m[h]));
            l[h] += p;
#pragma unroll
            for (int k = 0; k < DPL; ++k) acc[h][k] = fmaf(p, x[k], acc[h][k]);
        }
#pragma unroll
        for (int k = 0; k < DPL; ++k) x[k] = ahead[k];
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
        if (splits > 1) {
            float* rec = records + (((int64_t)row * a.num_heads + h0 + h) * splits + piece) * (lat + 2);
            rec[d] = visible > from ? sm_acc[h][d] : 0.f;
            if (d == 0) {
                rec[lat] = M;
                rec[lat + 1] = sum;
            }
            continue;
        }
        // (a row that sees nothing is zero; a NaN sum stays NaN)
        static_cast<T*>(a.out)[((int64_t)row * a.num_heads + h0 + h) * lat + d] =
            Elt<T>::from_f(visible > 0 ? sm_acc[h][d] / sum : 0.f);
    }
}

// Joins the pieces of a (row, head), in order.
template <typename T>
__global__ void __launch_bounds__(128) latent_simt_join_kernel(const LatentArgs a, int splits, const float* records) {
    pdl_wait_primary();
    pdl_launch_dependents();
    const int lat = a.latent_dim;
    const int64_t rh = (int64_t)blockIdx.x * a.num_heads + blockIdx.y;
    if (a.cu && (int)blockIdx.x >= a.cu[a.num_seqs]) return;  // behind the last request
    const float* rec = records + rh * splits * (lat + 2);
    float M = -INFINITY, sum = 0.f;
    for (int i = 0; i < splits; ++i) M = fmaxf(M, rec[(int64_t)i * (lat + 2) + lat]);
    const float ms = M == -INFINITY ? 0.f : M;
    for (int i = 0; i < splits; ++i)
        sum += exp2f(rec[(int64_t)i * (lat + 2) + lat] - ms) * rec[(int64_t)i * (lat + 2) + lat + 1];
    for (int d = threadIdx.x; d < lat; d += blockDim.x) {
        float o = 0.f;
        for (int i = 0; i < splits; ++i)
            o = fmaf(exp2f(rec[(int64_t)i * (lat + 2) + lat] - ms), rec[(int64_t)i * (lat + 2) + d], o);
        static_cast<T*>(a.out)[rh * lat + d] = Elt<T>::from_f(sum == 0.f ? 0.f : o / sum);
    }
}

// Pieces of each row's keys: enough CTAs for four on every SM, of 64 keys at
// least (1 x 32,768 fp32 tokens of 16 heads are 4 CTAs otherwise).
int simt_splits(int64_t total_q, int32_t num_heads, int32_t max_context) {
    const int64_t ctas = total_q * ((num_heads + GH - 1) / GH);
    const int64_t want = (4 * kSms + ctas - 1) / ctas, most = ((int64_t)max_context + 63) / 64;
    return (int)std::max<int64_t>(1, std::min<int64_t>(want, std::min<int64_t>(most, 1024)));
}

template <typename T>
cudaError_t launch_typed(const LatentArgs& a, float* records, cudaStream_t stream) {
    const int D = a.latent_dim + a.rope_dim, splits = simt_splits(a.total_q, a.num_heads, a.max_context);
    const dim3 grid((unsigned)a.total_q, (unsigned)((a.num_heads + GH - 1) / GH), (unsigned)splits), block(kWarps * 32);
    cudaError_t e = D <= 128   ? launch_pdl(latent_simt_kernel<T, 4>, grid, block, stream, a, splits, records)
                    : D <= 288 ? launch_pdl(latent_simt_kernel<T, 9>, grid, block, stream, a, splits, records)
                               : launch_pdl(latent_simt_kernel<T, 18>, grid, block, stream, a, splits, records);
    if (e != cudaSuccess || splits == 1) return e;
    return launch_pdl(latent_simt_join_kernel<T>, dim3((unsigned)a.total_q, (unsigned)a.num_heads), dim3(128), stream, a,
                      splits, (const float*)records);
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
