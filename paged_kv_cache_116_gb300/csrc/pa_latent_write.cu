// pa_latent_write.cu -- one row a token into a latent cache: the normalised
// latent vector and the rotated position part, with the queries' position
// parts rotated in the same kernel.
//
// For token t with x = kv[t] (latent_dim + rope_dim elements):
//   c   = x[0 : latent_dim] * w / sqrt(mean(x[0 : latent_dim]^2) + eps)
//         (without a weight w: as it is, bit for bit),
//   k_r = the rotation of x[latent_dim :] by the token's position,
// and the row [c | k_r] goes to its slot; q_out[t, h] gets q[t, h] (rope_dim
// elements) rotated by the same angles.  Angles and rotations are those of
// pa_rope.cu; sums, norms and rotations are fp32, rounded once.
//
// Bound: HBM.  Each byte is read and written once.  A CTA takes `tpb` tokens:
// their sines and cosines go to shared memory once and serve every head, a
// warp works a token's row (its vectors stay in registers between the sum of
// squares and the scaling), then every thread works 16-byte vectors of the
// queries, the two that hold both halves of 8 (16-bit) or 4 (fp32) pairs.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_launch.cuh"
#include "pa_rotary.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kCtasPerSm = 4;

template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) latent_write_kernel(const LatentWriteArgs p) {
    extern __shared__ float2 tab[];  // [tpb][rope_dim / 2] cosine, sine
    pdl_wait_primary();
    pdl_launch_dependents();
    const int64_t t0 = (int64_t)blockIdx.x * p.tpb;
    const int nt = (int)min((int64_t)p.tpb, p.n - t0);
    const int half = p.rope_dim / 2, lat = p.latent_dim, D = lat + p.rope_dim;
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
        const int t = i / half, pr = i - t * half;
        tab[i] = turn_of(p.positions[t0 + t], p.inv_freq[pr]);
    }
    __syncthreads();
    // the pair at o0, o1 (VEC pairs from `pr` on)
    auto first = [&](int pr) { return p.interleaved ? 2 * pr : pr; };
    auto second = [&](int pr) { return p.interleaved ? 2 * pr + VEC : pr + half; };  // (VEC 1: 2 pr + 1)

    if (blockIdx.y == 0) {
        constexpr int NV = 4, SPAN = 32 * VEC * NV;  // a lane's vectors at a time
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        for (int t = warp; t < nt; t += kThreads / 32) {
            const int64_t slot = p.slots[t0 + t];
            if (slot < 0) continue;  // a padding token
            const T* x = static_cast<const T*>(p.kv) + (t0 + t) * p.kv_stride;
            T* row = static_cast<T*>(p.cache) + slot * D;
            RVec<T, VEC> v[NV];
            auto fetch = [&](int c0) {
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int i = c0 + (k * 32 + lane) * VEC;
                    if (i < lat) v[k] = load_vec<T, VEC>(x + i);
                }
            };
            float inv = 1.f;
            fetch(0);
            if (p.norm_weight) {
                float sum = 0.f;
                for (int c0 = 0; c0 < lat; c0 += SPAN) {
                    if (c0) fetch(c0);
#pragma unroll
                    for (int k = 0; k < NV; ++k) {
                        if (c0 + (k * 32 + lane) * VEC >= lat) break;
                        float f[VEC];
                        unpack<T, VEC>(v[k], f);
#pragma unroll
                        for (int e = 0; e < VEC; ++e) sum = fmaf(f[e], f[e], sum);
                    }
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                inv = 1.f / sqrtf(sum / (float)lat + p.eps);
                if (lat > SPAN) fetch(0);
            }
            for (int c0 = 0; c0 < lat; c0 += SPAN) {
                if (c0) fetch(c0);
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int i = c0 + (k * 32 + lane) * VEC;
                    if (i >= lat) break;
                    if (p.norm_weight) {
                        float f[VEC], w[VEC];
                        unpack<T, VEC>(v[k], f);
                        unpack<T, VEC>(*reinterpret_cast<const RVec<T, VEC>*>(static_cast<const T*>(p.norm_weight) + i), w);
#pragma unroll
                        for (int e = 0; e < VEC; ++e) v[k].e[e] = Elt<T>::from_f(f[e] * inv * w[e]);
                    }
                    store_vec<T, VEC>(row + i, v[k]);
                }
            }
            for (int pr = lane * VEC; pr < half; pr += 32 * VEC) {
                const int o0 = lat + first(pr), o1 = lat + second(pr);
                RVec<T, VEC> a = load_vec<T, VEC>(x + o0), b = load_vec<T, VEC>(x + o1);
                float f[2][VEC];
                unpack<T, VEC>(a, f[0]);
                unpack<T, VEC>(b, f[1]);
                rotate<VEC>(f[0], f[1], tab + t * half + pr, p.interleaved);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    a.e[e] = Elt<T>::from_f(f[0][e]);
                    b.e[e] = Elt<T>::from_f(f[1][e]);
                }
                store_vec<T, VEC>(row + o0, a);
                store_vec<T, VEC>(row + o1, b);
            }
        }
    }

    // the queries: an item is VEC pairs of one head of one token
    constexpr int U = 4;  // items in flight
    const int R = half / VEC, items = p.num_heads * R, all = nt * items, step = gridDim.y * kThreads;
    for (int i0 = blockIdx.y * kThreads + threadIdx.x; i0 < all; i0 += U * step) {
        RVec<T, VEC> a[U], b[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * step;
            if (i >= all) break;
            const int t = i / items, r = i - t * items, h = r / R, pr = (r - h * R) * VEC;
            const T* s = static_cast<const T*>(p.q) + (t0 + t) * p.q_stride + h * p.q_head_stride;
            a[u] = load_vec<T, VEC>(s + first(pr));
            b[u] = load_vec<T, VEC>(s + second(pr));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * step;
            if (i >= all) break;
            const int t = i / items, r = i - t * items, h = r / R, pr = (r - h * R) * VEC;
            float f[2][VEC];
            unpack<T, VEC>(a[u], f[0]);
            unpack<T, VEC>(b[u], f[1]);
            rotate<VEC>(f[0], f[1], tab + t * half + pr, p.interleaved);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                a[u].e[e] = Elt<T>::from_f(f[0][e]);
                b[u].e[e] = Elt<T>::from_f(f[1][e]);
            }
            T* d = static_cast<T*>(p.q_out) + (t0 + t) * p.q_out_stride + h * p.q_out_head_stride;
            store_vec<T, VEC>(d + first(pr), a[u]);
            store_vec<T, VEC>(d + second(pr), b[u]);
        }
    }
}

template <typename T>
cudaError_t launch_typed(const LatentWriteArgs& a, cudaStream_t stream) {
    constexpr int V = 16 / (int)sizeof(T);
    const uintptr_t addr = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.q_out) |
                           reinterpret_cast<uintptr_t>(a.kv) | reinterpret_cast<uintptr_t>(a.norm_weight) |
                           reinterpret_cast<uintptr_t>(a.cache);
    const int64_t strides = a.q_stride | a.q_head_stride | a.q_out_stride | a.q_out_head_stride | a.kv_stride;
    const bool vec = (addr & 15) == 0 && strides % V == 0 && a.latent_dim % V == 0 && a.rope_dim % (2 * V) == 0;
    LatentWriteArgs p = a;
    // tokens per CTA: the batch in one wave of four CTAs per SM, at most 16
    // (the angles' table); few tokens: the heads' items over several CTAs each
    const int64_t slots = (int64_t)kSms * kCtasPerSm;
    p.tpb = (int)std::min<int64_t>(16, (a.n + slots - 1) / slots);
    const int64_t ctas = (a.n + p.tpb - 1) / p.tpb;
    const int64_t items = (int64_t)p.tpb * a.num_heads * (a.rope_dim / (vec ? 2 * V : 2));
    const int64_t parts =
        std::max<int64_t>(1, std::min<int64_t>({slots / 2 / ctas, (items + kThreads - 1) / kThreads, 65535}));
    const dim3 grid((unsigned)ctas, (unsigned)parts);
    const size_t smem = (size_t)p.tpb * (a.rope_dim / 2) * sizeof(float2);
    return vec ? launch_pdl_smem(latent_write_kernel<T, V>, grid, dim3(kThreads), smem, stream, p)
               : launch_pdl_smem(latent_write_kernel<T, 1>, grid, dim3(kThreads), smem, stream, p);
}

}  // namespace

cudaError_t launch_latent_write(const LatentWriteArgs& a, int dtype, cudaStream_t stream) {
    switch (dtype) {
        case 0: return launch_typed<float>(a, stream);
        case 1: return launch_typed<__nv_bfloat16>(a, stream);
        default: return launch_typed<__half>(a, stream);
    }
}

}  // namespace pa
