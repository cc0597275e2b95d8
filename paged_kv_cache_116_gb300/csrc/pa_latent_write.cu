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
// Bound: HBM, while every load is followed by stores to scattered 128-byte
// pieces (8,192 tokens of 128 heads: 287 MB in 53 us, 5.4 TB/s; a copy of as many
// dense bytes takes 46).  Each byte is read and written once.  A CTA takes `tpb` tokens:
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
    // Item r of R: two vectors that hold VEC whole pairs, each next to the same
    // vector of item r + 1: both halves of pairs r VEC .. (pairs i, i + half), or
    // pairs of the first and of the second half (pairs 2 i, 2 i + 1).
    const int R = half / VEC;
    auto first = [&](int r) { return VEC == 1 && p.interleaved ? 2 * r : r * VEC; };
    auto second = [&](int r) { return VEC == 1 && p.interleaved ? 2 * r + 1 : half + r * VEC; };
    auto turn = [&](RVec<T, VEC>& a, RVec<T, VEC>& b, int t, int r) {
        float f[2][VEC];
        unpack<T, VEC>(a, f[0]);
        unpack<T, VEC>(b, f[1]);
        const float2* cs = tab + t * half;
        if (VEC > 1 && p.interleaved) {
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const float2* c = cs + (v * half + r * VEC) / 2;
#pragma unroll
                for (int e = 0; e < VEC / 2; ++e) {
                    const float x = f[v][2 * e], y = f[v][2 * e + 1];
                    f[v][2 * e] = x * c[e].x - y * c[e].y;
                    f[v][2 * e + 1] = y * c[e].x + x * c[e].y;
                }
            }
        } else {
            rotate<VEC>(f[0], f[1], cs + r * VEC, false);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            a.e[e] = Elt<T>::from_f(f[0][e]);
            b.e[e] = Elt<T>::from_f(f[1][e]);
        }
    };

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
            for (int r = lane; r < R; r += 32) {
                RVec<T, VEC> a = load_vec<T, VEC>(x + lat + first(r)), b = load_vec<T, VEC>(x + lat + second(r));
                turn(a, b, t, r);
                store_vec<T, VEC>(row + lat + first(r), a);
                store_vec<T, VEC>(row + lat + second(r), b);
            }
        }
    }

    // The queries.  A thread finds its item (of a head) once and works it for
    // all tokens of the CTA; where a token's items do not fill the CTA, for every
    // `step`th token.
    constexpr int U = 2;  // tokens in flight (more spill: three and four took 87 and 98 us where two take 63)
    const int items = p.num_heads * R, step = items && items < kThreads ? kThreads / items : 1;
    const int begin = step > 1 ? threadIdx.x / items : 0;
    if (begin >= step) return;
    for (int it = step > 1 ? threadIdx.x - begin * items : blockIdx.y * kThreads + threadIdx.x; it < items;
         it += step > 1 ? items : gridDim.y * kThreads) {
        const int h = it / R, r = it - h * R;
        const T* s = static_cast<const T*>(p.q) + t0 * p.q_stride + h * p.q_head_stride;
        T* d = static_cast<T*>(p.q_out) + t0 * p.q_out_stride + h * p.q_out_head_stride;
        const int o0 = first(r), o1 = second(r);
        for (int t = begin; t < nt; t += U * step) {
            RVec<T, VEC> a[U], b[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (t + u * step >= nt) break;
                const T* x = s + (t + u * step) * p.q_stride;
                a[u] = load_vec<T, VEC>(x + o0);
                b[u] = load_vec<T, VEC>(x + o1);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (t + u * step >= nt) break;
                turn(a[u], b[u], t + u * step, r);
                T* y = d + (t + u * step) * p.q_out_stride;
                store_vec<T, VEC>(y + o0, a[u]);
                store_vec<T, VEC>(y + o1, b[u]);
            }
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
    const int64_t items = (int64_t)a.num_heads * (a.rope_dim / (vec ? 2 * V : 2));
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
