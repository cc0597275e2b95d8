// pa_rope.cu -- rotary positions on one or more axes, applied to q and k in
// the kernel that writes K and V to their slots.
//
// For token t and rotary pair i (rot_dim / 2 of them per head),
//   angle = positions[axis(i), t] * inv_freq[i],
//   (x1, x2) -> (x1 cos - x2 sin, x2 cos + x1 sin),
// where the pair is elements (i, i + rot_dim / 2) of the head, or (2i, 2i+1)
// when interleaved; elements from rot_dim on are passed through.  The rotated
// q goes to q_out, the rotated k and the unchanged v to row slot_mapping[t]
// of the pool, exactly where the plain write puts a row ("分页 KV Cache",
// PagedKVCache.write) -- or, into a quantized cache, as E4M3 codes with one
// scale per (token, KV head) row, quantized as the quantizing write does it
// from the fp32 rotated values (one rounding, not two).
//
// Angles.  A product of a far position and a frequency has no correct
// fraction of a turn in fp32 (at position 2^20 the spacing of fp32 is 1/8
// radian).  Here inv_freq[i] / (2 pi) becomes a 64-bit fraction of a turn F
// by one integer product of its significand with 2^64 / (2 pi); the
// position's turn is the low 64 bits of position * F (whole turns drop out of
// the wrap-around, negative positions included), and sincospif takes its upper
// 32 bits.  F is off by less than 1 + freq units of 2^-64 turns, which the
// position multiplies: below fp32's rounding of the angle (2^-26 turns) up to
// 2^37, 2^-18 turns at 2^45.  No fp64 instruction is spent on it.
//
// Bound: HBM.  q, k and v are read once and q_out and the rows written once.
// A block takes `tpb` tokens: their sines and cosines go to shared memory
// once and serve all heads; then every thread works 16-byte vectors, a
// rotated item being the two vectors that hold both halves of 8 (16-bit) or
// 4 (fp32) pairs, the same item for all of the block's tokens.
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_launch.cuh"

namespace pa {
namespace {

constexpr int kRopeThreads = 256;  // at most

// inv_freq / (2 pi) as a fraction of a turn in 64 bits (two's complement).
// freq = m 2^e with a 53-bit integer m: F = m * (2^64 / (2 pi)) * 2^e, whole
// turns dropped; the truncations are below one unit of 2^-64 turns times
// max(1, freq).
__device__ __forceinline__ uint64_t turn_fraction(double freq) {
    const uint64_t b = (uint64_t)__double_as_longlong(freq);
    const int ex = (int)((b >> 52) & 0x7ff);
    uint64_t m = b & 0xfffffffffffffull;
    if (ex) m |= 1ull << 52;
    const uint64_t c = 0x28be60db9391054aull;  // floor(2^64 / (2 pi))
    const uint64_t lo = m * c, hi = __umul64hi(m, c);
    const int sh = 1075 - (ex ? ex : 1);  // -e
    uint64_t f = 0;
    if (sh <= 0) f = -sh < 64 ? lo << -sh : 0;
    else if (sh < 64) f = (hi << (64 - sh)) | (lo >> sh);
    else if (sh < 128) f = hi >> (sh - 64);
    return (b >> 63) ? 0 - f : f;
}

template <typename T, int VEC> struct alignas(VEC == 1 ? sizeof(T) : 16) RVec { T e[VEC]; };

template <typename T, int VEC>
__device__ __forceinline__ RVec<T, VEC> load_vec(const T* p) {
    RVec<T, VEC> v;
    if constexpr (VEC == 1) {
        v.e[0] = *p;
    } else {
        uint4 r;
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
        memcpy(&v, &r, 16);
    }
    return v;
}
template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const RVec<T, VEC>& v) {
    *reinterpret_cast<RVec<T, VEC>*>(p) = v;
}

template <typename T, int VEC>
__device__ __forceinline__ void unpack(const RVec<T, VEC>& v, float (&x)[VEC]) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[e] = Elt<T>::to_f(v.e[e]);
}
// Rotates the pairs held in a and b; cs: their cosines and sines.
template <int VEC>
__device__ __forceinline__ void rotate(float (&a)[VEC], float (&b)[VEC], const float2* cs, bool interleaved) {
    if (VEC > 1 && interleaved) {
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) {
            const float2 c0 = cs[e], c1 = cs[VEC / 2 + e];
            const float x0 = a[2 * e], y0 = a[2 * e + 1], x1 = b[2 * e], y1 = b[2 * e + 1];
            a[2 * e] = x0 * c0.x - y0 * c0.y;
            a[2 * e + 1] = y0 * c0.x + x0 * c0.y;
            b[2 * e] = x1 * c1.x - y1 * c1.y;
            b[2 * e + 1] = y1 * c1.x + x1 * c1.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float2 c = cs[e];
            const float x = a[e], y = b[e];
            a[e] = x * c.x - y * c.y;
            b[e] = y * c.x + x * c.y;
        }
    }
}
// VEC codes of x / sc, as the quantizing write rounds them.
template <int VEC>
__device__ __forceinline__ void store_codes(uint8_t* d, const float (&x)[VEC], float sc) {
    uint32_t w[(VEC + 3) / 4] = {};
#pragma unroll
    for (int e = 0; e < VEC; ++e)
        w[e / 4] |= (uint32_t)__nv_cvt_float_to_fp8(__fdiv_rn(x[e], sc), __NV_SATFINITE, __NV_E4M3) << (8 * (e % 4));
    if constexpr (VEC == 8) *reinterpret_cast<uint2*>(d) = make_uint2(w[0], w[1]);
    else if constexpr (VEC == 4) *reinterpret_cast<uint32_t*>(d) = w[0];
    else *d = (uint8_t)w[0];
}

// VEC: elements per vector (16 bytes, or 1 where sizes or alignment do not
// allow it).  FP8: k and v rows are quantized into code pools.
// 1,024 threads per SM and two tokens in flight per thread: measured on 8,192
// tokens of 32 + 8 heads x 128 (bf16) against one to four in flight and two to
// six CTAs.
template <typename T, int VEC, bool FP8>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_write_kernel(const RopeArgs p) {
    constexpr int U = 2;  // tokens in flight per thread
    extern __shared__ float2 tab[];  // [tpb][rot / 2] cosine, sine; then the tokens' slots
    pdl_wait_primary();
    pdl_launch_dependents();
    const int64_t t0 = (int64_t)blockIdx.x * p.tpb;
    const int nt = (int)min((int64_t)p.tpb, p.n - t0);
    const int half = p.rot_dim / 2, hd = p.head_dim, Hq = p.num_heads, Hkv = p.num_kv_heads;
    int64_t* slots = reinterpret_cast<int64_t*>(tab + (size_t)p.tpb * half);
    const int NT = blockDim.x;
    for (int i = threadIdx.x; i < nt; i += NT) slots[i] = p.slots[t0 + i];
    for (int i = threadIdx.x; i < nt * half; i += NT) {
        const int t = i / half, pr = i - t * half;
        const int ax = p.pair_axis ? min(max(p.pair_axis[pr], 0), p.num_axes - 1) : 0;
        const double fr = p.inv_freq[pr];
        const uint64_t turns = (uint64_t)p.positions[(int64_t)ax * p.n + t0 + t] * turn_fraction(fr);
        // the nearest 32-bit fraction, as half turns in [-1, 1)
        const float x = (float)(int32_t)((turns + 0x80000000ull) >> 32) * 4.656612873077393e-10f;
        float s, c;
        sincospif(x, &s, &c);
        if (!isfinite(fr)) s = c = __int_as_float(0x7fc00000);
        tab[i] = make_float2(c, s);
    }
    __syncthreads();

    // A token's items, two vectors each: per head of q and k those that hold
    // both halves of VEC rotary pairs, then the rest of the head two by two;
    // per head of v all of it two by two.  A thread finds its item once and
    // works it for all tokens of the CTA.  Code pools: the items of a row are
    // neighbouring lanes (a power of two of them), which share the row's
    // maximum; the element-wise form (VEC 1) quantizes below instead.
    constexpr bool kCodes = FP8 && VEC > 1, kRowsBelow = FP8 && VEC == 1;
    const int R = half / VEC, per = R + ((hd - p.rot_dim) / VEC + 1) / 2;
    const int n_rot = (Hq + (kRowsBelow ? 0 : Hkv)) * per, vper = (hd / VEC + 1) / 2;
    const int items = n_rot + (kRowsBelow ? 0 : Hkv * vper);
    for (int it = blockIdx.y * NT + threadIdx.x; it < items; it += gridDim.y * NT) {
        const bool is_v = it >= n_rot;
        int head = is_v ? (it - n_rot) / vper : it / per;
        const int r = is_v ? it - n_rot - head * vper : it - head * per;
        const bool is_q = head < Hq && !is_v, turned = !is_v && r < R;
        if (!is_v && !is_q) head -= Hq;
        const T* src = static_cast<const T*>(is_v ? p.v : is_q ? p.q : p.k);
        const int64_t stride = is_v ? p.v_stride : is_q ? p.q_stride : p.k_stride;  // between tokens
        src += t0 * stride + (int64_t)head * hd;
        const int64_t row = (int64_t)(is_q ? Hq : Hkv) * hd;  // of the destination
        const int64_t dst = (is_q ? t0 * row : 0) + (int64_t)head * hd;
        const int pr = r * VEC;  // the first pair
        int o0, o1;
        if (turned) {
            o0 = p.interleaved ? 2 * pr : pr;
            o1 = p.interleaved ? o0 + VEC : o0 + half;
        } else {
            o0 = is_v ? 2 * r * VEC : p.rot_dim + 2 * (r - R) * VEC;
            o1 = o0 + VEC < hd ? o0 + VEC : -1;
        }
        for (int t = 0; t < nt; t += U) {
            RVec<T, VEC> a[U], b[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (t + u >= nt) break;
                const T* s = src + (t + u) * stride;
                a[u] = load_vec<T, VEC>(s + o0);
                if (VEC > 1 || o1 >= 0) b[u] = load_vec<T, VEC>(s + o1);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (t + u >= nt) break;
                const int64_t slot = is_q ? t + u : slots[t + u];
                if (slot < 0) continue;  // a padding token's k or v
                const float2* cs = tab + (t + u) * half + pr;
                if (kCodes && !is_q) {
                    float x[2][VEC];
                    unpack<T, VEC>(a[u], x[0]);
                    unpack<T, VEC>(b[u], x[1]);
                    if (turned) rotate<VEC>(x[0], x[1], cs, p.interleaved);
                    float amax = 0.f;
#pragma unroll
                    for (int e = 0; e < VEC; ++e) amax = fmaxf(amax, fmaxf(fabsf(x[0][e]), fabsf(x[1][e])));
                    const uint32_t lanes = (per == 32 ? 0xffffffffu : (1u << per) - 1u) << (threadIdx.x & 31 & ~(per - 1));
                    for (int o = 1; o < per; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(lanes, amax, o));
                    const float sc = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
                    uint8_t* d = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + dst + slot * row;
                    store_codes<VEC>(d + o0, x[0], sc);
                    store_codes<VEC>(d + o1, x[1], sc);
                    if (r == 0) {
                        const int64_t blk = slot / p.block_size, off = slot - blk * p.block_size;
                        (is_v ? p.v_scales : p.k_scales)[(blk * Hkv + head) * p.block_size + off] = sc;
                    }
                    continue;
                }
                T* d = static_cast<T*>(is_q ? p.q_out : is_v ? p.v_cache : p.k_cache) + dst + slot * row;
                if (turned) {
                    float x[2][VEC];
                    unpack<T, VEC>(a[u], x[0]);
                    unpack<T, VEC>(b[u], x[1]);
                    rotate<VEC>(x[0], x[1], cs, p.interleaved);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        a[u].e[e] = Elt<T>::from_f(x[0][e]);
                        b[u].e[e] = Elt<T>::from_f(x[1][e]);
                    }
                }
                store_vec<T, VEC>(d + o0, a[u]);
                if (VEC > 1 || o1 >= 0) store_vec<T, VEC>(d + o1, b[u]);
            }
        }
    }

    if constexpr (kRowsBelow) {
        const T* k = static_cast<const T*>(p.k);
        const T* v = static_cast<const T*>(p.v);
        // one warp per (token, KV head, K|V) row: lane l holds pairs l, l+32,
        // ... of the rotated part and elements rot + l, ... of the rest
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        for (int row = blockIdx.y * (NT / 32) + warp; row < nt * Hkv * 2; row += gridDim.y * (NT / 32)) {
            const int is_v = row & 1, h = (row >> 1) % Hkv, t = (row >> 1) / Hkv;
            const int64_t tok = t0 + t, slot = slots[t];
            if (slot < 0) continue;
            const T* src = is_v ? v + tok * p.v_stride + (int64_t)h * hd : k + tok * p.k_stride + (int64_t)h * hd;
            const int rot = is_v ? 0 : p.rot_dim, hf = rot / 2;
            float x[4], y[4], z[8], amax = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int pr = lane + 32 * i;
                if (pr >= hf) break;
                const float2 c = tab[t * half + pr];
                const float x0 = Elt<T>::to_f(src[p.interleaved ? 2 * pr : pr]);
                const float y0 = Elt<T>::to_f(src[p.interleaved ? 2 * pr + 1 : pr + hf]);
                x[i] = x0 * c.x - y0 * c.y;
                y[i] = y0 * c.x + x0 * c.y;
                amax = fmaxf(amax, fmaxf(fabsf(x[i]), fabsf(y[i])));
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int e = rot + lane + 32 * i;
                if (e >= hd) break;
                z[i] = Elt<T>::to_f(src[e]);
                amax = fmaxf(amax, fabsf(z[i]));
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
            const float sc = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
            uint8_t* d = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + (slot * Hkv + h) * hd;
            auto code = [&](float f) {
                return (uint8_t)__nv_cvt_float_to_fp8(__fdiv_rn(f, sc), __NV_SATFINITE, __NV_E4M3);
            };
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int pr = lane + 32 * i;
                if (pr >= hf) break;
                d[p.interleaved ? 2 * pr : pr] = code(x[i]);
                d[p.interleaved ? 2 * pr + 1 : pr + hf] = code(y[i]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int e = rot + lane + 32 * i;
                if (e >= hd) break;
                d[e] = code(z[i]);
            }
            if (lane == 0) {
                const int64_t blk = slot / p.block_size, off = slot - blk * p.block_size;
                (is_v ? p.v_scales : p.k_scales)[(blk * Hkv + h) * p.block_size + off] = sc;
            }
        }
    }
}

template <typename T, bool FP8>
cudaError_t launch_rope_typed(const RopeArgs& a, cudaStream_t stream) {
    constexpr int V = 16 / (int)sizeof(T);
    const bool al = ((reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k) |
                      reinterpret_cast<uintptr_t>(a.v) | reinterpret_cast<uintptr_t>(a.q_out)) & 15) == 0;
    const int row_items = a.head_dim / (2 * V);  // code pools: a power of two up to a warp
    const bool vec = al && a.head_dim % (2 * V) == 0 && a.rot_dim % (2 * V) == 0 && a.q_stride % V == 0 &&
                     a.k_stride % V == 0 && a.v_stride % V == 0 &&
                     (!FP8 || ((row_items & (row_items - 1)) == 0 && row_items <= 32));
    RopeArgs p = a;
    // Threads per CTA: the number that the items of a token fill best (128
    // items left half of 256 threads idle: 1,999 code-pool tokens 9.5 us, 7.5
    // so).  Tokens per CTA: more spread the angles' and the items' setup over
    // more tokens; the batch in one wave of 1,024 threads per SM (8,192 tokens:
    // 37 us so, 39.5 in two waves).  Few tokens: their items over several CTAs
    // each, which repeat the angles.
    const int items = (a.num_heads + 2 * a.num_kv_heads) * (a.head_dim / (vec ? 2 * V : 2));
    auto filled = [&](int n) { return (int64_t)((items + n - 1) / n) * n; };
    int threads = 128;
    for (int n = 160; n <= kRopeThreads; n += 32)
        if (filled(n) < filled(threads)) threads = n;
    const int64_t slots = kSms * (1024 / threads);
    p.tpb = (int)std::min<int64_t>(16, (a.n + slots - 1) / slots);
    const int64_t ctas = (a.n + p.tpb - 1) / p.tpb;
    const int64_t parts = std::max<int64_t>(1, std::min<int64_t>(slots / 2 / ctas, (items + threads - 1) / threads));
    const dim3 grid((unsigned)ctas, (unsigned)parts);
    const size_t smem = (size_t)p.tpb * ((a.rot_dim / 2) * sizeof(float2) + sizeof(int64_t));
    return vec ? launch_pdl_smem(rope_write_kernel<T, V, FP8>, grid, dim3((unsigned)threads), smem, stream, p)
               : launch_pdl_smem(rope_write_kernel<T, 1, FP8>, grid, dim3((unsigned)threads), smem, stream, p);
}

}  // namespace

cudaError_t launch_rope_write(const RopeArgs& a, int dtype, bool fp8, cudaStream_t stream) {
    switch (dtype) {
        case 0: return fp8 ? launch_rope_typed<float, true>(a, stream) : launch_rope_typed<float, false>(a, stream);
        case 1: return fp8 ? launch_rope_typed<__nv_bfloat16, true>(a, stream)
                           : launch_rope_typed<__nv_bfloat16, false>(a, stream);
        default: return fp8 ? launch_rope_typed<__half, true>(a, stream)
                            : launch_rope_typed<__half, false>(a, stream);
    }
}

}  // namespace pa
