// pa_rotary.cuh -- angles and rotations shared by the kernels that write
// rotated rows (pa_rope.cu, pa_latent_write.cu).
#pragma once

#include <stdint.h>
#include <string.h>

#include "pa_device.cuh"

namespace pa {

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

// Cosine and sine of position * freq (pa_rope.cu says how exact they are).
__device__ __forceinline__ float2 turn_of(int64_t position, double freq) {
    const uint64_t turns = (uint64_t)position * turn_fraction(freq);
    // the nearest 32-bit fraction, as half turns in [-1, 1)
    const float x = (float)(int32_t)((turns + 0x80000000ull) >> 32) * 4.656612873077393e-10f;
    float s, c;
    sincospif(x, &s, &c);
    if (!isfinite(freq)) s = c = __int_as_float(0x7fc00000);
    return make_float2(c, s);
}

}  // namespace pa
