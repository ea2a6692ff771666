// Elements and activations of the operators around a recurrent layer.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "tc_ptx.cuh"

namespace gla {

__device__ __forceinline__ float get(const float *p) { return *p; }
__device__ __forceinline__ float get(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void put(float *p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// kV elements of T at once, in memory and as floats: 16 bytes, 8 or one element.
template <typename T, int kV>
struct Pack;
template <>
struct Pack<float, 1> {
    using raw = float;
    static __device__ __forceinline__ void unpack(raw v, float (&f)[1]) { f[0] = v; }
    static __device__ __forceinline__ raw pack(const float (&f)[1]) { return f[0]; }
};
template <>
struct Pack<__nv_bfloat16, 1> {
    using raw = uint16_t;
    static __device__ __forceinline__ void unpack(raw v, float (&f)[1]) { f[0] = __uint_as_float((uint32_t)v << 16); }
    static __device__ __forceinline__ raw pack(const float (&f)[1]) {
        return __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
    }
};
template <>
struct Pack<float, 4> {
    using raw = uint4;
    static __device__ __forceinline__ void unpack(raw v, float (&f)[4]) {
        f[0] = __uint_as_float(v.x);
        f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z);
        f[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ raw pack(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};
template <>
struct Pack<__nv_bfloat16, 8> {
    using raw = uint4;
    static __device__ __forceinline__ void unpack(raw v, float (&f)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ raw pack(const float (&f)[8]) {
        return make_uint4(tc::pack_bf16(f[0], f[1]), tc::pack_bf16(f[2], f[3]), tc::pack_bf16(f[4], f[5]),
                          tc::pack_bf16(f[6], f[7]));
    }
};
template <>
struct Pack<__nv_bfloat16, 4> {
    using raw = uint2;
    static __device__ __forceinline__ void unpack(raw v, float (&f)[4]) {
        f[0] = __uint_as_float(v.x << 16);
        f[1] = __uint_as_float(v.x & 0xffff0000u);
        f[2] = __uint_as_float(v.y << 16);
        f[3] = __uint_as_float(v.y & 0xffff0000u);
    }
    static __device__ __forceinline__ raw pack(const float (&f)[4]) {
        return make_uint2(tc::pack_bf16(f[0], f[1]), tc::pack_bf16(f[2], f[3]));
    }
};

// The logistic function 1 / (1 + 2^(-u log2 e)). Results that are rounded to bf16 take the hardware's
// approximate exponential and reciprocal, flushing denormals: good to a few 2^-22 of the value, and where u < 0 to
// another 2^-23 |u|, from the rounding of u log2 e.
template <typename T>
__device__ __forceinline__ float logistic(float u) {
    if (sizeof(T) == 4) return 1.f / (1.f + expf(-u));
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(u * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}
// u and its derivative under the activation (0 none, 1 silu, 2 gelu).
template <typename T>
__device__ __forceinline__ float act_of(float u, int act) {
    if (act == 1) return u * logistic<T>(u);
    if (act == 2) return 0.5f * u * (1.f + erff(u * 0.70710678f));
    return u;
}
template <typename T>
__device__ __forceinline__ float act_grad(float u, int act) {
    if (act == 1) {
        const float s = logistic<T>(u);
        return s * (1.f + u * (1.f - s));
    }
    if (act == 2)
        return 0.5f * (1.f + erff(u * 0.70710678f)) + u * expf(-0.5f * u * u) * 0.39894228f;
    return 1.f;
}

}  // namespace gla
