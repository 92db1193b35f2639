// dense.cuh -- element types and activations of the dense layers (group norm,
// linear, dropout).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/mqc.h"

namespace mqc {

// Values are widened exactly and rounded once, to nearest even.
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// Two consecutive elements in one 32-bit word (16-bit types).
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const T lo = from_f32<T>(a), hi = from_f32<T>(b);
    return static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(&lo)) |
           (static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(&hi)) << 16);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// One 16-byte vector of elements, as floats: 4 (fp32) or 8 (16-bit types).
template <typename T>
struct Vec {
    static constexpr int n = 16 / sizeof(T);
    __device__ static __forceinline__ void widen(const uint4 &w, float (&v)[n]) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2<T>(u[i]);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
    __device__ static __forceinline__ uint4 narrow(const float (&v)[n]) {
        return make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
    }
};
template <>
struct Vec<float> {
    static constexpr int n = 4;
    __device__ static __forceinline__ void widen(const uint4 &w, float (&v)[n]) {
        v[0] = __uint_as_float(w.x);
        v[1] = __uint_as_float(w.y);
        v[2] = __uint_as_float(w.z);
        v[3] = __uint_as_float(w.w);
    }
    __device__ static __forceinline__ uint4 narrow(const float (&v)[n]) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
};

// Activations in fp32.  ReLU passes NaN on.  SiLU uses CUDA's fast exponential
// and division (a relative error of a few 2^-23 where the value matters).
// GELU takes the normal distribution from Abramowitz and Stegun 7.1.26
// (Handbook of Mathematical Functions, 1964): erfc(x) = t (a1 + ... + a5 t^4)
// exp(-x^2), t = 1 / (1 + p x), off by at most 1.5e-7: one reciprocal and one
// exponential without a branch (erff has two ranges, and lanes of both in a
// warp pay for both).
struct Relu {
    __device__ static __forceinline__ float value(float z) { return z < 0.f ? 0.f : z; }
    __device__ static __forceinline__ float slope(float z) { return z > 0.f ? 1.f : 0.f; }
};
struct Silu {
    __device__ static __forceinline__ float value(float z) { return __fdividef(z, 1.f + __expf(-z)); }
    // q (1 + z (1 - q)), q = sigmoid(z)
    __device__ static __forceinline__ float slope(float z) {
        const float q = __fdividef(1.f, 1.f + __expf(-z));
        return q * (1.f + z * (1.f - q));
    }
};
struct Gelu {
    // Phi(z), with e = exp(-z^2 / 2)
    __device__ static __forceinline__ float phi(float z, float e) {
        const float t = __fdividef(1.f, fmaf(0.3275911f * 0.70710678118654752f, fabsf(z), 1.f));
        float c = fmaf(1.061405429f, t, -1.453152027f);
        c = fmaf(c, t, 1.421413741f);
        c = fmaf(c, t, -0.284496736f);
        c = fmaf(c, t, 0.254829592f);
        c = 0.5f * c * t * e;
        return z > 0.f ? 1.f - c : c;
    }
    __device__ static __forceinline__ float value(float z) { return z * phi(z, __expf(-0.5f * z * z)); }
    __device__ static __forceinline__ float slope(float z) {
        const float e = __expf(-0.5f * z * z);
        return fmaf(z * 0.39894228040143268f, e, phi(z, e));
    }
};

// v = act(v); s = act'(z).  One branch for all N elements.
template <int N>
__device__ __forceinline__ void act_values(int act, float (&v)[N]) {
    if (act == MQC_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = Relu::value(v[i]);
    } else if (act == MQC_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = Silu::value(v[i]);
    } else if (act == MQC_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = Gelu::value(v[i]);
    }
}
template <int N>
__device__ __forceinline__ void act_slopes(int act, const float (&z)[N], float (&s)[N]) {
    if (act == MQC_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = Relu::slope(z[i]);
    } else if (act == MQC_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = Silu::slope(z[i]);
    } else if (act == MQC_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = Gelu::slope(z[i]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = 1.f;
    }
}
__device__ __forceinline__ float act_value(int act, float z) {
    float v[1] = {z};
    act_values(act, v);
    return v[0];
}

}  // namespace mqc
