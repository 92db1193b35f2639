// dense.cuh -- element types and activations of the dense layers (group norm,
// linear, dropout).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/mqc.h"

namespace mqc {

// Dependent launches: the second kernel of a call starts when the first one's
// last blocks have, and sets up meanwhile; before it touches what the first
// one leaves (or overwrites what it reads) it waits for that grid's end.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

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

// Two fp32 values in one register pair: sm_100 adds, multiplies and fuses both
// with one instruction, each rounded as the plain operation is.
__device__ __forceinline__ uint64_t bits2(float2 v) {
    uint64_t b;
    asm("mov.b64 %0, {%1, %2};" : "=l"(b) : "f"(v.x), "f"(v.y));
    return b;
}
__device__ __forceinline__ float2 float2_of(uint64_t b) {
    float2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(b));
    return v;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return float2_of(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return float2_of(r);
}
__device__ __forceinline__ float2 mul2_ftz(float2 a, float2 b) {   // subnormal results as zero
    uint64_t r;
    asm("mul.rn.ftz.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return float2_of(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
    return float2_of(r);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// 2^x and 1/x, subnormals as zero (a relative error of about 2^-22).
__device__ __forceinline__ float2 exp2_2(float2 v) {
    float2 r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(v.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(v.y));
    return r;
}
__device__ __forceinline__ float2 rcp_2(float2 v) {
    float2 r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(v.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(v.y));
    return r;
}

// Activations in fp32, two elements at a time.  ReLU passes NaN on.  GELU takes
// the normal distribution at -a as P(t) exp(-a^2 / 2), t = 1 / (1 + 0.4 a), a
// form of Hastings' (Approximations for Digital Computers, 1955), with one
// reciprocal and one exponential and without a branch (erff has two ranges, and
// lanes of both in a warp pay for both).  P, of degree 8, is a fit of this
// form's own, by reweighted least squares (Lawson's iteration) on the relative
// error over a = 0 .. 13.5, which stays below 7e-8: so tails keep their bits.
// (Degree 5 in t, Abramowitz and Stegun 7.1.26, is off by 1.5e-7 absolutely:
// 0.05% at z = -4, more than a rounding to 16 bits.)
struct Relu {
    __device__ static __forceinline__ float2 value(float2 z) {
        return make_float2(z.x < 0.f ? 0.f : z.x, z.y < 0.f ? 0.f : z.y);
    }
    __device__ static __forceinline__ float2 slope(float2 z) {
        return make_float2(z.x > 0.f ? 1.f : 0.f, z.y > 0.f ? 1.f : 0.f);
    }
};
struct Silu {
    __device__ static __forceinline__ float2 sigmoid(float2 z) {
        return rcp_2(add2(exp2_2(mul2(z, both(-1.4426950408889634f))), both(1.f)));
    }
    __device__ static __forceinline__ float2 value(float2 z) { return mul2(z, sigmoid(z)); }
    // q + q z (1 - q), q = sigmoid(z)
    __device__ static __forceinline__ float2 slope_of(float2 z, float2 q) {
        const float2 m = make_float2(-q.x, -q.y);
        return fma2(q, fma2(m, z, z), q);
    }
    __device__ static __forceinline__ float2 slope(float2 z) { return slope_of(z, sigmoid(z)); }
};
// The same with one reciprocal for two elements, of the product of their
// denominators, where exponentials and reciprocals (an eighth of the rate of
// other arithmetic) bound a pass; an element's last bits then depend on its
// neighbour.  The denominators, up to 2^127 (an exponent that is larger or NaN
// becomes 127), are scaled by 2^-63, so that their product stays between 2^-126
// and 2^128; the last multiplication takes the scale out again and flushes what
// is below the normal numbers: sigmoid is 0 from z = -88 on, and z sigmoid with
// it.  128x256x14x14 bf16 backward takes 19.6 us; a branch to reciprocals of
// their own took 20.2, a bound of 2^62 with 0 for all below 19.7, and that
// bound alone, 18.8 us, would leave z = -1e20 at -22.
struct SiluPair {
    __device__ static __forceinline__ float2 sigmoid(float2 z) {
        constexpr float s = 0x1p-63f;
        float2 t = mul2(z, both(-1.4426950408889634f));
        t = make_float2(fminf(t.x, 127.f), fminf(t.y, 127.f));
        const float2 d = fma2(exp2_2(t), both(s), both(s));
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d.x * d.y));
        return mul2_ftz(mul2(make_float2(d.y, d.x), both(r)), both(s));
    }
    __device__ static __forceinline__ float2 value(float2 z) { return mul2(z, sigmoid(z)); }
    __device__ static __forceinline__ float2 slope(float2 z) { return Silu::slope_of(z, sigmoid(z)); }
};
struct Gelu {
    // P(t), in single operations, whose constants are immediates: pairs would
    // hold them in registers over a loop that may never take this branch
    // (128x256x14x14 bf16 backward with SiLU 20.3 us, now 19.6)
    __device__ static __forceinline__ float tail(float t) {
        float c = fmaf(-0.0400001481f, t, 0.202324226f);
        c = fmaf(c, t, -0.376809597f);
        c = fmaf(c, t, 0.254076332f);
        c = fmaf(c, t, -0.0142213432f);
        c = fmaf(c, t, 0.159076944f);
        c = fmaf(c, t, 0.155645937f);
        c = fmaf(c, t, 0.15992038f);
        return fmaf(c, t, -1.27575968e-05f);
    }
    // Phi(z), with e = exp(-z^2 / 2)
    __device__ static __forceinline__ float2 phi(float2 z, float2 e) {
        const float2 a = make_float2(fabsf(z.x), fabsf(z.y));
        const float2 t = rcp_2(fma2(a, both(0.4f), both(1.f)));
        float2 c = mul2(make_float2(tail(t.x), tail(t.y)), e);
        return make_float2(z.x > 0.f ? 1.f - c.x : c.x, z.y > 0.f ? 1.f - c.y : c.y);
    }
    __device__ static __forceinline__ float2 bell(float2 z) {
        return exp2_2(mul2(mul2(z, both(-0.5f * 1.4426950408889634f)), z));
    }
    __device__ static __forceinline__ float2 value(float2 z) { return mul2(z, phi(z, bell(z))); }
    __device__ static __forceinline__ float2 slope(float2 z) {
        const float2 e = bell(z);
        return fma2(mul2(z, both(0.39894228040143268f)), e, phi(z, e));
    }
};

// v = act(v); s = act'(z).  One branch for all N elements.  PAIR: SiLU with
// shared reciprocals.
template <bool FIRST, typename A, typename B>
struct Either { using type = A; };
template <typename A, typename B>
struct Either<false, A, B> { using type = B; };
template <typename A, int N>
__device__ __forceinline__ void map_values(float (&v)[N]) {
#pragma unroll
    for (int i = 0; i + 1 < N; i += 2) {
        const float2 r = A::value(make_float2(v[i], v[i + 1]));
        v[i] = r.x;
        v[i + 1] = r.y;
    }
    if (N % 2) v[N - 1] = A::value(both(v[N - 1])).x;
}
template <typename A, int N>
__device__ __forceinline__ void map_slopes(const float (&z)[N], float (&s)[N]) {
#pragma unroll
    for (int i = 0; i + 1 < N; i += 2) {
        const float2 r = A::slope(make_float2(z[i], z[i + 1]));
        s[i] = r.x;
        s[i + 1] = r.y;
    }
    if (N % 2) s[N - 1] = A::slope(both(z[N - 1])).x;
}
template <bool PAIR = false, int N>
__device__ __forceinline__ void act_values(int act, float (&v)[N]) {
    if (act == MQC_ACT_RELU) map_values<Relu>(v);
    else if (act == MQC_ACT_SILU) map_values<typename Either<PAIR, SiluPair, Silu>::type>(v);
    else if (act == MQC_ACT_GELU) map_values<Gelu>(v);
}
template <bool PAIR = false, int N>
__device__ __forceinline__ void act_slopes(int act, const float (&z)[N], float (&s)[N]) {
    if (act == MQC_ACT_RELU) {
        map_slopes<Relu>(z, s);
    } else if (act == MQC_ACT_SILU) {
        map_slopes<typename Either<PAIR, SiluPair, Silu>::type>(z, s);
    } else if (act == MQC_ACT_GELU) {
        map_slopes<Gelu>(z, s);
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

// Elementwise arithmetic on N fp32 values, two at a time where N is even.
template <int N>
__device__ __forceinline__ void add_to(float (&a)[N], const float (&b)[N]) {
#pragma unroll
    for (int i = 0; i + 1 < N; i += 2) {
        const float2 r = add2(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]));
        a[i] = r.x;
        a[i + 1] = r.y;
    }
    if (N % 2) a[N - 1] += b[N - 1];
}
template <int N>
__device__ __forceinline__ void mul_to(float (&a)[N], const float (&b)[N]) {
#pragma unroll
    for (int i = 0; i + 1 < N; i += 2) {
        const float2 r = mul2(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]));
        a[i] = r.x;
        a[i + 1] = r.y;
    }
    if (N % 2) a[N - 1] *= b[N - 1];
}
// r = a b + c
template <int N>
__device__ __forceinline__ void fma_to(float (&r)[N], const float (&a)[N], const float (&b)[N], const float (&c)[N]) {
#pragma unroll
    for (int i = 0; i + 1 < N; i += 2) {
        const float2 v = fma2(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]), make_float2(c[i], c[i + 1]));
        r[i] = v.x;
        r[i + 1] = v.y;
    }
    if (N % 2) r[N - 1] = fmaf(a[N - 1], b[N - 1], c[N - 1]);
}

}  // namespace mqc
