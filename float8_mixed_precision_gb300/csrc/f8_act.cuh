// Activations of a linear's epilogue and their slopes, on two fp32 elements at a
// time, for the GEMM epilogue and the backward pass.
//
// SiLU and tanh-GELU are z p with p = 1 / (1 + 2^-v), v = z log2 e or 2 u log2 e,
// by the hardware's 2^x and reciprocal (their relative errors, 2^-22 each, and
// that of v's rounding, |v| 2^-24, stay far below bf16's half step of 2^-9).
// GELU needs Phi in relative terms on the negative side, where 1 + erf would
// cancel: for x = |z|,
//   Phi(-x) = exp(-x^2 / 2) t Q(t),   t = 1 / (1 + 0.375 x),
// since exp(x^2 / 2) Phi(-x) falls like 1 / x.  Q is a polynomial of degree 8,
// fitted here to 2.3e-7 of the function's value over all x >= 0 (4.6e-7 in fp32).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "f8.h"

namespace f8 {
namespace act {

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

__device__ __forceinline__ float exp2_fast(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float rcp_fast(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

constexpr float kLog2E = 1.44269504f;
constexpr float kTanhC = 0.797884561f;  // sqrt(2 / pi)
constexpr float kTanhK = 0.044715f;
// past |z| = 16 the cubic's share no longer changes either value in fp32's range
constexpr float kTanhMax2 = 256.0f;

// 1 / (1 + 2^-v)
__device__ __forceinline__ float2 sigmoid2(float2 v)
{
    const float2 d = __fadd2_rn(both(1.0f), make_float2(exp2_fast(-v.x), exp2_fast(-v.y)));
    return make_float2(rcp_fast(d.x), rcp_fast(d.y));
}

// v of tanh-GELU, and min(z^2, 256)
__device__ __forceinline__ float2 tanh_arg(float2 z, float2 &zz)
{
    zz = __fmul2_rn(z, z);
    zz = make_float2(fminf(zz.x, kTanhMax2), fminf(zz.y, kTanhMax2));
    const float2 c = __ffma2_rn(zz, both(2.0f * kLog2E * kTanhC * kTanhK), both(2.0f * kLog2E * kTanhC));
    return __fmul2_rn(z, c);
}

// Phi(z), and e = exp(-z^2 / 2)
__device__ __forceinline__ float2 normal_cdf(float2 z, float2 &e)
{
    const float2 x = make_float2(fabsf(z.x), fabsf(z.y));
    const float2 d = __ffma2_rn(x, both(0.375f), both(1.0f));
    const float2 t = make_float2(rcp_fast(d.x), rcp_fast(d.y));
    const float2 w = __fmul2_rn(__fmul2_rn(z, z), both(-0.5f * kLog2E));
    e = make_float2(exp2_fast(w.x), exp2_fast(w.y));
    float2 q = __ffma2_rn(t, both(-0.0329106866f), both(0.136878276f));
    q = __ffma2_rn(q, t, both(-0.186518065f));
    q = __ffma2_rn(q, t, both(0.0506291793f));
    q = __ffma2_rn(q, t, both(0.0156298455f));
    q = __ffma2_rn(q, t, both(0.0886375539f));
    q = __ffma2_rn(q, t, both(0.128445827f));
    q = __ffma2_rn(q, t, both(0.149604573f));
    q = __ffma2_rn(q, t, both(0.149603386f));
    q = __fmul2_rn(__fmul2_rn(q, t), e);
    return make_float2(z.x < 0.0f ? q.x : 1.0f - q.x, z.y < 0.0f ? q.y : 1.0f - q.y);
}

template <int ACT>
__device__ __forceinline__ float2 value(float2 z)
{
    if (ACT == F8_ACT_RELU)
        return make_float2(z.x < 0.0f ? 0.0f : z.x, z.y < 0.0f ? 0.0f : z.y);
    if (ACT == F8_ACT_RELU2) {
        z = make_float2(z.x < 0.0f ? 0.0f : z.x, z.y < 0.0f ? 0.0f : z.y);
        return __fmul2_rn(z, z);
    }
    if (ACT == F8_ACT_SILU)
        return __fmul2_rn(z, sigmoid2(__fmul2_rn(z, both(kLog2E))));
    if (ACT == F8_ACT_GELU) {
        float2 e;
        return __fmul2_rn(z, normal_cdf(z, e));
    }
    if (ACT == F8_ACT_GELU_TANH) {
        float2 zz;
        return __fmul2_rn(z, sigmoid2(tanh_arg(z, zz)));
    }
    return z;
}

// act'(z).  With p the sigmoid, z p has the slope p + p z (1 - p) v', v' = 1 for
// SiLU and 2 u' for tanh-GELU; z Phi has Phi + z exp(-z^2 / 2) / sqrt(2 pi).
template <int ACT>
__device__ __forceinline__ float2 slope(float2 z)
{
    if (ACT == F8_ACT_RELU)  // NaN passes
        return make_float2(z.x <= 0.0f ? 0.0f : (z.x > 0.0f ? 1.0f : z.x),
                           z.y <= 0.0f ? 0.0f : (z.y > 0.0f ? 1.0f : z.y));
    if (ACT == F8_ACT_RELU2)
        return make_float2(z.x <= 0.0f ? 0.0f : 2.0f * z.x, z.y <= 0.0f ? 0.0f : 2.0f * z.y);
    if (ACT == F8_ACT_SILU) {
        const float2 p = sigmoid2(__fmul2_rn(z, both(kLog2E)));
        const float2 q = __ffma2_rn(p, both(-1.0f), both(1.0f));
        return __fmul2_rn(p, __ffma2_rn(z, q, both(1.0f)));
    }
    if (ACT == F8_ACT_GELU) {
        float2 e;
        const float2 c = normal_cdf(z, e);
        return __ffma2_rn(__fmul2_rn(z, e), both(0.398942280f), c);
    }
    if (ACT == F8_ACT_GELU_TANH) {
        float2 zz;
        const float2 p = sigmoid2(tanh_arg(z, zz));
        const float2 q = __ffma2_rn(p, both(-1.0f), both(1.0f));
        const float2 du = __ffma2_rn(zz, both(6.0f * kTanhC * kTanhK), both(2.0f * kTanhC));
        // p z q first: it is 0 wherever z is too large for z u' to hold
        return __ffma2_rn(__fmul2_rn(__fmul2_rn(p, z), q), du, p);
    }
    return both(1.0f);
}

} // namespace act
} // namespace f8
