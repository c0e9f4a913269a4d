// The activations of a layer and their derivatives, in fp32.
#pragma once

#include "../../include/dense_int8_matrix.h"

namespace gemm {

__device__ __forceinline__ float rcp_approx(float x) {   // within one unit in the last place; 1 / inf = 0
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// exp(x) within (2 + 1.16 |x|) 2^-23 of itself (the product's rounding, and two
// units of ex2); below 2^-126 it is 0.  Without ftz each call carries the
// scaling of denormal results, four instructions more.
__device__ __forceinline__ float exp_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950409f));
    return r;
}
// log(x) of a normal x.
__device__ __forceinline__ float log_approx(float x) {
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r * 0.69314718056f;
}
// 1 / (1 + exp(-x)): no cancellation on either side, 0 and 1 at the infinities.
__device__ __forceinline__ float sigmoid(float x) { return rcp_approx(1.f + exp_approx(-x)); }

constexpr float kGeluTanhTwice = 1.5957691216f;    // 2 sqrt(2 / pi)
constexpr float kGeluTanhCube = 0.044715f;
constexpr float kNormalPeak = 0.39894228040f;      // 1 / sqrt(2 pi)

// Phi(-|v|), the normal distribution's tail, and exp(-v^2 / 2), which its
// derivative needs too.  With x = |v| / sqrt(2), erfc(x) exp(x^2) is a smooth
// function of t = 1 / (1 + 0.425 x): t times a polynomial of degree 7, fitted
// here over x <= 12 for the least relative error, 2.7e-7 (in exact arithmetic), so
// that the tail keeps its digits (1 + erf would cancel there): with fp32's
// roundings and the exponential's it is within (12.8 + 0.83 v^2) 2^-23 of itself.
// erfcf costs six times as much.
__device__ __forceinline__ float normal_tail(float v, float& e) {
    const float t = rcp_approx(fmaf(fabsf(v), 0.30052038f, 1.f));   // 0.425 / sqrt(2)
    e = exp_approx(-0.5f * v * v);
    float q = 0.0688852072f;
    q = fmaf(q, t, -0.3024713099f);
    q = fmaf(q, t, 0.3894520700f);
    q = fmaf(q, t, -0.0868048817f);
    q = fmaf(q, t, 0.2465598583f);
    q = fmaf(q, t, 0.2032268792f);
    q = fmaf(q, t, 0.2414486110f);
    q = fmaf(q, t, 0.2397032976f);
    return 0.5f * (q * t) * e;
}

template <int ACT>
__device__ __forceinline__ float activate(float v) {
    if constexpr (ACT == GEMM_ACT_RELU) return v > 0.f || v != v ? v : 0.f;
    if constexpr (ACT == GEMM_ACT_GELU) {
        float e;
        const float tail = normal_tail(v, e);
        return v * (v > 0.f ? 1.f - tail : tail);
    }
    if constexpr (ACT == GEMM_ACT_GELU_TANH) return v * sigmoid(kGeluTanhTwice * (v + kGeluTanhCube * v * v * v));
    if constexpr (ACT == GEMM_ACT_SILU) return v * sigmoid(v);
    return v;
}

// g times the derivative at z.
template <int ACT>
__device__ __forceinline__ float activate_gradient(float g, float z) {
    if constexpr (ACT == GEMM_ACT_RELU) return z > 0.f ? g : z != z ? z : 0.f;
    if constexpr (ACT == GEMM_ACT_GELU) {
        float e;
        const float tail = normal_tail(z, e);
        return g * fmaf(z * kNormalPeak, e, z > 0.f ? 1.f - tail : tail);
    }
    if constexpr (ACT == GEMM_ACT_GELU_TANH) {
        // past |z| = 20 the slope is 0 or 1 to the last bit; there z^3 could overflow against s (1 - s) = 0
        const float x = fminf(fmaxf(z, -20.f), 20.f);
        const float s = sigmoid(kGeluTanhTwice * (x + kGeluTanhCube * x * x * x));
        const float slope = fmaf(x * s * (1.f - s), kGeluTanhTwice * fmaf(3.f * kGeluTanhCube, x * x, 1.f), s);
        return z != z ? z : g * slope;
    }
    if constexpr (ACT == GEMM_ACT_SILU) {
        const float s = sigmoid(z);
        return g * (s * fmaf(z, 1.f - s, 1.f));
    }
    return g;
}

// v[i] = act(v[i]), or with GEMM_ACT_GRADIENT v[i] times the derivative at z(i).
template <int ACT, int N, typename Z>
__device__ __forceinline__ void activate_each(float (&v)[N], Z z) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if constexpr ((ACT & GEMM_ACT_GRADIENT) != 0)
            v[i] = activate_gradient<ACT & ~GEMM_ACT_GRADIENT>(v[i], z(i));
        else
            v[i] = activate<ACT>(v[i]);
    }
}

}  // namespace gemm
