// The activations of a layer and their derivatives, in fp32.
#pragma once

#include "../../include/dense_int8_matrix.h"

namespace gemm {

__device__ __forceinline__ float rcp_approx(float x) {   // within one unit in the last place; 1 / inf = 0
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// 1 / (1 + exp(-x)): no cancellation on either side, 0 and 1 at the infinities.
__device__ __forceinline__ float sigmoid(float x) { return rcp_approx(1.f + __expf(-x)); }

constexpr float kGeluTanhTwice = 1.5957691216f;    // 2 sqrt(2 / pi)
constexpr float kGeluTanhCube = 0.044715f;
constexpr float kRootHalf = 0.70710678119f;
constexpr float kNormalPeak = 0.39894228040f;      // 1 / sqrt(2 pi)

template <int ACT>
__device__ __forceinline__ float activate(float v) {
    if constexpr (ACT == GEMM_ACT_RELU) return v > 0.f || v != v ? v : 0.f;
    // erfc of the negative argument: 1 + erf would cancel in the left tail
    if constexpr (ACT == GEMM_ACT_GELU) return v * (0.5f * erfcf(-v * kRootHalf));
    if constexpr (ACT == GEMM_ACT_GELU_TANH) return v * sigmoid(kGeluTanhTwice * (v + kGeluTanhCube * v * v * v));
    if constexpr (ACT == GEMM_ACT_SILU) return v * sigmoid(v);
    return v;
}

// g times the derivative at z.
template <int ACT>
__device__ __forceinline__ float activate_gradient(float g, float z) {
    if constexpr (ACT == GEMM_ACT_RELU) return z > 0.f ? g : z != z ? z : 0.f;
    if constexpr (ACT == GEMM_ACT_GELU)
        return g * fmaf(z * kNormalPeak, __expf(-0.5f * z * z), 0.5f * erfcf(-z * kRootHalf));
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

// v[i] = act(v[i]), or v[i] times the derivative at z(i): one uniform branch
// for the N values.
template <int N, typename Z>
__device__ __forceinline__ void activate_all(int act, bool grad, float (&v)[N], Z z) {
#define GEMM_ACT_CASE(ACT)                                        \
    case ACT:                                                     \
        if (grad) {                                               \
            _Pragma("unroll") for (int i = 0; i < N; ++i) v[i] = activate_gradient<ACT>(v[i], z(i)); \
        } else {                                                  \
            _Pragma("unroll") for (int i = 0; i < N; ++i) v[i] = activate<ACT>(v[i]);                \
        }                                                         \
        break;
    switch (act) {
        GEMM_ACT_CASE(GEMM_ACT_RELU)
        GEMM_ACT_CASE(GEMM_ACT_GELU)
        GEMM_ACT_CASE(GEMM_ACT_GELU_TANH)
        GEMM_ACT_CASE(GEMM_ACT_SILU)
        default: break;
    }
#undef GEMM_ACT_CASE
}

}  // namespace gemm
