// Activations of the products with a packed layer, and their slopes, in fp32
// (gptq_activation in the header).  Each is written so that no intermediate
// value overflows into a NaN for a finite x, and so that the small values left
// of zero keep their relative accuracy (erfc and 1 / (1 + exp) instead of
// 1 + erf and 1 + tanh).  exp and the quotient are CUDA's approximate forms: a
// few units of 2^-23 plus the rounding of exp's argument.  Values go to bf16
// outputs (2^-8; with the exact forms a 256 x 256 output tile spent 56 us in its
// GELU, almost half of what its product takes; 16 us with one branch per value).
// Slopes also enter the fp32 bias gradient: over every bf16 x they are within 2.8
// units of 2^-24 of the true slope, where the formulas in plain fp32 with exact
// exp and tanh are within 1.6 (GELU), 9 (GELU_TANH) and 16 (SILU).
#pragma once

#include <cuda_runtime.h>

#include "../../include/gptq.h"

namespace gptq {

constexpr float kSqrt2OverPi = 0.79788456080286535588f;
constexpr float kInvSqrt2 = 0.70710678118654752440f;
constexpr float kInvSqrt2Pi = 0.39894228040143267794f;
constexpr float kGeluCubic = 0.044715f;

constexpr float kLog2E = 1.44269504088896340736f;

// 1 / (1 + 2^y); 2^y overflows to +inf beyond y = 128: 0 then
__device__ __forceinline__ float inv_one_plus_exp2(float y) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(y));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}
// ... and its product with one minus itself, p = 2^y / (1 + 2^y)^2, for the slopes
// (as h (1 - h) it loses all bits where h comes near 1: a SILU slope was off by
// 16 units of 2^-24, a GELU_TANH one by 32, and dbias is an fp32 output).  p is 0
// where 2^y or 2^-y is out of range.
__device__ __forceinline__ float logistic(float y, float& p) {
    float e, h;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(y));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(h) : "f"(1.f + e));
    p = h * (fminf(e, 0x1p125f) * h);   // (inf * 0 otherwise)
    return h;
}
__device__ __forceinline__ float sigmoid_f(float x) { return inv_one_plus_exp2(-kLog2E * x); }

// (1 + tanh(u)) / 2 = 1 / (1 + exp(-2u)), u = sqrt(2/pi) (x + 0.044715 x^3); the
// exponent of 2 in it
__device__ __forceinline__ float gelu_tanh_exponent(float x) {
    constexpr float k1 = -2.f * kLog2E * kSqrt2OverPi, k3 = k1 * kGeluCubic;
    return x * fmaf(k3, x * x, k1);
}
__device__ __forceinline__ float gelu_tanh_half(float x) { return inv_one_plus_exp2(gelu_tanh_exponent(x)); }

__device__ __forceinline__ float activate(float x, int act) {
    switch (act) {
        case GPTQ_ACT_RELU: return x < 0.f ? 0.f : x;  // a NaN stays one
        case GPTQ_ACT_GELU: return 0.5f * x * erfcf(-x * kInvSqrt2);
        case GPTQ_ACT_GELU_TANH: return x * gelu_tanh_half(x);
        case GPTQ_ACT_SILU: return x * sigmoid_f(x);
        default: return x;
    }
}

// N values at once (one branch on the activation)
template <int N>
__device__ __forceinline__ void activate_all(float (&v)[N], int act) {
    switch (act) {
        case GPTQ_ACT_RELU:
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] = activate(v[j], GPTQ_ACT_RELU);
            break;
        case GPTQ_ACT_GELU:
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] = activate(v[j], GPTQ_ACT_GELU);
            break;
        case GPTQ_ACT_GELU_TANH:
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] = activate(v[j], GPTQ_ACT_GELU_TANH);
            break;
        case GPTQ_ACT_SILU:
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] = activate(v[j], GPTQ_ACT_SILU);
            break;
        default: break;
    }
}

__device__ __forceinline__ float activate_slope(float x, int act) {
    switch (act) {
        case GPTQ_ACT_RELU: return x > 0.f ? 1.f : 0.f;
        case GPTQ_ACT_GELU:
            return 0.5f * erfcf(-x * kInvSqrt2) + x * kInvSqrt2Pi * __expf(-0.5f * x * x);
        case GPTQ_ACT_GELU_TANH: {
            float p;
            const float h = logistic(gelu_tanh_exponent(x), p);
            // p is 0 where x^2 may overflow
            return p == 0.f ? h
                            : h + 2.f * x * p * kSqrt2OverPi * (1.f + 3.f * kGeluCubic * x * x);
        }
        case GPTQ_ACT_SILU: {
            float p;
            const float s = logistic(-kLog2E * x, p);
            return p == 0.f ? s : s + x * p;   // p is 0 where x may be infinite
        }
        default: return 1.f;
    }
}

}  // namespace gptq
