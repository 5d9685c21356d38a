// act.hpp -- activations of the feed-forward block, fp32 to fp32, shared by
// the GEMM's epilogue and the experts' kernels.
//
//   silu       x / (1 + e^-x)
//   gelu       x/2 erfc(-x / sqrt 2)
//   gelu_tanh  x / (1 + e^-2u),  u = sqrt(2/pi) (x + 0.044715 x^3)
//              (= x/2 (1 + tanh u))
//
// Each takes one exponential and one reciprocal by the hardware's instructions:
// e^-a through a log2(e) carries the exponent's roundings, at most 3 a 2^-24 with a <= 88,
// the reciprocal 2^-23, so a result is within 2^-15 of its value, against bf16's 2^-9;
// one below 2^-119 may come out as zero, where those instructions leave out the
// subnormal range.  What is not finite follows the formulas.
#pragma once
#include <hip/hip_runtime.h>

enum { ACT_NONE = 0, ACT_RELU = 1, ACT_SILU = 2, ACT_GELU = 3, ACT_GELU_TANH = 4 };

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float rcp_fast(float x) { return __builtin_amdgcn_rcpf(x); }

// x / (1 + 2^-y)
__device__ __forceinline__ float logistic_of(float x, float y) { return x * rcp_fast(1.0f + exp2_fast(-y)); }

// No sum of a product is left to the compiler to fuse or not, which it would choose for
// each kernel by itself: a row's result is the same in all of them.
template <int ACT>
__device__ __forceinline__ float act_one(float x) {
#pragma clang fp contract(off)
    constexpr float LOG2E = 1.44269504f;
    if constexpr (ACT == ACT_RELU) return x < 0.0f ? 0.0f : x;
    if constexpr (ACT == ACT_SILU) return logistic_of(x, x * LOG2E);
    if constexpr (ACT == ACT_GELU_TANH) {
        constexpr float C = 2.0f * 0.797884561f * LOG2E;   // 2 sqrt(2/pi) log2(e)
        return logistic_of(x, x * __builtin_fmaf(C * 0.044715f, x * x, C));
    }
    if constexpr (ACT == ACT_GELU) {
        // erfc(a / sqrt 2) = e^(-a^2/2) t P(t), t = 1 / (1 + 0.44 a / sqrt 2), a = |x|: P is
        // the polynomial of degree 7 whose largest relative error over 0 <= a / sqrt 2 <= 12
        // is least (1.9e-7), fitted to erfc's values.  No cancellation: for x < 0 the
        // result is x/2 erfc, for x >= 0 it is x - x/2 erfc with erfc <= 1.
        const float a = __builtin_fabsf(x);
        const float t = rcp_fast(__builtin_fmaf(0.311126977f, a, 1.0f));
        float p = 0.0714833736f;
        p = __builtin_fmaf(p, t, -0.279080987f);
        p = __builtin_fmaf(p, t, 0.298737288f);
        p = __builtin_fmaf(p, t, -0.0221683588f);
        p = __builtin_fmaf(p, t, 0.216923311f);
        p = __builtin_fmaf(p, t, 0.21695715f);
        p = __builtin_fmaf(p, t, 0.248931631f);
        p = __builtin_fmaf(p, t, 0.248216793f);
        const float h = 0.5f * (p * t), e = exp2_fast(x * x * (-0.5f * LOG2E));   // half erfc: h e
        return x * (x < 0.0f ? h * e : __builtin_fmaf(-h, e, 1.0f));
    }
    return x;
}

// The activation of N values, chosen by a wave-uniform code: one branch for all.
template <int N>
__device__ __forceinline__ void act_all(float (&v)[N], int act) {
    switch (act) {
    case ACT_RELU:
#pragma unroll
        for (int e = 0; e < N; e++) v[e] = act_one<ACT_RELU>(v[e]);
        break;
    case ACT_SILU:
#pragma unroll
        for (int e = 0; e < N; e++) v[e] = act_one<ACT_SILU>(v[e]);
        break;
    case ACT_GELU:
#pragma unroll
        for (int e = 0; e < N; e++) v[e] = act_one<ACT_GELU>(v[e]);
        break;
    case ACT_GELU_TANH:
#pragma unroll
        for (int e = 0; e < N; e++) v[e] = act_one<ACT_GELU_TANH>(v[e]);
        break;
    default: break;
    }
}
