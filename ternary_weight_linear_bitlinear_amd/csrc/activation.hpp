// Activations of the products' epilogue and their derivatives, in fp32.
//
// sigmoid(u) = 1 / (1 + 2^(-u log2 e)) with the hardware's exp2 and reciprocal
// (one ulp each). gelu with the error function needs e(x) = erfc(x / sqrt 2)
// for x >= 0, computed as 2^(-x^2 log2(e) / 2) times a polynomial in
// t = 1 / (1 + p x) (the form of Abramowitz & Stegun 7.1.26; the
// coefficients here are a fit of exp(x^2 / 2) erfc(x / sqrt 2) made for this
// file, see kErfcPoly). The tails decay with their function instead of ending at
// a multiple of fp32's step; their relative error is that of an exponent
// rounded to fp32: (1.5 z^2 + 24) 2^-24 at most for gelu (2e-6 at z = -6, 8e-6 at
// -13), (2 |z| + 8) 2^-24 for silu. Beside bf16's half step of 2^-8 that is nothing,
// so the exponent is not split in two. All of it is branch-free: at 2048 x 11008
// outputs each instruction per output costs about 0.6 us of a compute unit's
// vector time.
#pragma once

#include <hip/hip_runtime.h>

namespace bl {

constexpr int kActNone = 0, kActRelu = 1, kActRelu2 = 2, kActSilu = 3, kActGelu = 4,
              kActGeluTanh = 5;
constexpr int kActCount = 6;

#if defined(__HIPCC__)

constexpr float kLog2E = 1.44269504088896340736f;
constexpr float kGeluTanhC = 1.59576912160573071176f;  // 2 sqrt(2 / pi)
constexpr float kGeluTanhA = 0.044715f;
constexpr float kInvSqrt2Pi = 0.39894228040143267794f;

__device__ __forceinline__ float sigmoid_fast(float u) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2E * u));
}

// exp(x^2 / 2) erfc(x / sqrt 2) = t (c0 + c1 t + ... + c7 t^7), t = 1 / (1 + 0.3 x):
// least squares on Chebyshev nodes of t for x in [0, 14], reweighted towards
// the largest relative error. With these fp32 coefficients the fit is off by 1.7e-7
// relative, by 4.5e-7 as evaluated in fp32.
constexpr float kErfcP = 0.3f;
constexpr int kErfcTerms = 8;
constexpr float kErfcPoly[kErfcTerms] = {
    0.23925860226154327f,  0.24150793254375458f, 0.19982682168483734f, 0.2571238577365875f,
    -0.10736848413944244f, 0.4127083718776703f,  -0.31440699100494385f, 0.07134975492954254f};

// erfc(x / sqrt 2) for x = |z|; `g` = exp(-x^2 / 2).
__device__ __forceinline__ float erfc_sqrt2(float x, float g) {
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(kErfcP, x, 1.0f));
    float p = kErfcPoly[kErfcTerms - 1];
#pragma unroll
    for (int i = kErfcTerms - 2; i >= 0; --i) p = __builtin_fmaf(p, t, kErfcPoly[i]);
    return p * t * g;
}
__device__ __forceinline__ float half_gauss(float z) {  // exp(-z^2 / 2)
    return __builtin_amdgcn_exp2f(-0.5f * kLog2E * z * z);
}

__device__ __forceinline__ float gelu_erf(float z) {
    // z Phi(z) = max(z, 0) - |z| erfc(|z| / sqrt 2) / 2 on both sides
    const float x = fabsf(z);
    return __builtin_fmaf(-0.5f * x, erfc_sqrt2(x, half_gauss(z)), fmaxf(z, 0.0f));
}
// sigmoid(2 u), u = sqrt(2 / pi) (z + a z^3): 2^(-2 u log2 e) takes the constants in
__device__ __forceinline__ float gelu_tanh_gate(float z, float zz) {
    constexpr float k0 = -kLog2E * kGeluTanhC, k1 = k0 * kGeluTanhA;
    const float e = __builtin_amdgcn_exp2f(z * __builtin_fmaf(k1, zz, k0));
    return __builtin_amdgcn_rcpf(1.0f + e);
}
__device__ __forceinline__ float gelu_tanh(float z) {  // z (1 + tanh u) / 2 = z sigmoid(2 u)
    return z * gelu_tanh_gate(z, z * z);
}

// z = act(z) for each element; one branch (uniform over a launch) for all C.
template <int C>
__device__ __forceinline__ void activate_all(float (&z)[C], int act) {
    switch (act) {
        case kActRelu:
#pragma unroll
            for (int e = 0; e < C; ++e) z[e] = fmaxf(z[e], 0.0f);
            break;
        case kActRelu2:
#pragma unroll
            for (int e = 0; e < C; ++e) z[e] = fmaxf(z[e], 0.0f) * fmaxf(z[e], 0.0f);
            break;
        case kActSilu:
#pragma unroll
            for (int e = 0; e < C; ++e) z[e] = z[e] * sigmoid_fast(z[e]);
            break;
        case kActGelu:
#pragma unroll
            for (int e = 0; e < C; ++e) z[e] = gelu_erf(z[e]);
            break;
        case kActGeluTanh:
#pragma unroll
            for (int e = 0; e < C; ++e) z[e] = gelu_tanh(z[e]);
            break;
        default: break;
    }
}

__device__ __forceinline__ float silu_slope(float z) {
    const float p = sigmoid_fast(z);
    return p * __builtin_fmaf(z, 1.0f - p, 1.0f);
}
__device__ __forceinline__ float gelu_erf_slope(float z) {
    // Phi(z) + z phi(z)
    const float g = half_gauss(z);
    const float e = 0.5f * erfc_sqrt2(fabsf(z), g);
    return __builtin_fmaf(z * kInvSqrt2Pi, g, z < 0.0f ? e : 1.0f - e);
}
__device__ __forceinline__ float gelu_tanh_slope(float z) {
    const float zz = fminf(z * z, 1e4f);  // p is 0 or 1 long before; keeps 0 * du finite
    const float p = gelu_tanh_gate(z, zz);
    const float du = kGeluTanhC * __builtin_fmaf(3.0f * kGeluTanhA, zz, 1.0f);
    return __builtin_fmaf(z * p * (1.0f - p), du, p);
}

// g = g * act'(z) for each element (relu's slope at 0 is 0).
template <int C>
__device__ __forceinline__ void times_slope(float (&g)[C], const float (&z)[C], int act) {
    switch (act) {
        case kActRelu:
#pragma unroll
            for (int e = 0; e < C; ++e) g[e] = z[e] > 0.0f ? g[e] : 0.0f;
            break;
        case kActRelu2:
#pragma unroll
            for (int e = 0; e < C; ++e) g[e] = g[e] * (2.0f * fmaxf(z[e], 0.0f));
            break;
        case kActSilu:
#pragma unroll
            for (int e = 0; e < C; ++e) g[e] = g[e] * silu_slope(z[e]);
            break;
        case kActGelu:
#pragma unroll
            for (int e = 0; e < C; ++e) g[e] = g[e] * gelu_erf_slope(z[e]);
            break;
        case kActGeluTanh:
#pragma unroll
            for (int e = 0; e < C; ++e) g[e] = g[e] * gelu_tanh_slope(z[e]);
            break;
        default: break;
    }
}

// Gradients of act(z) u for the gradient g of it: u becomes g act(z) (u's), z
// becomes g u act'(z) (z's). Value and slope share their exponential.
__device__ __forceinline__ void gated_grad(float g, float &z, float &u, float a, float slope) {
    z = g * u * slope;
    u = g * a;
}
template <int C>
__device__ __forceinline__ void gated_grads(const float (&g)[C], float (&z)[C], float (&u)[C], int act) {
    switch (act) {
        case kActRelu:
#pragma unroll
            for (int e = 0; e < C; ++e) gated_grad(g[e], z[e], u[e], fmaxf(z[e], 0.0f), z[e] > 0.0f ? 1.0f : 0.0f);
            break;
        case kActRelu2:
#pragma unroll
            for (int e = 0; e < C; ++e) {
                const float r = fmaxf(z[e], 0.0f);
                gated_grad(g[e], z[e], u[e], r * r, 2.0f * r);
            }
            break;
        case kActSilu:
#pragma unroll
            for (int e = 0; e < C; ++e) {
                const float p = sigmoid_fast(z[e]);
                gated_grad(g[e], z[e], u[e], z[e] * p, p * __builtin_fmaf(z[e], 1.0f - p, 1.0f));
            }
            break;
        case kActGelu:
#pragma unroll
            for (int e = 0; e < C; ++e) {
                const float x = fabsf(z[e]), n = half_gauss(z[e]), c = 0.5f * erfc_sqrt2(x, n);
                gated_grad(g[e], z[e], u[e], __builtin_fmaf(-x, c, fmaxf(z[e], 0.0f)),
                           __builtin_fmaf(z[e] * kInvSqrt2Pi, n, z[e] < 0.0f ? c : 1.0f - c));
            }
            break;
        case kActGeluTanh:
#pragma unroll
            for (int e = 0; e < C; ++e) {
                const float zz = fminf(z[e] * z[e], 1e4f);  // as in gelu_tanh_slope
                const float p = gelu_tanh_gate(z[e], zz);
                const float du = kGeluTanhC * __builtin_fmaf(3.0f * kGeluTanhA, zz, 1.0f);
                gated_grad(g[e], z[e], u[e], z[e] * p, __builtin_fmaf(z[e] * p * (1.0f - p), du, p));
            }
            break;
        default:
#pragma unroll
            for (int e = 0; e < C; ++e) gated_grad(g[e], z[e], u[e], z[e], 1.0f);
            break;
    }
}

#endif

}  // namespace bl
