// Activations of the dense products, and their derivatives, in 32-bit floats.
//
//   silu       z s,  s = 1 / (1 + exp(-z));        slope s (1 + z (1 - s))
//   gelu       z Phi(z);                           slope Phi(z) + z phi(z)
//   gelu_tanh  z s(c (z + k z^3)), c = 2 sqrt(2/pi), k = 0.044715, since
//              1 + tanh(t/2) = 2 s(t);             slope s + z s (1 - s) c (1 + 3 k z^2)
//
// phi(z) = exp(-z^2/2) / sqrt(2 pi) and Phi its integral.  For a = |z|, Phi(-a) =
// exp(-a^2/2) R(a) with R smooth and of one sign, so a polynomial in t = 1 / (1 +
// c a) without constant term gives it with a small error relative to itself, also
// far out where 1 + erf has cancelled: 8 coefficients by weighted least squares
// (iterated towards the least largest error) over 0 <= a <= 14, error 2.1e-7.  One
// exponential and one reciprocal serve value and slope.
//
// Errors of the value relative to it, measured: the exponential's argument is rounded,
// so they grow with it, gelu 8.0e-7 (|z| < 4), 7.5e-6 (13), gelu_tanh 1.5e-6 (4),
// 6.8e-6 (8), 1.3e-5 (10), silu 3.1e-7 (4), 3.6e-6 (60).  Further out on
// the negative side the exponential or the sigmoid is below the smallest float and
// the value 0 (it is 5e-39, 1.2e-37 and 1.0e-36 there).  Slopes are within 2e-6.
#pragma once

#include "ffn_internal.h"

namespace gemm_rs {
namespace ffn {

enum Act { kActNone, kActRelu, kActGelu, kActGeluTanh, kActSilu, kActs };

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float rcp_fast(float x) { return __builtin_amdgcn_rcpf(x); }
// 1 / (1 + exp(-x)); 0 and 1 far out
__device__ __forceinline__ float sigmoid(float x) { return rcp_fast(1.0f + exp2_fast(-1.44269504f * x)); }

// Phi(z) and exp(-z^2/2)
__device__ __forceinline__ float normal_cdf(float z, float *e) {
    const float a = fabsf(z);
    *e = exp2_fast(-0.72134752f * (a * a));
    const float t = rcp_fast(fmaf(0.3125f, a, 1.0f));
    float r = 0.03526223823428154f;
    r = fmaf(r, t, -0.13551603257656097f);
    r = fmaf(r, t, 0.13984039425849915f);
    r = fmaf(r, t, -0.004023127723485231f);
    r = fmaf(r, t, 0.10512357205152512f);
    r = fmaf(r, t, 0.10976135730743408f);
    r = fmaf(r, t, 0.12488832324743271f);
    r = fmaf(r, t, 0.12466337531805038f);
    const float below = *e * (r * t);
    return z < 0 ? below : 1.0f - below;
}

constexpr float kTanhC = 1.5957691216057308f, kTanhK = 0.044715f;
// z^2, kept finite: far out the sigmoid is 0 or 1 and it is multiplied by 0
__device__ __forceinline__ float square_capped(float z) { return fminf(z * z, 1e30f); }
__device__ __forceinline__ float gelu_tanh_gate(float z) {
    return sigmoid(kTanhC * z * fmaf(kTanhK, square_capped(z), 1.0f));
}

template <int N>
__device__ __forceinline__ void activate(int act, float (&z)[N]) {
    switch (act) {
    case kActRelu:
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] = z[i] < 0 ? 0.0f : z[i];      // (NaN stays)
        break;
    case kActGelu:
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float e;
            z[i] *= normal_cdf(z[i], &e);
        }
        break;
    case kActGeluTanh:
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] *= gelu_tanh_gate(z[i]);
        break;
    case kActSilu:
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] *= sigmoid(z[i]);
        break;
    default: break;
    }
}

// value = act(z), slope = act'(z); relu's slope at 0 is 0
template <int N>
__device__ __forceinline__ void activate_both(int act, const float (&z)[N], float (&value)[N], float (&slope)[N]) {
    switch (act) {
    case kActRelu:
#pragma unroll
        for (int i = 0; i < N; ++i) {
            value[i] = z[i] < 0 ? 0.0f : z[i];
            slope[i] = z[i] > 0 ? 1.0f : z[i] <= 0 ? 0.0f : z[i];
        }
        break;
    case kActGelu:
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float e;
            const float p = normal_cdf(z[i], &e);
            value[i] = z[i] * p;
            slope[i] = fmaf(z[i], 0.3989422804f * e, p);
        }
        break;
    case kActGeluTanh:
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float s = gelu_tanh_gate(z[i]);
            value[i] = z[i] * s;
            slope[i] = fmaf(value[i] * (1.0f - s), kTanhC * fmaf(3 * kTanhK, square_capped(z[i]), 1.0f), s);
        }
        break;
    case kActSilu:
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float s = sigmoid(z[i]);
            value[i] = z[i] * s;
            slope[i] = s * fmaf(z[i], 1.0f - s, 1.0f);
        }
        break;
    default:
#pragma unroll
        for (int i = 0; i < N; ++i) {
            value[i] = z[i];
            slope[i] = 1.0f;
        }
    }
}

}  // namespace ffn
}  // namespace gemm_rs
