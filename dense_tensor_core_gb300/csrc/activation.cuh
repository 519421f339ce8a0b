// activation.cuh -- the activation functions of the feed-forward operators and their derivatives,
// in fp32, on short register arrays.
//
//   relu(z) = max(z, 0)                      gelu(z) = z Phi(z), Phi the normal distribution
//   silu(z) = z s(z), s(z) = 1 / (1 + e^-z)  gelu_tanh(z) = 0.5 z (1 + tanh u)
//                                            u = sqrt(2/pi) (z + 0.044715 z^3)
// 0.5 (1 + tanh u) = s(2u), so silu and gelu_tanh are z times a logistic function of z: one
// exponential and one reciprocal. The exponential and the division are the fast forms: a few ulp, and
// an ulp per unit of the exponent's argument, at most 2^-15 of the result over the range of fp32, which
// is far below half an ulp of the 16-bit outputs.
//
// gelu needs Phi(z) to that relative error too, down its negative tail, where 0.5 + 0.5 erf(z / sqrt 2)
// cancels (4 % off at z = -5). Phi(-a) = e^(-a^2/2) m(a) for a >= 0 with m(a) = e^(a^2/2) Phi(-a), the
// normal distribution's Mills ratio times its density at 0: smooth, 1/2 at 0 and like 1 / (a sqrt(2 pi))
// far out. With t = 1 / (1 + 0.3 a), m = t P(t), P a polynomial of degree 7 fitted to the least largest
// relative error over a in [0, 14] (weighted least squares at Chebyshev nodes): 1.5e-7, 5e-7 as computed
// in fp32. Phi(z) for z >= 0 is 1 - Phi(-z). The derivative Phi(z) + z phi(z) has the same exponential.
// Measured with GELU, bias, residual and the kept sum, us, this and erfcf: 4096 x 4096 x 8192 183 and
// 187; 4096 x 4096 x 1024, where the epilogue shows, 58 and 83.
//
// The gated forms take a pair (g, u): swiglu = silu(g) u, geglu = gelu(g) u.
#pragma once

#include <stdint.h>

namespace dtc {

// Codes of gemm_activation in include/dtc_ffn.h.
constexpr int kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4,
              kActSwiglu = 5, kActGeglu = 6;
__host__ __device__ constexpr bool act_gated(int a) { return a >= kActSwiglu; }
// The function a gated form applies to its gate.
__host__ __device__ constexpr int act_of_gate(int a) {
    return a == kActSwiglu ? kActSilu : a == kActGeglu ? kActGelu : a;
}

constexpr float kGeluC1 = 0.7978845608028654f;      // sqrt(2/pi)
constexpr float kGeluC3 = 0.044715f;
constexpr float kRsqrt2Pi = 0.3989422804014327f;    // 1/sqrt(2 pi)
// P's coefficients, the highest power first.
__device__ __forceinline__ constexpr float mills(int i) {
    constexpr float c[8] = {0.03567477688193321f, -0.15720310807228088f, 0.20635353028774261f, -0.05368367210030556f,
                            0.12856164574623108f, 0.09991348534822464f,  0.12075395882129669f, 0.11962930113077164f};
    return c[i];
}

// 1 / (1 + e^-v). For v below about -87.3 the fast division gives 0 (its divisor is above 2^126), the
// limit of the exact value: an absolute error below 2^-125.
__device__ __forceinline__ float logistic(float v) { return __fdividef(1.0f, 1.0f + __expf(-v)); }

// Phi(z), the normal distribution function; e receives e^(-z^2/2).
__device__ __forceinline__ float normal_cdf(float z, float& e) {
    const float a = fabsf(z);
    const float t = __fdividef(1.0f, fmaf(0.3f, a, 1.0f));
    e = __expf(-0.5f * z * z);
    float p = mills(0);
#pragma unroll
    for (int i = 1; i < 8; ++i) p = fmaf(p, t, mills(i));
    const float h = p * t * e;
    return z < 0.0f ? h : 1.0f - h;
}

// z * s for s = logistic(v) in [0, 1]: 0 at z = -infinity, the limit, instead of -inf * 0.
__device__ __forceinline__ float times_logistic(float z, float s) { return s == 0.0f ? 0.0f : z * s; }

__device__ __forceinline__ float gelu_tanh_arg(float z) {
    return 2.0f * kGeluC1 * z * fmaf(kGeluC3 * z, z, 1.0f);
}

// f(z) of an ungated code, for all entries of an array; the switch stands outside the loop.
template <int N>
__device__ __forceinline__ void act_forward(float (&z)[N], int act) {
    switch (act) {
        case kActRelu:
#pragma unroll
            for (int i = 0; i < N; ++i) z[i] = z[i] < 0.0f ? 0.0f : z[i];
            break;
        case kActGelu:
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float e;
                const float p = normal_cdf(z[i], e);
                z[i] = times_logistic(z[i], p);
            }
            break;
        case kActGeluTanh:
#pragma unroll
            for (int i = 0; i < N; ++i) z[i] = times_logistic(z[i], logistic(gelu_tanh_arg(z[i])));
            break;
        case kActSilu:
#pragma unroll
            for (int i = 0; i < N; ++i) z[i] = times_logistic(z[i], logistic(z[i]));
            break;
        default: break;
    }
}

// f(z) and f'(z) of an ungated code: z becomes f(z), d receives f'(z).
template <int N>
__device__ __forceinline__ void act_both(float (&z)[N], float (&d)[N], int act) {
    switch (act) {
        case kActRelu:
#pragma unroll
            for (int i = 0; i < N; ++i) {
                d[i] = z[i] > 0.0f ? 1.0f : 0.0f;
                z[i] = z[i] < 0.0f ? 0.0f : z[i];
            }
            break;
        case kActGelu:
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float e;
                const float p = normal_cdf(z[i], e);
                const float q = kRsqrt2Pi * e;
                d[i] = q == 0.0f ? p : fmaf(z[i], q, p);
                z[i] = times_logistic(z[i], p);
            }
            break;
        case kActGeluTanh:
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float s = logistic(gelu_tanh_arg(z[i]));
                const float t = s * (1.0f - s);
                const float du = 2.0f * kGeluC1 * fmaf(3.0f * kGeluC3 * z[i], z[i], 1.0f);
                d[i] = t == 0.0f ? s : fmaf(z[i] * du, t, s);
                z[i] = times_logistic(z[i], s);
            }
            break;
        case kActSilu:
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float s = logistic(z[i]);
                const float t = s * (1.0f - s);
                d[i] = t == 0.0f ? s : fmaf(z[i], t, s);
                z[i] = times_logistic(z[i], s);
            }
            break;
        default:
#pragma unroll
            for (int i = 0; i < N; ++i) d[i] = 1.0f;
            break;
    }
}

}  // namespace dtc
