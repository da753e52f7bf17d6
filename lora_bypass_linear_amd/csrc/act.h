// act.h -- the gated block's activations and their derivatives in fp32, free of
// branches: a tile's end evaluates them on up to 64 outputs a lane.
#pragma once

#include "lyc_device.h"
#include "pair.h"

namespace lyc {

// exp(t) 2^s, t below 88 + s log(2), to about two ulps: the product t log2(e) in
// two pieces, so that the exponent's own rounding (2^-24 of up to 128) does not
// reach the result.  (hi + s has no rounding: s is 0, or 64 against a hi of 112 to
// 192 of the other sign)
__device__ __forceinline__ float exp_f32(float t, float s = 0.f) {
    constexpr float L = 1.44269502f, LL = 1.92596303e-8f;   // log2(e) = L + LL
    const float hi = t * L;
    const float lo = __builtin_fmaf(t, LL, __builtin_fmaf(t, L, -hi));
    const float e = __builtin_amdgcn_exp2f(hi + s);
    return __builtin_fmaf(e, lo * 0.693147182f, e);
}

// 1 / d to an ulp, d finite and normal
__device__ __forceinline__ float rcp_f32(float d) {
    const float r = __builtin_amdgcn_rcpf(d);
    return __builtin_fmaf(__builtin_fmaf(-d, r, 1.f), r, r);
}

//   silu       g p(g)                                           slope p + g p (1 - p)
//   gelu_tanh  g p(u), u = 2 sqrt(2/pi) (g + 0.044715 g^3)      slope p + g p (1 - p) u'
// with p(u) = 1 / (1 + exp(-u)) (1/2 (1 + tanh z) is p(2 z)): u = g (b g^2 + a).
// exp(-u) leaves the fp32 range below u = -87, where g p is still a normal value:
// there it is taken 2^-64 fold (1 + e is e, so r is p 2^64) and the factor put
// back at the end.  Below -112 both results are under fp32's smallest value.  u is
// taken of g within +-1e6, where p has long been 0 or 1, so that no infinity
// meets another; a NaN passes through the factor g.
template <bool GRAD>
__device__ __forceinline__ float act_logistic(float a, float b, float g, float* slope) {
    const float c = __builtin_amdgcn_fmed3f(g, -1e6f, 1e6f), c2 = c * c;
    const float u = c * __builtin_fmaf(b, c2, a);
    const bool far = u < -87.f;
    const float back = u < -112.f ? 0.f : far ? 0x1p-64f : 1.f;
    const float e = exp_f32(__builtin_fminf(-u, 112.f), far ? -64.f : 0.f);
    const float r = rcp_f32(1.f + e);
    if constexpr (GRAD) *slope = __builtin_fmaf(g * r * (e * r), __builtin_fmaf(3.f * b, c2, a), r) * back;
    return g * r * back;
}

// The same for 16-bit results: exp2 and the reciprocal as the hardware gives them
// (an ulp each), the exponent rounded once.  Off by 2^-23 |u| of the result
// where that is near 0 (negative u) and by a few 2^-24 elsewhere, a 2^-12th of
// bf16's and a 2^-9th of fp16's rounding at |u| = 8.  exp2 overflows to infinity,
// whose reciprocal is 0; only g^2 is kept finite, for b = 0.
__device__ __forceinline__ float act_logistic16(float a, float b, float g) {
    const float u = g * __builtin_fmaf(b, __builtin_fminf(g * g, 1e30f), a);
    return g * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(u * -1.44269502f));
}

// Value and slope for 16-bit gradients, with the error of each in units of 2^-24
// relative (fp32 ulps at most), n_slope relative to mass = |t| + p, slope = t + p:
// the exponent's rounding 1.2 |u| (the tanh form's u 3 |u| more), which counts
// q-fold in p and p-fold in q = 1 - p; exp2 2, the sum 1, the reciprocal 2, so p 5
// and q 6; g p one more, t 16 with its products and u'.  Below u = -87, where p
// nears fp32's smallest normal value, both bounds are infinite (and e is kept
// finite, or q = e r would be a product of infinity and 0).
__device__ __forceinline__ float act_logistic16_grad(float a, float b, float g, float* slope, float* mass,
                                                     float* n_act, float* n_slope) {
    const float g2 = __builtin_fminf(g * g, 1e30f), u = g * __builtin_fmaf(b, g2, a);
    const float e = __builtin_fminf(__builtin_amdgcn_exp2f(u * -1.44269502f), 3e38f);
    const float p = __builtin_amdgcn_rcpf(1.f + e), v = g * p;
    const float t = v * (e * p) * __builtin_fmaf(3.f * b, g2, a);
    const float nu = u < -87.f ? __builtin_inff() : (b != 0.f ? 4.25f : 1.25f) * __builtin_fabsf(u);
    *slope = t + p;
    *mass = __builtin_fabsf(t) + p;
    *n_act = nu + 6.f;
    *n_slope = nu + 16.f;
    return v;
}

//   gelu   g Phi(g)      slope Phi(g) + g exp(-g^2 / 2) / sqrt(2 pi)
// Phi(-|g|) = 1/2 exp(-z^2) erfcx(z), z = |g| / sqrt(2), keeps its relative
// accuracy where 1 + erf cancels.  (1 + 2 z) erfcx(z) is smooth in s = (z - 5/2) /
// (z + 5/2): a polynomial of degree 9 fitted at Chebyshev nodes of z up to 13.5
// (beyond, exp(-z^2) is 0) is within 3e-8 of it, 4e-7 with fp32's roundings.
// exp(-z^2) takes z^2 = g^2 / 2 in two pieces.  FAR: the slope keeps its accuracy
// where exp(-z^2) is below fp32's smallest normal value (it is taken 2^64 fold).
template <bool GRAD, bool FAR = false>
__device__ __forceinline__ float act_gelu(float g, float* slope, float* mass) {
    const float c = __builtin_amdgcn_fmed3f(g, -1e6f, 1e6f), h = 0.5f * c;
    const float hi = h * c, lo = __builtin_fmaf(h, c, -hi);
    const bool far = FAR && hi > 80.f;
    const float back = far ? 0x1p-64f : 1.f;
    float e = exp_f32(-hi, far ? 64.f : 0.f);
    e = __builtin_fmaf(-e, lo, e);
    const float z = __builtin_fabsf(c) * 0.707106769f;
    const float d = __builtin_fmaf(2.f, z, 1.f), k = z + 2.5f;
    const float r = rcp_f32(k * d);
    const float s = (z - 2.5f) * d * r;
    float y = 0.000472367508f;
    y = __builtin_fmaf(y, s, 0.000361906888f);
    y = __builtin_fmaf(y, s, -0.00428514602f);
    y = __builtin_fmaf(y, s, 0.00100247574f);
    y = __builtin_fmaf(y, s, 0.0327323899f);
    y = __builtin_fmaf(y, s, -0.102982864f);
    y = __builtin_fmaf(y, s, 0.157633707f);
    y = __builtin_fmaf(y, s, -0.0990233123f);
    y = __builtin_fmaf(y, s, -0.122356921f);
    y = __builtin_fmaf(y, s, 1.26483822f);
    const float tail = 0.5f * e * (y * k * r) * back;
    const float cdf = g < 0.f ? tail : 1.f - tail;
    if constexpr (GRAD) {
        const float t = g * 0.398942292f * e * back;
        *slope = t + cdf;
        *mass = __builtin_fabsf(t) + cdf;   // (both off by less than 16 units of 2^-24)
    }
    return g * cdf;
}

// The same in 64 bits, for the few values that an fp32 one cannot round.  (A NaN
// stays one; at an infinity the value's product with p = 0 is one.)
__device__ __forceinline__ double act_f64(int act, double g, double* slope) {
    if (act == ACT_GELU) {
        const double cdf = 0.5 * erfc(g * -0.70710678118654752);
        *slope = cdf + g * exp(-0.5 * g * g) * 0.39894228040143268;
        return g * cdf;
    }
    const double a = act == ACT_GELU_TANH ? 1.5957691216057308 : 1.0;
    const double b = act == ACT_GELU_TANH ? 0.071354816272600243 : 0.0;
    const double u = g * (a + b * g * g);
    const double e = exp(-__builtin_fabs(u)), r = 1.0 / (1.0 + e), er = e * r;
    const double p = u < 0.0 ? er : r, q = u < 0.0 ? r : er;
    *slope = p + g * p * q * (a + 3.0 * b * g * g);
    return g * p;
}

// the logistic form's coefficients
__device__ __forceinline__ void act_coeffs(int act, float& a, float& b) {
    a = act == ACT_GELU_TANH ? 1.59576917f : 1.f;
    b = act == ACT_GELU_TANH ? 0.0713548139f : 0.f;
}

}  // namespace lyc
