// The row functions of the decode steps (dense cache and paged cache): the
// normaliser value of a score, the constants and the integer power of the
// re-weighting, in log2 units (z = log2(e) x).
#pragma once

#include "lssar_internal.cuh"
#include "tc_ptx.cuh"

namespace lssar {

// log2(1 + 2^z) without overflow for any z, to 2^-19 of its value also where that is
// small: a row whose keys all point away from the query has z down to -116, and
// lg2(1 + u), u = 2^-|z|, is off by 2^-22 and 0 from z = -24 on.  log2(1 + u) = u P(u), P of
// degree 6 with the least largest relative error on [0, 1] (exchange algorithm): 1.3e-6,
// 1.4e-6 with its steps in fp32.  One special function and seven FMAs, two scores at a
// time: 2 sequences of 128K tokens, LSSAR, take 63.8 us; with lg2 and its series below
// u = 2^-6 they took 67.8.
__device__ __forceinline__ float2 softplus2(float2 z) {
    const float2 u = make_float2(ptx::ex2(-fabsf(z.x)), ptx::ex2(-fabsf(z.y)));
    const auto both = [](float c) { return make_float2(c, c); };
    float2 r = __ffma2_rn(both(0.020401185378432274f), u, both(-0.09579754620790482f));
    r = __ffma2_rn(r, u, both(0.2152845412492752f));
    r = __ffma2_rn(r, u, both(-0.339089035987854f));
    r = __ffma2_rn(r, u, both(0.4776683747768402f));
    r = __ffma2_rn(r, u, both(-0.7211594581604004f));
    r = __ffma2_rn(r, u, both(1.4426932334899902f));
    return __ffma2_rn(r, u, make_float2(fmaxf(z.x, 0.f), fmaxf(z.y, 0.f)));
}

__device__ __forceinline__ float sigmoid2(float z) {   // 1 / (1 + 2^-z)
    return ptx::rcp(1.f + ptx::ex2(-z));
}

// The normaliser values of two scores (softmax modes: relative to the max m).
__device__ __forceinline__ float2 phi(int mode, float2 z, float m) {
    if (mode == kSoftmax || mode == kSoftmaxRw) return make_float2(ptx::ex2(z.x - m), ptx::ex2(z.y - m));
    if (mode == kSigmoidRw) return make_float2(sigmoid2(z.x), sigmoid2(z.y));
    return softplus2(z);
}
__device__ __forceinline__ float phi(int mode, float z, float m) { return phi(mode, make_float2(z, z), m).x; }

// What makes re-weighted weights of a row's scores: x, the maximum m (softmax) or
// 2^-min(m, 0), which brings phi, down to 2^-116, to about 1; theta, the offset; kappa,
// 1 / (the largest difference from it); beta, 1 for a uniform row, whose kappa is 0.
struct RowConstants {
    float x, kappa, beta, theta;
};

// The row constants from the row's maximum and normaliser sum.  (An error in kappa's
// last bits scales all of the row's weights alike.)  A row is uniform where the largest
// difference is within 1e-5 of the maximum, a few times what the evaluation of phi and
// of its sum leaves of nearly equal ones; the band is relative, as those errors are.
__device__ __forceinline__ RowConstants row_constants(int mode, int n, float2 st) {
    const bool raw = mode == kSoftmaxRw;
    const float m = st.x, lift = raw ? 1.f : ptx::ex2(-fminf(m, 0.f));
    const float theta = n <= 3 ? 0.f : st.y * lift / (float)n;
    const float top = phi(mode, m, m) * lift, den = top - theta;
    RowConstants rc = {raw ? m : lift, 0.f, 1.f, theta};
    if (den > 1e-5f * top) {
        rc.kappa = ptx::rcp(den);
        rc.beta = 0.f;
    }
    if (isnan(st.y)) rc.kappa = NAN;
    return rc;
}

// Two scores' re-weighted weights before the power: at most 1 but for kappa's rounding
// (the difference is formed before it is scaled, so that its rounding is its own).
__device__ __forceinline__ float2 above_offset(int mode, float2 z, RowConstants rc) {
    const float2 f = phi(mode, z, rc.x), t = make_float2(-rc.theta, -rc.theta);
    float2 y = mode == kSoftmaxRw ? __fadd2_rn(f, t) : __ffma2_rn(f, make_float2(rc.x, rc.x), t);
    y = __ffma2_rn(y, make_float2(rc.kappa, rc.kappa), make_float2(rc.beta, rc.beta));
    return make_float2(fmaxf(y.x, 0.f), fmaxf(y.y, 0.f));
}

__device__ __forceinline__ float2 powi(float2 x, int p) {
    float2 r = make_float2(1.f, 1.f);
    while (p) {
        if (p & 1) r = __fmul2_rn(r, x);
        x = __fmul2_rn(x, x);
        p >>= 1;
    }
    return r;
}

}  // namespace lssar
