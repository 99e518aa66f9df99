// The row functions of the decode steps (dense cache and paged cache): the
// normaliser value of a score and the integer power of the re-weighting, in
// log2 units (z = log2(e) x).
#pragma once

#include "lssar_internal.cuh"
#include "tc_ptx.cuh"

namespace lssar {

// log2(1 + 2^z) without overflow for any z (MUFU ex2 / lg2, as in the
// prefill kernel)
__device__ __forceinline__ float sp2_any(float z) {
    return fmaxf(z, 0.f) + ptx::lg2(1.f + ptx::ex2(-fabsf(z)));
}

__device__ __forceinline__ float sigmoid2(float z) {   // 1 / (1 + 2^-z)
    return ptx::rcp(1.f + ptx::ex2(-z));
}

// The normaliser value of a score (softmax modes: relative to the max m).
__device__ __forceinline__ float phi(int mode, float z, float m) {
    if (mode == kSoftmax || mode == kSoftmaxRw) return ptx::ex2(z - m);
    if (mode == kSigmoidRw) return sigmoid2(z);
    return sp2_any(z);
}

__device__ __forceinline__ float powi(float x, int p) {
    float r = 1.f;
    while (p) {
        if (p & 1) r *= x;
        x *= x;
        p >>= 1;
    }
    return r;
}

}  // namespace lssar
