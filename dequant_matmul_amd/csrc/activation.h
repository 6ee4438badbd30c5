// The activations of include/fqm.h (enum fqm_act), in fp32.
#pragma once

#include "fqm_internal.h"

namespace fqm {
namespace {

// exp(x) to 2 ulp where it is a normal number, 0 below those: x log2(e) in two parts, the
// hardware's exp2 of the first.  x is held to where exp leaves fp32's range on either side, so that an
// infinite x makes no NaN (a NaN becomes some number: callers multiply by what it came from).
__device__ __forceinline__ float exp_fast(float x) {
    x = __builtin_amdgcn_fmed3f(x, -104.f, 90.f);
    const float t = x * 1.44269504f;                                 // log2(e) rounded to fp32;
    const float lo = fmaf(x, 1.44269504f, -t) + x * 1.92596299e-8f;  // t's rounding and the rest of log2(e)
    return __builtin_amdgcn_exp2f(t) * fmaf(0.693147181f, lo, 1.f);
}
// 1 / (1 + exp(-x)) to 4 ulp
__device__ __forceinline__ float logistic(float x) { return __builtin_amdgcn_rcpf(1.f + exp_fast(-x)); }

__device__ __forceinline__ float activate_one(int act, float v) {
    switch (act) {
        case FQM_ACT_RELU: return v < 0.f ? 0.f : v;  // a NaN stays one
        case FQM_ACT_SILU: return v * logistic(v);
        // erfc keeps the digits that 1 + erf loses where Phi is small
        case FQM_ACT_GELU: return 0.5f * v * erfcf(v * -0.70710678118654752f);
        // (1 + tanh z) / 2 = 1 / (1 + exp(-2 z))
        case FQM_ACT_GELU_TANH: return v * logistic(1.5957691216057308f * (v + 0.044715f * v * v * v));
        case FQM_ACT_SIGMOID: return v == v ? logistic(v) : v;
        case FQM_ACT_TANH: return tanhf(v);
        default: return v;
    }
}
template <int ACT, int V>
__device__ __forceinline__ void activate_as(float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = activate_one(ACT, v[i]);
}
// V values by one branch: what runs of it is short and lies together.
template <int V>
__device__ __forceinline__ void activate(int act, float (&v)[V]) {
    if (act == FQM_ACT_NONE) return;
    if (act == FQM_ACT_SILU) activate_as<FQM_ACT_SILU>(v);
    else if (act == FQM_ACT_RELU) activate_as<FQM_ACT_RELU>(v);
    else if (act == FQM_ACT_GELU) activate_as<FQM_ACT_GELU>(v);
    else if (act == FQM_ACT_GELU_TANH) activate_as<FQM_ACT_GELU_TANH>(v);
    else if (act == FQM_ACT_SIGMOID) activate_as<FQM_ACT_SIGMOID>(v);
    else if (act == FQM_ACT_TANH) activate_as<FQM_ACT_TANH>(v);
}

}  // namespace
}  // namespace fqm
