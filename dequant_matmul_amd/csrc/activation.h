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
// 1 / (1 + exp(-x)) to 4 ulp, 0 where that is below 2^-126 (x < -87.3: the reciprocal gives no denormal numbers).
__device__ __forceinline__ float logistic(float x) { return __builtin_amdgcn_rcpf(1.f + exp_fast(-x)); }

// v / (1 + exp(-z)) to 9 * 2^-24 of it, below 2^-126 to a step of 2^-149.  LOW: z may be below -64 (|v| >= 1 there).  Then the
// sum is exp(-z) to fp32, and v exp(z) is formed as v exp(z + 64) exp(-64): nothing leaves fp32's range ahead of the result,
// and z + 64 is exact wherever that is not 0.  Other values are the same with and without LOW, to the bit (so no addition
// behind is fused with the products).
template <bool LOW>
__device__ __forceinline__ float times_logistic(float v, float z) {
#pragma clang fp contract(off)
    const bool low = LOW && z < -64.f;
    const float e = exp_fast(low ? z + 64.f : -z);
    const float y = v * (low ? e : __builtin_amdgcn_rcpf(1.f + e));
    return low ? y * 1.60381089e-28f : y;
}

template <int ACT, int V>
__device__ __forceinline__ void activate_as(float (&v)[V]) {
    if constexpr (ACT == FQM_ACT_SILU || ACT == FQM_ACT_GELU_TANH || ACT == FQM_ACT_SIGMOID) {
        float z[V], least = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            // (1 + tanh x) / 2 = 1 / (1 + exp(-2 x))
            z[i] = ACT == FQM_ACT_GELU_TANH ? 1.5957691216057308f * (v[i] + 0.044715f * v[i] * v[i] * v[i]) : v[i];
            least = fminf(least, z[i]);
            if (ACT == FQM_ACT_SIGMOID) v[i] = v[i] == v[i] ? 1.f : v[i];
        }
        // One uniform branch for the wave's values: a test for each costs a block of 8192 x 5120 with a SiLU gate a value
        // 8 % (97 -> 105 us) and the gated product of 2048 rows 1.3 % (360 -> 365), this way they cost 0.7 and 0.3 %.
        if (__builtin_expect(__ballot(least < -64.f) != 0, 0)) {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = times_logistic<true>(v[i], z[i]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = times_logistic<false>(v[i], z[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (ACT == FQM_ACT_RELU) v[i] = v[i] < 0.f ? 0.f : v[i];  // a NaN stays one
            // erfc keeps the digits that 1 + erf loses where Phi is small
            if (ACT == FQM_ACT_GELU) v[i] = 0.5f * v[i] * erfcf(v[i] * -0.70710678118654752f);
            if (ACT == FQM_ACT_TANH) v[i] = tanhf(v[i]);
        }
    }
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
