// The activations of include/fqm.h (enum fqm_act), in fp32.
#pragma once

#include "fqm_internal.h"

namespace fqm {
namespace {

__device__ __forceinline__ float activate(int act, float v) {
    switch (act) {
        case FQM_ACT_RELU: return v < 0.f ? 0.f : v;  // a NaN stays one
        case FQM_ACT_SILU: return v / (1.f + expf(-v));
        // erfc keeps the digits that 1 + erf loses where Phi is small
        case FQM_ACT_GELU: return 0.5f * v * erfcf(v * -0.70710678118654752f);
        // (1 + tanh z) / 2 = 1 / (1 + exp(-2 z))
        case FQM_ACT_GELU_TANH: return v / (1.f + expf(-1.5957691216057308f * (v + 0.044715f * v * v * v)));
        case FQM_ACT_SIGMOID: return 1.f / (1.f + expf(-v));
        case FQM_ACT_TANH: return tanhf(v);
        default: return v;
    }
}

}  // namespace
}  // namespace fqm
