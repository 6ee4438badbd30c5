// Internal declarations of the operators around the products: the residual
// norm, the low-rank adapters, the products grouped by expert and their routing,
// the product with an epilogue, the norms around a block.
#pragma once

#include "fqm_internal.h"

namespace fqm {

// Workgroup barrier for LDS alone: LDS operations are complete, global loads
// and stores of the wave stay in flight (__syncthreads waits for them too).
__device__ __forceinline__ void lds_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0) only
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Between LDS writes of a wave's lanes and reads of the same places by its other
// lanes: a wave's LDS operations are in order, this makes the compiler keep them
// so (no instruction).
__device__ __forceinline__ void wave_lds_order() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

hipError_t launch_add_rms_norm(const fqm_norm& a, hipStream_t s);

size_t lora_workspace(const fqm_adapters& a, int64_t M);
hipError_t launch_lora(const fqm_adapters& a, const uint16_t* x, const int32_t* index, const void* base,
                       int base_f32, void* y, int y_f32, int64_t M, float* ws, hipStream_t s);

size_t grouped_workspace(const fqm_weights& w, const fqm_groups& g);
hipError_t launch_grouped(const fqm_weights& w, const fqm_groups& g, void* ws, hipStream_t s);

size_t linear_workspace(const fqm_weights& w, const fqm_epilogue& a);
hipError_t launch_linear(const fqm_weights& w, const fqm_epilogue& a, void* ws, hipStream_t s);

size_t route_workspace(const fqm_routing& a);
hipError_t launch_route(const fqm_routing& a, void* ws, hipStream_t s);

hipError_t launch_block_norm(const fqm_block& a, hipStream_t s);

}  // namespace fqm
