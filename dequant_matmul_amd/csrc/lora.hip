// Low-rank adapters of many requests beside one projection:
//   y[m] = base[m] + scale[i] * B_i (A_i x[m]),  i = index[m].
// Two launches: the products t = A_i x in fp32 into the workspace, then their
// expansion added to base.
#include "fqm_layer.h"

namespace fqm {
namespace {

__device__ __forceinline__ int rank_of(const fqm_adapters& a, int i) {
    return a.ranks ? max(0, min(a.ranks[i], a.rank)) : a.rank;
}

// One wave per (row m, rank entry r): t[m][r] = A_i[r] . x[m].
__global__ __launch_bounds__(256) void lora_shrink(const fqm_adapters a, const uint16_t* __restrict__ x,
                                                   const int32_t* __restrict__ index, float* __restrict__ t, int64_t M) {
    const int64_t job = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int64_t m = job / a.rank;
    const int r = (int)(job - m * a.rank), lane = threadIdx.x & 63;
    if (m >= M) return;
    const int i = index[m];
    if ((unsigned)i >= (unsigned)a.count || r >= rank_of(a, i)) return;
    const uint16_t* A = a.A + ((int64_t)i * a.rank + r) * a.ld_A;
    const uint16_t* X = x + m * a.cols;
    float acc = 0.f;
    for (int64_t k = 8 * lane; k < a.cols; k += 512) {
        const uint4 av = *reinterpret_cast<const uint4*>(A + k), xv = *reinterpret_cast<const uint4*>(X + k);
        const uint32_t aw[4] = {av.x, av.y, av.z, av.w}, xw[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            acc = fmaf(bf16lo(aw[e]), bf16lo(xw[e]), acc);
            acc = fmaf(bf16hi(aw[e]), bf16hi(xw[e]), acc);
        }
    }
    acc = wave_sum(acc);
    if (lane == 0) t[m * a.rank + r] = acc;
}

// One thread per output (m, n).
__global__ __launch_bounds__(256) void lora_expand(const fqm_adapters a, const int32_t* __restrict__ index,
                                                   const float* __restrict__ t, const void* base, int base_f32,
                                                   void* y, int y_f32) {
    const int64_t m = blockIdx.y, n = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (n >= a.rows) return;
    const int i = index[m];
    float acc = 0.f;
    if ((unsigned)i < (unsigned)a.count) {
        const uint16_t* B = a.B + ((int64_t)i * a.rows + n) * a.ld_B;
        const int rank = rank_of(a, i);
        for (int r = 0; r < rank; ++r) acc = fmaf(bf16_to_f32(B[r]), t[m * a.rank + r], acc);
        if (a.scale) acc *= a.scale[i];
    }
    const int64_t at = m * a.rows + n;
    if (base)
        acc += base_f32 ? static_cast<const float*>(base)[at] : bf16_to_f32(static_cast<const uint16_t*>(base)[at]);
    if (y_f32) static_cast<float*>(y)[at] = acc;
    else static_cast<uint16_t*>(y)[at] = __builtin_bit_cast(uint16_t, (__bf16)acc);
}

}  // namespace

size_t lora_workspace(const fqm_adapters& a, int64_t M) { return (size_t)M * a.rank * sizeof(float); }

hipError_t launch_lora(const fqm_adapters& a, const uint16_t* x, const int32_t* index, const void* base,
                       int base_f32, void* y, int y_f32, int64_t M, float* ws, hipStream_t s) {
    const int64_t jobs = (M * a.rank + 3) / 4;
    if (jobs > 0x7fffffff || M > 65535) return hipErrorInvalidValue;
    hipLaunchKernelGGL(lora_shrink, dim3((unsigned)jobs), dim3(256), 0, s, a, x, index, ws, M);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(lora_expand, dim3((unsigned)((a.rows + 255) / 256), (unsigned)M), dim3(256), 0, s, a, index, ws,
                       base, base_f32, y, y_f32);
    return hipGetLastError();
}

}  // namespace fqm
