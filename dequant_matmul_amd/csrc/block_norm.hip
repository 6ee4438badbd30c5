// The norms on both sides of a block, with what lies between them:
//   u = sum_t x_t,   v = u * w1 / sqrt(mean(u^2) + eps),
//   h = residual_scale * residual + scale * act(gate) * v,
//   y = h * w2 / sqrt(mean(h^2) + eps),
// w1 and w2 the norms' weights plus an offset; y in bf16, fp32 or 8 bits with
// one scale per row.
//
// A row is read once into registers (chunks of 8 values, chunk c on thread c mod
// NT) and stays there over both reductions, so memory is touched once.
// Sums, statistics and scales are fp32; h is rounded only where total is stored.
#include <algorithm>

#include "activation.h"
#include "fqm_layer.h"
#include "row_values.h"

namespace fqm {
namespace {

constexpr int kMaxThreads = 1024;  // per row
constexpr int kMaxWaves = kMaxThreads / 64;

// One chunk's values of a row of either type, n of them (the others 0).
template <bool F32>
__device__ __forceinline__ void add_chunk(const void* p, int64_t e, int n, float (&h)[kVec]) {
    if (n == kVec) {
        Raw<F32> r;
        r.load(p, e);
        r.add(h);
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (i < n) h[i] += Raw<F32>::one(p, e + i);
    }
}
__device__ __forceinline__ void add_chunk_of(int dtype, const void* p, int64_t e, int n, float (&h)[kVec]) {
    if (dtype == FQM_F32) add_chunk<true>(p, e, n, h);
    else add_chunk<false>(p, e, n, h);
}

// The sum and the maximum of a row's values over its nt threads (nt > 64: over
// the workgroup, s holds a value per wave of each).
__device__ __forceinline__ void row_reduce(int nt, float& sum, float& mx, float (*s)[kMaxWaves]) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1)
        if (nt > o) {  // uniform
            sum += __shfl_xor(sum, o, 64);
            mx = fmaxf(mx, __shfl_xor(mx, o, 64));
        }
    if (nt > 64) {  // uniform over the grid: then one row per workgroup
        const int wave = threadIdx.x >> 6, waves = nt >> 6;
        if ((threadIdx.x & 63) == 0) s[0][wave] = sum, s[1][wave] = mx;
        __syncthreads();
        sum = 0.f, mx = 0.f;
        for (int i = 0; i < waves; ++i) {
            sum += s[0][i];
            mx = fmaxf(mx, s[1][i]);
        }
    }
}

// One row per threadIdx.y; blockDim.x threads per row (16, 32, or a multiple of
// 64: a row's lanes are a part of one wave or whole waves), NV chunks each.
template <int NV, bool XF32, bool RF32>
__global__ __launch_bounds__(kMaxThreads) void block_norm_kernel(const fqm_block a) {
    __shared__ float s_red[2][2][kMaxWaves];
    const int nt = blockDim.x;
    const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = row < a.rows;
    const int cols = (int)a.cols;
    int n[NV], c0[NV];
    float h[NV][kVec];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        c0[v] = kVec * (threadIdx.x + v * nt);
        n[v] = live ? max(0, min(kVec, cols - c0[v])) : 0;
#pragma unroll
        for (int i = 0; i < kVec; ++i) h[v][i] = 0.f;
    }
    for (int t = 0; t < a.terms; ++t)
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (n[v] > 0) add_chunk<XF32>(a.x, row * a.ld_x + t * a.ld_term + c0[v], n[v], h[v]);

    float r = 1.f, mx = 0.f;
    if (a.post) {
        float sq = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < kVec; ++i) sq = fmaf(h[v][i], h[v][i], sq);
        row_reduce(nt, sq, mx, s_red[0]);
        r = 1.f / sqrtf(sq / (float)cols + a.eps);
    }
    r *= a.scale;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        if (n[v] == 0) continue;
        float f[kVec];
        if (a.post) {
#pragma unroll
            for (int i = 0; i < kVec; ++i) f[i] = a.post_weight ? a.weight_offset : 1.f;
            if (a.post_weight) add_chunk_of(a.post_dtype, a.post_weight, c0[v], n[v], f);
#pragma unroll
            for (int i = 0; i < kVec; ++i) h[v][i] *= f[i];
        }
        if (a.gate) {
#pragma unroll
            for (int i = 0; i < kVec; ++i) f[i] = 0.f;
            const int64_t e = row * a.ld_gate;
            if (a.step_gate) add_chunk_of(a.gate_dtype, a.gate, e + c0[v], n[v], f);
            else {
                const float one = a.gate_dtype == FQM_F32 ? Raw<true>::one(a.gate, e) : Raw<false>::one(a.gate, e);
#pragma unroll
                for (int i = 0; i < kVec; ++i) f[i] = one;
            }
            activate<kVec>(a.gate_act, f);
#pragma unroll
            for (int i = 0; i < kVec; ++i) h[v][i] *= f[i];
        }
#pragma unroll
        for (int i = 0; i < kVec; ++i) f[i] = 0.f;
        if (a.residual) add_chunk<RF32>(a.residual, row * a.ld_res + c0[v], n[v], f);
#pragma unroll
        for (int i = 0; i < kVec; ++i) h[v][i] = i < n[v] ? fmaf(h[v][i], r, a.residual ? a.residual_scale * f[i] : 0.f) : 0.f;
        if (a.total) {
            const int64_t e = row * a.ld_total + c0[v];
            if (a.residual ? RF32 : XF32) store_f32(a.total, e, h[v], n[v]);
            else store_bf16(a.total, e, h[v], n[v]);
        }
    }
    if (!a.y) return;  // uniform

    float sq = 0.f;
    float w[NV][kVec];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) w[v][i] = a.weight ? a.weight_offset : 1.f;
        if (a.weight && n[v] > 0) add_chunk_of(a.weight_dtype, a.weight, c0[v], n[v], w[v]);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            sq = fmaf(h[v][i], h[v][i], sq);
            w[v][i] *= h[v][i];  // from here on w holds h * weight
            mx = fmaxf(mx, fabsf(w[v][i]));
            // fmaxf passes a NaN over: an 8-bit row with one (or an infinity) gets a NaN for its scale here
            if (a.y_dtype == FQM_I8) sq = fmaf(w[v][i], 0.f, sq);
        }
    }
    row_reduce(nt, sq, mx, s_red[1]);
    if (!live) return;
    r = 1.f / sqrtf(sq / (float)cols + a.eps);
    const int64_t yr = row * a.ld_y;
    if (a.y_dtype == FQM_I8) {
        // y's row factor r is common: max|y| = r * max|h w|, y / scale = h w * 127 / max|h w|.  A row of zeros has
        // scale 0 with eps = 0 too, where r is infinite; the codes are 0 exactly where the scale cannot be used
        const float scale = sq == 0.f && mx == 0.f ? 0.f : r * mx / 127.f;
        const bool use = scale > 0.f && scale <= 3.4e38f;
        const float k = mx < 1e-30f ? 0x1p100f : 1.f;  // 127 / mx stays finite
        const float f = use ? 127.f / (mx * k) : 0.f;
        if (threadIdx.x == 0) a.y_scale[row] = scale;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            int c[kVec];
#pragma unroll
            for (int i = 0; i < kVec; ++i) c[i] = use ? (int)fminf(127.f, fmaxf(-127.f, rintf(w[v][i] * k * f))) : 0;
            if (n[v] > 0) store_i8(a.y, yr + c0[v], c, n[v]);
        }
    } else {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
#pragma unroll
            for (int i = 0; i < kVec; ++i) w[v][i] *= r;
            if (n[v] > 0) {
                if (a.y_dtype == FQM_F32) store_f32(a.y, yr + c0[v], w[v], n[v]);
                else store_bf16(a.y, yr + c0[v], w[v], n[v]);
            }
        }
    }
}

template <int NV>
hipError_t launch_nv(const fqm_block& a, dim3 grid, dim3 block, hipStream_t s) {
    const bool xf = a.x_dtype == FQM_F32, rf = a.residual ? a.res_dtype == FQM_F32 : xf;
    if (xf && rf) hipLaunchKernelGGL((block_norm_kernel<NV, true, true>), grid, block, 0, s, a);
    else if (xf) hipLaunchKernelGGL((block_norm_kernel<NV, true, false>), grid, block, 0, s, a);
    else if (rf) hipLaunchKernelGGL((block_norm_kernel<NV, false, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((block_norm_kernel<NV, false, false>), grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_block_norm(const fqm_block& a, hipStream_t s) {
    const int chunks = (int)((a.cols + kVec - 1) / kVec);
    const int nt = chunks <= 16 ? 16 : chunks <= 32 ? 32 : std::min(kMaxThreads, (chunks + 63) / 64 * 64);
    const int rpb = nt <= 64 ? 256 / nt : 1;
    const int64_t blocks = (a.rows + rpb - 1) / rpb;
    if (blocks > 0x7fffffff) return hipErrorInvalidValue;
    const dim3 grid((unsigned)blocks), block((unsigned)nt, (unsigned)rpb);
    const int nv = (chunks + nt - 1) / nt;
    if (nv <= 1) return launch_nv<1>(a, grid, block, s);
    if (nv <= 2) return launch_nv<2>(a, grid, block, s);
    if (nv <= 4) return launch_nv<4>(a, grid, block, s);
    return hipErrorInvalidValue;
}

}  // namespace fqm
