// Products grouped by expert, weights in the per-row table formats:
//   Y[dst[i]] = row_scale[i] * (W_e X[src[i]]) for the rows i of group e.
#include "fqm_layer.h"

namespace fqm {
namespace {

// One wave per row of one expert's W; it loops over the group's rows.
template <int BITS>
__global__ __launch_bounds__(256) void grouped_rows(const uint8_t* __restrict__ packed, int64_t ld,
                                                    const uint16_t* __restrict__ lut, const fqm_groups g, int N, int K) {
    constexpr int ENTRIES = 1 << BITS;
    __shared__ uint16_t s_lut[4][ENTRIES];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int e = blockIdx.y, n = blockIdx.x * 4 + wave;
    const int64_t row = (int64_t)e * N + min(n, N - 1);
    if (lane < ENTRIES) s_lut[wave][lane] = lut[row * ENTRIES + lane];
    __syncthreads();
    if (n >= N) return;
    const int lo = max(0, min((int)g.M, g.offsets[e])), hi = max(0, min((int)g.M, g.offsets[e + 1]));
    for (int i = lo; i < hi; ++i) {
        const int64_t xr = g.src ? g.src[i] : i;
        float acc = 0.f;
        if (xr >= 0 && xr < g.x_rows)
            for (int k = lane; k < K; k += 64) {
                const int bit = BITS * k;
                const uint8_t* p = packed + row * ld + (bit >> 3);
                const uint32_t two = p[0] | ((bit & 7) + BITS > 8 ? p[1] << 8 : 0);
                const float w = bf16_to_f32(s_lut[wave][(two >> (bit & 7)) & (ENTRIES - 1)]);
                const float x = g.x_dtype == FQM_I8 ? (float)static_cast<const int8_t*>(g.X)[xr * K + k]
                                                    : bf16_to_f32(static_cast<const uint16_t*>(g.X)[xr * K + k]);
                acc = fmaf(w, x, acc);
            }
        acc = wave_sum(acc);
        if (g.x_scale && xr >= 0 && xr < g.x_rows) acc *= g.x_scale[xr];
        if (g.row_scale) acc *= g.row_scale[i];
        const int64_t yr = g.dst ? g.dst[i] : i;
        if (lane == 0 && yr >= 0 && yr < g.y_rows) {
            if (g.y_dtype == FQM_F32) static_cast<float*>(g.Y)[yr * N + n] = acc;
            else static_cast<uint16_t*>(g.Y)[yr * N + n] = __builtin_bit_cast(uint16_t, (__bf16)acc);
        }
    }
}

}  // namespace

size_t grouped_workspace(const fqm_weights& w, const fqm_groups& g) { return 0; }

hipError_t launch_grouped(const fqm_weights& w, const fqm_groups& g, void* ws, hipStream_t s) {
    const int N = (int)(w.rows / g.count), K = (int)w.cols;
    const dim3 grid((unsigned)((N + 3) / 4), (unsigned)g.count);
    if (w.format == FQM_LUT6)
        hipLaunchKernelGGL(grouped_rows<6>, grid, dim3(256), 0, s, w.lut6.packed, w.lut6.ld, w.lut6.lut, g, N, K);
    else
        hipLaunchKernelGGL(grouped_rows<4>, grid, dim3(256), 0, s, w.lut4.packed, w.lut4.ld, w.lut4.lut, g, N, K);
    return hipGetLastError();
}

}  // namespace fqm
