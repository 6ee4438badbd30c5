// What the one-row-per-wave kernels do with their sums.
#pragma once

#include "linear.h"

namespace fqm {
namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

// y as it is (PlainOut) or fqm_linear's epilogue (LinearOut).  row(group, r, per): the row of W of wave r of `per` in
// workgroup `group`, some row past the end; x_piece(t): x's t-th 16-byte piece, all batch rows as one; done(...): lane
// 63 of wave r holds the sums.
struct PlainOut {
    const uint16_t* x;
    void* y;
    int y_f32, rows;
    __device__ __forceinline__ int row(int group, int r, int per) const { return min(group * per + r, rows - 1); }
    template <int NX>
    __device__ __forceinline__ u32x4_t x_piece(int t) const { return reinterpret_cast<const u32x4_t*>(x)[t]; }
    template <int PER, int B>
    __device__ __forceinline__ void done(int group, int r, const float (&sum)[B], float (*)[B]) const {
        const int row_u = group * PER + r;
        if ((threadIdx.x & 63) != 63 || row_u >= rows) return;
#pragma unroll
        for (int b = 0; b < B; ++b) {
            if (y_f32)
                reinterpret_cast<float*>(y)[(int64_t)b * rows + row_u] = sum[b];
            else
                reinterpret_cast<uint16_t*>(y)[(int64_t)b * rows + row_u] = f32_to_bf16(sum[b]);
        }
    }
};
struct LinearOut {
    const Linear p;
    __device__ __forceinline__ int row(int group, int r, int per) const {
        if (!p.a.gated) return min(group * per + r, p.n - 1);
        const int h = per / 2, second = r >= h;
        return min(group * h + r - second * h, p.n - 1) + second * p.n;
    }
    template <int NX>
    __device__ __forceinline__ u32x4_t x_piece(int t) const {
        const int b = t / NX;
        return *reinterpret_cast<const u32x4_t*>(p.a.X + b * p.a.ld_x + 8 * (t - b * NX));
    }
    template <int PER, int B>
    __device__ __forceinline__ void done(int group, int r, const float (&sum)[B], float (*s_sum)[B]) const {
        const int lane = threadIdx.x & 63;
        if (!p.a.gated) {
            const int c = group * PER + r;
            if (lane != 63 || c >= p.n) return;
#pragma unroll
            for (int b = 0; b < B; ++b) {
                float v[1] = {sum[b]};
                finish<false, 1>(p, b, c, v, v, 1);
            }
            return;
        }
        if (lane == 63) {
#pragma unroll
            for (int b = 0; b < B; ++b) s_sum[r][b] = sum[b];
        }
        __syncthreads();
        const int t = threadIdx.x, o = t / B, b = t - o * B, c = group * (PER / 2) + o;
        if (o >= PER / 2 || c >= p.n) return;
        float v[1] = {s_sum[o][b]};
        const float w[1] = {s_sum[o + PER / 2][b]};
        finish<true, 1>(p, b, c, v, w, 1);
    }
};

}  // namespace
}  // namespace fqm
