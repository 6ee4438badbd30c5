// The product with its epilogue, weights in the per-row table formats:
//   v = W x + bias,   y = residual + act(v)   or   residual + act(v[0..n)) v[n..2n).
//
// Tiles of X rows times W rows on the matrix cores (lut_gemm_tile.h).  Where W
// is two stacked matrices, a wave's 32 rows of W are 16 of the first and the same
// 16 of the second, so that both factors of an output are in the same wave.
// Few tiles are split along K; the parts' sums go through the workspace and a
// second launch adds them in order and applies the epilogue.
#include <algorithm>

#include "activation.h"
#include "fqm_layer.h"
#include "lut_gemm_tile.h"

namespace fqm {
namespace {

// What every workgroup needs of a call.
struct Linear {
    fqm_epilogue a;
    const uint8_t* packed;
    int64_t ld;
    const uint16_t* lut;
    int N, K;  // rows and columns of W
    int n;     // columns of Y
};

// Tile columns of the two stacked matrices: block b of 32 holds outputs n0 + 16 b
// .. + 15, the first matrix's rows in columns 0..15, the second's in 16..31.
struct StackedRows {
    int n, n0;
    __device__ __forceinline__ int output(int r) const { return n0 + 16 * (r >> 5) + (r & 15); }
    __device__ __forceinline__ bool has(int r) const { return output(r) < n; }
    __device__ __forceinline__ int row(int r) const { return min(output(r), n - 1) + (r >> 4 & 1) * n; }
};

__device__ __forceinline__ float load_value(const void* p, int dtype, int64_t at) {
    return dtype == FQM_F32 ? static_cast<const float*>(p)[at] : bf16_to_f32(static_cast<const uint16_t*>(p)[at]);
}
__device__ __forceinline__ void store_value(void* p, int dtype, int64_t at, float v) {
    if (dtype == FQM_F32) static_cast<float*>(p)[at] = v;
    else static_cast<uint16_t*>(p)[at] = __builtin_bit_cast(uint16_t, (__bf16)v);
}
__device__ __forceinline__ float bias_of(const fqm_epilogue& a, int row) {
    return a.bias ? load_value(a.bias, a.bias_dtype, row) : 0.f;
}
// u of row m and column c to its place
__device__ __forceinline__ void finish(const fqm_epilogue& a, int64_t m, int c, float u) {
    if (a.residual) u += load_value(a.residual, a.res_dtype, m * a.ld_res + c);
    store_value(a.Y, a.y_dtype, m * a.ld_y + c, u);
}

// Workgroup b: M tile tt % mtiles and N tile nt0 + tt / mtiles, tt = b / ksplit, over the
// K steps of its part b % ksplit.  PARTIAL: the fp32 tile goes to part[b].
template <int BITS, int BM, int NW, bool GATED, bool PARTIAL>
__global__ __launch_bounds__(64 * NW) void linear_tile_kernel(const Linear p, int mtiles, int nt0, int ksplit,
                                                              float* __restrict__ part) {
    constexpr int BN = 32 * NW;
    FQM_GEMM_TILE_LDS(BITS, BM, NW);
    const fqm_epilogue& a = p.a;
    const int b = blockIdx.x, tt = b / ksplit, ks = b - tt * ksplit;
    const int mt = tt % mtiles, nt = nt0 + tt / mtiles;
    const int64_t m0 = (int64_t)mt * BM;
    const int rows = (int)min((int64_t)BM, a.M - m0), ksteps = p.K / BK;
    const int t0 = (int)((int64_t)ks * ksteps / ksplit), t1 = (int)((int64_t)(ks + 1) * ksteps / ksplit);
    auto x_off = [&](int row) { return (uint32_t)min(row, rows - 1) * (uint32_t)a.ld_x * 2u; };
    const uint16_t* X = a.X + m0 * a.ld_x;
    auto tile = [&](auto wr, auto out) {
        gemm_tile<BITS, BM, NW>(FQM_GEMM_TILE_LDS_ARGS, X, 0, x_off, p.packed, p.ld, p.lut, wr, t0, t1 - t0, out);
    };
    const int lane = threadIdx.x & 63, j = lane & 31, g = lane >> 5, wn = threadIdx.x >> 6;
    auto row_of = [&](int i, int r) { return 32 * i + (r & 3) + 8 * (r >> 2) + 4 * g; };
    if constexpr (PARTIAL) {
        auto out = [&](int row, int col, float v) { part[(size_t)b * (BM * BN) + row * BN + col] = v; };
        if constexpr (GATED) tile(StackedRows{p.n, nt * (BN / 2)}, out);
        else tile(RunOfRows{p.N, nt * BN}, out);
    } else if constexpr (GATED) {
        const StackedRows wr{p.n, nt * (BN / 2)};
        const int c = wr.output(32 * wn + j);
        const float bias = bias_of(a, wr.row(32 * wn + j));
        tile(wr, [&](int i, const f32x16& acc) {
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const float v = acc[r] + bias, o = __shfl_xor(v, 16, 64);
                const int row = row_of(i, r);
                if (j < 16 && row < rows && c < p.n) finish(a, m0 + row, c, activate(a.act, v) * o);
            }
        });
    } else {
        const RunOfRows wr{p.N, nt * BN};
        const int c = wr.n0 + 32 * wn + j;
        const float bias = bias_of(a, wr.row(32 * wn + j));
        tile(wr, [&](int i, const f32x16& acc) {
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int row = row_of(i, r);
                if (row < rows && c < p.n) finish(a, m0 + row, c, activate(a.act, acc[r] + bias));
            }
        });
    }
}

// Y of the split tiles: the parts' sums in order, then the epilogue.  One output a thread.
template <int BM, int NW, bool GATED>
__global__ __launch_bounds__(256) void linear_reduce(const Linear p, const float* __restrict__ part, int mtiles, int nt0,
                                                     int ksplit, int64_t outputs) {
    constexpr int BN = 32 * NW, OUT = GATED ? BN / 2 : BN;
    const fqm_epilogue& a = p.a;
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (e >= outputs) return;
    const int64_t tt = e / (BM * OUT);
    const int rem = (int)(e - tt * (BM * OUT)), row = rem / OUT, o = rem - row * OUT;
    const int64_t m = (tt % mtiles) * BM + row;
    const int c = (int)(nt0 + tt / mtiles) * OUT + o;
    if (m >= a.M || c >= p.n) return;
    const int col = GATED ? 32 * (o >> 4) + (o & 15) : o;
    const float* q = part + (size_t)tt * ksplit * (BM * BN) + row * BN + col;
    float v = 0.f, w = 0.f;
    for (int k = 0; k < ksplit; ++k) {
        v += q[(size_t)k * (BM * BN)];
        if (GATED) w += q[(size_t)k * (BM * BN) + 16];
    }
    float u = activate(a.act, v + bias_of(a, c));
    if (GATED) u *= w + bias_of(a, p.n + c);
    finish(a, m, c, u);
}

// cols == 0: the sums are of nothing.
__global__ __launch_bounds__(256) void linear_of_nothing(const Linear p, int64_t outputs) {
    const fqm_epilogue& a = p.a;
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (e >= outputs) return;
    const int64_t m = e / p.n;
    const int c = (int)(e - m * p.n);
    float u = activate(a.act, bias_of(a, c));
    if (a.gated) u *= bias_of(a, p.n + c);
    finish(a, m, c, u);
}

struct LinearPlan {
    int bm, nw, mtiles, ntiles, ksplit;
    size_t part_bytes;
};

LinearPlan linear_plan(int64_t N, int64_t K, int64_t M, bool gated) {
    LinearPlan p;
    p.bm = M <= 32 ? 32 : M <= 256 ? 64 : 256;
    p.nw = p.bm == 256 ? 8 : 4;
    const int64_t per = gated ? 16 * p.nw : 32 * p.nw, n = gated ? N / 2 : N;
    p.mtiles = (int)((M + p.bm - 1) / p.bm);
    p.ntiles = (int)((n + per - 1) / per);
    const int64_t tiles = (int64_t)p.mtiles * p.ntiles, want = p.bm == 256 ? 256 : 768;
    p.ksplit = (int)std::max<int64_t>(1, std::min<int64_t>({want / std::max<int64_t>(tiles, 1), K / BK / 8, (int64_t)8}));
    p.part_bytes = p.ksplit > 1 ? (size_t)tiles * p.ksplit * p.bm * 32 * p.nw * 4 : 0;
    return p;
}

template <int BITS, int BM, int NW, bool GATED>
hipError_t launch_tiles(const Linear& p, const LinearPlan& plan, float* part, hipStream_t s) {
    const int64_t tiles = (int64_t)plan.mtiles * plan.ntiles, grid = tiles * plan.ksplit;
    if (grid > 0x7fffffff) return hipErrorInvalidValue;
    if (plan.ksplit == 1) {
        hipLaunchKernelGGL((linear_tile_kernel<BITS, BM, NW, GATED, false>), dim3((unsigned)grid), dim3(64 * NW), 0, s, p,
                           plan.mtiles, 0, 1, nullptr);
        return hipGetLastError();
    }
    hipLaunchKernelGGL((linear_tile_kernel<BITS, BM, NW, GATED, true>), dim3((unsigned)grid), dim3(64 * NW), 0, s, p,
                       plan.mtiles, 0, plan.ksplit, part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t outputs = tiles * BM * (GATED ? 16 * NW : 32 * NW);
    hipLaunchKernelGGL((linear_reduce<BM, NW, GATED>), dim3((unsigned)((outputs + 255) / 256)), dim3(256), 0, s, p, part,
                       plan.mtiles, 0, plan.ksplit, outputs);
    return hipGetLastError();
}

template <int BITS, bool GATED>
hipError_t launch_bits(const Linear& p, void* ws, hipStream_t s) {
    const LinearPlan plan = linear_plan(p.N, p.K, p.a.M, GATED);
    float* part = static_cast<float*>(ws);
    if (plan.bm == 32) return launch_tiles<BITS, 32, 4, GATED>(p, plan, part, s);
    if (plan.bm == 64) return launch_tiles<BITS, 64, 4, GATED>(p, plan, part, s);
    return launch_tiles<BITS, 256, 8, GATED>(p, plan, part, s);
}

}  // namespace

size_t linear_workspace(const fqm_weights& w, const fqm_epilogue& a) {
    return w.cols == 0 ? 0 : linear_plan(w.rows, w.cols, a.M, a.gated).part_bytes;
}

hipError_t launch_linear(const fqm_weights& w, const fqm_epilogue& a, void* ws, hipStream_t s) {
    Linear p;
    p.a = a;
    const bool six = w.format == FQM_LUT6;
    p.packed = six ? w.lut6.packed : w.lut4.packed;
    p.ld = six ? w.lut6.ld : w.lut4.ld;
    p.lut = six ? w.lut6.lut : w.lut4.lut;
    p.N = (int)w.rows;
    p.K = (int)w.cols;
    p.n = a.gated ? p.N / 2 : p.N;
    if (p.K == 0) {
        const int64_t outputs = a.M * p.n, grid = (outputs + 255) / 256;
        if (grid > 0x7fffffff) return hipErrorInvalidValue;
        hipLaunchKernelGGL(linear_of_nothing, dim3((unsigned)grid), dim3(256), 0, s, p, outputs);
        return hipGetLastError();
    }
    if (six) return a.gated ? launch_bits<6, true>(p, ws, s) : launch_bits<6, false>(p, ws, s);
    return a.gated ? launch_bits<4, true>(p, ws, s) : launch_bits<4, false>(p, ws, s);
}

}  // namespace fqm
