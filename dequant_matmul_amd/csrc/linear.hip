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

// V values (2 or 4) at their element's alignment (gfx950's global accesses take any).
template <int V>
struct Values {
    typedef float f32 __attribute__((ext_vector_type(V)));
    typedef f32 f32_at __attribute__((aligned(4)));
    typedef uint16_t u16 __attribute__((ext_vector_type(V)));
    typedef u16 u16_at __attribute__((aligned(2)));
};

__device__ __forceinline__ float load_value(const void* p, int dtype, int64_t at) {
    return dtype == FQM_F32 ? static_cast<const float*>(p)[at] : bf16_to_f32(static_cast<const uint16_t*>(p)[at]);
}
// n of them, the others 0
template <int V>
__device__ __forceinline__ void load_values(const void* p, int dtype, int64_t at, int n, float (&v)[V]) {
    if (n == V && dtype == FQM_F32) {
        const auto q = *reinterpret_cast<const typename Values<V>::f32_at*>(static_cast<const float*>(p) + at);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = q[i];
    } else if (n == V) {
        const auto q = *reinterpret_cast<const typename Values<V>::u16_at*>(static_cast<const uint16_t*>(p) + at);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = bf16_to_f32(q[i]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = i < n ? load_value(p, dtype, at + i) : 0.f;
    }
}
template <int V>
__device__ __forceinline__ void store_values(void* p, int dtype, int64_t at, const float (&v)[V], int n) {
    typename Values<V>::u16 h;
#pragma unroll
    for (int i = 0; i < V; ++i) h[i] = __builtin_bit_cast(uint16_t, (__bf16)v[i]);
    float* pf = static_cast<float*>(p) + at;
    uint16_t* ph = static_cast<uint16_t*>(p) + at;
    if (n == V && dtype == FQM_F32) {
        typename Values<V>::f32 q;
#pragma unroll
        for (int i = 0; i < V; ++i) q[i] = v[i];
        *reinterpret_cast<typename Values<V>::f32_at*>(pf) = q;
    } else if (n == V) {
        *reinterpret_cast<typename Values<V>::u16_at*>(ph) = h;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < n) {
                if (dtype == FQM_F32) pf[i] = v[i];
                else ph[i] = h[i];
            }
    }
}

// Outputs c .. c + V - 1 of row m (n of them) from their sums v, and w of the second matrix.
template <bool GATED, int V>
__device__ __forceinline__ void finish(const Linear& p, int64_t m, int c, float (&v)[V], const float (&w)[V], int n) {
    const fqm_epilogue& a = p.a;
    if (n <= 0) return;
    float b[V], wb[V], r[V];
    if (a.residual) load_values<V>(a.residual, a.res_dtype, m * a.ld_res + c, n, r);
    if (a.bias) {
        load_values<V>(a.bias, a.bias_dtype, c, n, b);
        if (GATED) load_values<V>(a.bias, a.bias_dtype, p.n + c, n, wb);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        v[i] = activate(a.act, a.bias ? v[i] + b[i] : v[i]);
        if (GATED) v[i] *= a.bias ? w[i] + wb[i] : w[i];
        if (a.residual) v[i] += r[i];
    }
    store_values<V>(a.Y, a.y_dtype, m * a.ld_y + c, v, n);
}

typedef __attribute__((address_space(3))) float lds_f;

// A wave's 32 x 32 block of sums, as the matrix instruction leaves it (lane l, item r: row
// (r % 4) + 8 (r / 4) + 4 (l / 32), column l % 32), through 1 KB of LDS of its own to neighbouring
// outputs on a lane: 8 rows at a time, items 4 q .. 4 q + 3.  m, c: Y's row and column of the block's
// first; rows: how many of its rows there are.
template <bool GATED>
__device__ __forceinline__ void finish_block(const Linear& p, lds8* own, const f32x16& acc, int64_t m, int c, int rows) {
    constexpr int V = GATED ? 2 : 4;  // outputs of a lane
    const int lane = threadIdx.x & 63, j = lane & 31, g = lane >> 5;
    lds_f* put = (lds_f*)own + 128 * g + j;
    const int row = lane >> 3, o = V * (lane & 7);
    const lds_f* get = (lds_f*)own + 32 * row + o;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
#pragma unroll
        for (int r = 0; r < 4; ++r) put[32 * r] = acc[4 * q + r];
        wave_lds_order();
        float v[V], w[V];
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = get[i], w[i] = GATED ? get[16 + i] : 0.f;
        wave_lds_order();
        if (8 * q + row < rows) finish<GATED, V>(p, m + 8 * q + row, c + o, v, w, min(V, p.n - c - o));
    }
}

// Workgroup b: M tile tt % mtiles and N tile nt0 + tt / mtiles, tt = b / ksplit, over the
// K steps of its part b % ksplit.  PARTIAL: the fp32 tile goes to part[b].
template <int BITS, int BM, int NW, bool GATED, bool PARTIAL>
__global__ __launch_bounds__(64 * NW) void linear_tile_kernel(const Linear p, int mtiles, int nt0, int ksplit,
                                                              float* __restrict__ part) {
    constexpr int BN = 32 * NW, OUT = GATED ? BN / 2 : BN;
    FQM_GEMM_TILE_LDS(BITS, BM, NW);
    const fqm_epilogue& a = p.a;
    const int b = blockIdx.x, tt = b / ksplit, ks = b - tt * ksplit;
    const int mt = tt % mtiles, nt = nt0 + tt / mtiles;
    const int64_t m0 = (int64_t)mt * BM;
    const int rows = (int)min((int64_t)BM, a.M - m0), ksteps = p.K / BK;
    const int t0 = (int)((int64_t)ks * ksteps / ksplit), t1 = (int)((int64_t)(ks + 1) * ksteps / ksplit);
    auto x_off = [&](int row) { return (uint32_t)min(row, rows - 1) * (uint32_t)a.ld_x * 2u; };
    auto tile = [&](auto wr) {
        const uint16_t* X = a.X + m0 * a.ld_x;
        if constexpr (PARTIAL)
            gemm_tile<BITS, BM, NW>(FQM_GEMM_TILE_LDS_ARGS, X, 0, x_off, p.packed, p.ld, p.lut, wr, t0, t1 - t0,
                                    [&](int row, int col, float v) { part[(size_t)b * (BM * BN) + row * BN + col] = v; });
        else
            gemm_tile<BITS, BM, NW>(FQM_GEMM_TILE_LDS_ARGS, X, 0, x_off, p.packed, p.ld, p.lut, wr, t0, t1 - t0,
                                    [&](int i, const f32x16& acc) {
                                        const int wn = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
                                        finish_block<GATED>(p, (lds8*)s_x0 + 1024 * wn, acc, m0 + 32 * i, nt * OUT + OUT / NW * wn,
                                                            rows - 32 * i);
                                    });
    };
    if constexpr (GATED) tile(StackedRows{p.n, nt * OUT});
    else tile(RunOfRows{p.N, nt * OUT});
}

// Y of the split tiles: the parts' sums in order, then the epilogue.  4 outputs a thread.
template <int BM, int NW, bool GATED>
__global__ __launch_bounds__(256) void linear_reduce(const Linear p, const float* __restrict__ part, int mtiles, int nt0,
                                                     int ksplit, int64_t groups) {
    constexpr int BN = 32 * NW, OUT = GATED ? BN / 2 : BN;
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (e >= groups) return;
    const int64_t tt = e / (BM * OUT / 4);
    const int rem = (int)(e - tt * (BM * OUT / 4)), row = rem / (OUT / 4), o = 4 * (rem - row * (OUT / 4));
    const int64_t m = (tt % mtiles) * BM + row;
    const int c = (int)(nt0 + tt / mtiles) * OUT + o;
    if (m >= p.a.M || c >= p.n) return;
    typedef float f32x4 __attribute__((ext_vector_type(4)));
    const float* q = part + (size_t)tt * ksplit * (BM * BN) + row * BN + (GATED ? 32 * (o >> 4) + (o & 15) : o);
    float v[4] = {0.f, 0.f, 0.f, 0.f}, w[4] = {0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < ksplit; ++k) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(q + (size_t)k * (BM * BN));
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += x[i];
        if (GATED) {
            const f32x4 y = *reinterpret_cast<const f32x4*>(q + (size_t)k * (BM * BN) + 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] += y[i];
        }
    }
    finish<GATED, 4>(p, m, c, v, w, min(4, p.n - c));
}

// cols == 0: the sums are of nothing.
__global__ __launch_bounds__(256) void linear_of_nothing(const Linear p, int64_t outputs) {
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (e >= outputs) return;
    const int64_t m = e / p.n;
    const int c = (int)(e - m * p.n);
    float v[2] = {0.f, 0.f};
    const float w[2] = {0.f, 0.f};
    if (p.a.gated) finish<true, 2>(p, m, c, v, w, 1);
    else finish<false, 2>(p, m, c, v, w, 1);
}

// Tiles and what is split.  Up to 256 rows all tiles are split alike, so that the
// grid has enough workgroups; above, whole rounds of 256-row tiles (one per compute
// unit) run as one launch and the N tiles that are left for a partial round are split
// along K into as many parts as make that round shortest.
struct LinearPlan {
    int bm, nw, mtiles, ntiles;
    int nt_main;      // N tiles [0, nt_main) are not split
    int ksplit;       // K parts of the others
    int64_t tail;     // the others
    size_t part_bytes;
};

// Of the current device (without one, an MI355X's).
int compute_units() {
    int dev = 0, cus = 0;
    if (hipGetDevice(&dev) != hipSuccess || hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess) {
        (void)hipGetLastError();
        return 256;
    }
    return std::max(cus, 1);
}

LinearPlan linear_plan(int64_t N, int64_t K, int64_t M, bool gated) {
    LinearPlan p;
    p.bm = M <= 32 ? 32 : M <= 256 ? 64 : 256;
    p.nw = p.bm == 256 ? 8 : 4;
    const int64_t per = gated ? 16 * p.nw : 32 * p.nw, n = gated ? N / 2 : N, steps = K / BK;
    p.mtiles = (int)((M + p.bm - 1) / p.bm);
    p.ntiles = p.nt_main = (int)((n + per - 1) / per);
    p.ksplit = 1;
    p.tail = 0;
    const int64_t tiles = (int64_t)p.mtiles * p.ntiles;
    if (p.bm < 256) {
        const int64_t parts = std::min<int64_t>({768 / tiles, steps / 8, (int64_t)8});
        if (parts > 1) p.ksplit = (int)parts, p.nt_main = 0;
    } else if (const int64_t slots = compute_units(); tiles % slots) {
        const int nt_main = (int)(tiles / slots * slots / p.mtiles);
        const int64_t tail = (int64_t)(p.ntiles - nt_main) * p.mtiles;
        int64_t best = (tail + slots - 1) / slots * steps;
        for (int64_t k = 2; k <= steps / 8 && tail * k * (256 * 256 * 4) <= ((int64_t)256 << 20); ++k) {
            const int64_t len = (tail * k + slots - 1) / slots * ((steps + k - 1) / k);
            if (len < best) best = len, p.ksplit = (int)k, p.nt_main = nt_main;
        }
    }
    p.tail = (int64_t)(p.ntiles - p.nt_main) * p.mtiles;
    p.part_bytes = (size_t)p.tail * p.ksplit * p.bm * 32 * p.nw * 4;
    return p;
}

template <int BITS, int BM, int NW, bool GATED>
hipError_t launch_tiles(const Linear& p, const LinearPlan& plan, float* part, hipStream_t s) {
    const int64_t main_tiles = (int64_t)plan.nt_main * plan.mtiles, grid = plan.tail * plan.ksplit;
    if (main_tiles > 0x7fffffff || grid > 0x7fffffff) return hipErrorInvalidValue;
    hipError_t e = hipSuccess;
    if (main_tiles > 0) {
        hipLaunchKernelGGL((linear_tile_kernel<BITS, BM, NW, GATED, false>), dim3((unsigned)main_tiles), dim3(64 * NW), 0, s, p,
                           plan.mtiles, 0, 1, nullptr);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (plan.tail == 0) return e;
    hipLaunchKernelGGL((linear_tile_kernel<BITS, BM, NW, GATED, true>), dim3((unsigned)grid), dim3(64 * NW), 0, s, p,
                       plan.mtiles, plan.nt_main, plan.ksplit, part);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const int64_t groups = plan.tail * BM * (GATED ? 4 * NW : 8 * NW);
    if ((groups + 255) / 256 > 0x7fffffff) return hipErrorInvalidValue;
    hipLaunchKernelGGL((linear_reduce<BM, NW, GATED>), dim3((unsigned)((groups + 255) / 256)), dim3(256), 0, s, p, part,
                       plan.mtiles, plan.nt_main, plan.ksplit, groups);
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
