// Per-row LUT GEMM (prefill): Y[m][n] = sum_k X[m][k] * lut[n][code[n][k]],
// 6-bit codes (64-entry tables) or 4-bit codes (16-entry tables).
//
// Source: "Qwen3.8-27B - BenQ 6-bit", "What BenQ stores": decode is the
// row-wise gather of codes into the row's table, fused into the matrix
// product so the decoded matrix is never written out ("Why equal-width
// shells" places 8 tiers in 4 bits, read the same way).  The text below
// gives the 6-bit sizes; 4-bit codes take 16 bytes per lane per step and
// 2 KB table planes.  Each workgroup owns a
// BM x BN tile of Y and contracts it on the bf16 matrix cores
// (v_mfma_f32_32x32x16_bf16, fp32 accumulate); the decoded weights are exact
// (the table entries are bf16).
//
// Decode straight into matrix operands.  The workgroup's 8 waves share the
// 256 X rows of the tile; each wave owns 32 rows of W (columns of Y).  For
// each 16-wide k slice, lane (j, g) of the wave
// (j = lane % 32, g = lane / 32) needs 8 consecutive weights of W row j as its
// B operand: it takes the 8 codes from registers (loaded from global memory
// three steps ahead, 24 bytes per lane per step), gathers the 8 bf16 values from
// row j's table in LDS and packs them into the operand.  The same B operand
// feeds eight MFMAs (the tile's eight 32-row blocks of X), so each gathered
// weight serves 256 rows of X.  W never passes through LDS as a tile, and no
// code bytes are staged in LDS.
//
// k order.  Inside a K step of 64, lane half g takes the step's codes
// [32 g, 32 g + 32) (bytes [24 g, 24 g + 24) of the row's 48-byte chunk) and
// slice q of the step uses k = 32 g + 8 q + e (e = 0..7).  The X operand reads
// use the same k order (16-byte chunk 4 g + q of the X row), so each product
// pairs the right X and W values; only the order of the fp32 sums differs
// from the plain k order.
//
// Table layout (bank-sliced).  Entry e of tile row r (0..255) sits at
//   8192 (r / 64) + 128 e + 4 (r % 32) + 2 ((r / 32) % 2),
// so the 32 lanes of a half-wave (the 32 rows of one 32-row group, any
// codes) hit 32 distinct banks: gathers never conflict.  A code c becomes the
// gather address (c << 7) | base_lane, i.e. one shift and one v_and_or_b32.
//
// X: three 256 x 64 bf16 tile buffers (128-byte rows, 16-byte chunks
// XOR-swizzled by (row / 2) % 8 so the operand reads of 16 rows hit 16
// distinct bank groups), filled by direct global -> LDS loads one step ahead.
// One workgroup barrier per step publishes the next X tile; with three
// buffers it needs no wait for the wave's LDS reads, so the operand reads
// and gathers stay one and two slices ahead of the MFMAs across it.  LDS:
// 96 KB of X and 32 KB of tables, one workgroup per compute unit.
//
// Tile order: workgroups are dispatched round-robin over the 8 XCDs, and
// workgroup b computes M tile b % mtiles, so with M = 8 * BM each XCD keeps
// one X panel (BM x K bf16, 2.6 MB at K = 5120) in its own L2 while the W
// panels stream through.
#include <algorithm>

#include "lut_gemm_tile.h"

namespace fqm {
namespace {

// Tile heights: BM rows of X per workgroup (256 for prefill; 64 for small M,
// where a 256-row tile would mostly multiply padding).
constexpr int BM_BIG = 256, BM_SMALL = 64;
constexpr int NWAVE = 8, BN = 32 * NWAVE;

#define FQM_GEMM_ARGS                                                                                    \
    const uint16_t *__restrict__ X, const uint8_t *__restrict__ packed, int64_t ld,                      \
        const uint16_t *__restrict__ lut, uint16_t *__restrict__ Y, float *__restrict__ part, int M, int N, \
        int K, int mtiles, int nt0, int ksplit
// Workgroup b computes tile (M tile tt % mtiles, N tile nt0 + tt / mtiles),
// tt = b / ksplit, over the K steps of its split b % ksplit.  PARTIAL:
// the fp32 tile (all BM x BN values) goes to part[b]; otherwise the bf16
// outputs inside M x N go to Y.  Rows past M repeat row M - 1 (never stored);
// the host keeps M * K * 2 below 2^31.
template <int BITS, bool PARTIAL, int BM>
__device__ __forceinline__ void plan_tile(FQM_GEMM_ARGS) {
    const int b = blockIdx.x;
    const int tt = b / ksplit, ks = b - tt * ksplit;
    const int mt = tt % mtiles, nt = nt0 + tt / mtiles;
    const int m0 = mt * BM, n0 = nt * BN;
    const int ksteps = K / BK;
    const int t0 = (int)((int64_t)ks * ksteps / ksplit), t1 = (int)((int64_t)(ks + 1) * ksteps / ksplit);
    auto x_off = [&](int row) { return (uint32_t)(min(row, M - 1 - m0) * K) * 2u; };
    FQM_GEMM_TILE_LDS(BITS, BM, NWAVE);
    gemm_tile<BITS, BM, NWAVE>(FQM_GEMM_TILE_LDS_ARGS, X, (uint32_t)m0 * (uint32_t)K * 2u, x_off, packed, ld, lut, N, n0, t0, t1 - t0,
                               [&](int row, int col, float v) {
                                   if constexpr (PARTIAL) {
                                       part[(size_t)b * (BM * BN) + row * BN + col] = v;
                                   } else {
                                       const int m = m0 + row, n = n0 + col;
                                       if (m < M && n < N) Y[(int64_t)m * N + n] = f32_to_bf16(v);
                                   }
                               });
}
template <bool PARTIAL>
__global__ __launch_bounds__(64 * NWAVE) void lut6_gemm_kernel(FQM_GEMM_ARGS) {
    plan_tile<6, PARTIAL, BM_BIG>(X, packed, ld, lut, Y, part, M, N, K, mtiles, nt0, ksplit);
}
// 64-row tiles: 56 KB of LDS and at most 128 VGPRs (four waves per SIMD), so
// two workgroups share a CU
template <bool PARTIAL>
__global__ __launch_bounds__(64 * NWAVE) __attribute__((amdgpu_waves_per_eu(4))) void lut6_gemm_small_kernel(
    FQM_GEMM_ARGS) {
    plan_tile<6, PARTIAL, BM_SMALL>(X, packed, ld, lut, Y, part, M, N, K, mtiles, nt0, ksplit);
}
template <bool PARTIAL>
__global__ __launch_bounds__(64 * NWAVE) void lut4_gemm_kernel(FQM_GEMM_ARGS) {
    plan_tile<4, PARTIAL, BM_BIG>(X, packed, ld, lut, Y, part, M, N, K, mtiles, nt0, ksplit);
}
template <bool PARTIAL>
__global__ __launch_bounds__(64 * NWAVE) __attribute__((amdgpu_waves_per_eu(4))) void lut4_gemm_small_kernel(
    FQM_GEMM_ARGS) {
    plan_tile<4, PARTIAL, BM_SMALL>(X, packed, ld, lut, Y, part, M, N, K, mtiles, nt0, ksplit);
}
#undef FQM_GEMM_ARGS

// Y for the split tiles: the ksplit fp32 partial tiles of tile tt summed in
// split order (a fixed order), rounded once to bf16.  Thread: 4 consecutive
// columns of one tile row.
template <int BM>
__global__ __launch_bounds__(256) void lut6_gemm_reduce(const float* __restrict__ part, uint16_t* __restrict__ Y,
                                                        int M, int N, int mtiles, int nt0, int ksplit,
                                                        int64_t groups) {
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;  // (tile, row, column group)
    if (e >= groups) return;
    constexpr int G = BN / 4;
    const int64_t tt = e / (BM * G);
    const int rem = (int)(e - tt * (BM * G));
    const int ml = rem / G, nl = 4 * (rem - ml * G);
    const int mt = (int)(tt % mtiles), nt = nt0 + (int)(tt / mtiles);
    const int m = mt * BM + ml, n = nt * BN + nl;
    if (m >= M) return;
    const float* p = part + (size_t)tt * ksplit * (BM * BN) + ml * BN + nl;
    float4 sum = *reinterpret_cast<const float4*>(p);
    for (int k = 1; k < ksplit; ++k) {
        const float4 v = *reinterpret_cast<const float4*>(p + (size_t)k * (BM * BN));
        sum.x += v.x; sum.y += v.y; sum.z += v.z; sum.w += v.w;
    }
    uint16_t* y = Y + (int64_t)m * N + n;
    if (n + 0 < N) y[0] = f32_to_bf16(sum.x);
    if (n + 1 < N) y[1] = f32_to_bf16(sum.y);
    if (n + 2 < N) y[2] = f32_to_bf16(sum.z);
    if (n + 3 < N) y[3] = f32_to_bf16(sum.w);
}

// Tile plan.  Whole rounds of tiles (one per resident workgroup: one per
// compute unit for 256-row tiles, two for 64-row tiles)
// run as one launch.  The N tiles left for a last, partial round are split
// along K into ksplit parts (of at least MIN_SPLIT_STEPS steps; at most
// MAX_SPLIT_SMALL parts for 64-row tiles, whose fp32 partials would
// otherwise outweigh the weights) and their fp32 partial tiles are reduced
// afterwards.  ksplit minimises the last round's length in K steps,
// ceil(tail * k / slots) * ceil(steps / k): for 32 tail tiles of 80 steps on
// 256 slots that is 8 parts (one round of 10 steps); for 160 tiles of 272
// steps (the 5120 x 17408 layer at 2048 rows) 3 parts, two rounds of 91
// steps instead of one round of 272 on 160 of the 256 compute units.  Ties
// take the fewer parts, and the partials are capped at MAX_SPLIT_BYTES.
constexpr int MIN_SPLIT_STEPS = 8;
constexpr int MAX_SPLIT_SMALL = 4;
constexpr int64_t MAX_SPLIT_BYTES = (int64_t)256 << 20;
constexpr int64_t SMALL_M_MAX = 64;  // M up to this takes 64-row tiles (measured: faster up to 64 rows, slower at 128 and 256)

struct GemmPlan {
    int bm = BM_BIG;      // tile height
    int mtiles = 0, ntiles = 0;
    int nt_main = 0;      // N tiles [0, nt_main) in the direct launch
    int ksplit = 1;       // K parts of each remaining tile
    int64_t tail = 0;     // remaining tiles ((ntiles - nt_main) * mtiles)
    size_t ws_bytes = 0;  // tail * ksplit fp32 partial tiles
};

GemmPlan gemm_plan(int64_t rows, int64_t cols, int64_t M, int cus) {
    GemmPlan p;
    const bool small = M <= SMALL_M_MAX;
    p.bm = small ? BM_SMALL : BM_BIG;
    p.mtiles = (int)((M + p.bm - 1) / p.bm);
    p.ntiles = (int)((rows + BN - 1) / BN);
    p.nt_main = p.ntiles;
    const int64_t tiles = (int64_t)p.mtiles * p.ntiles, slots = (int64_t)std::max(cus, 1) * (small ? 2 : 1);
    if (tiles % slots == 0) return p;
    const int nt_main = (int)((tiles / slots) * slots / p.mtiles);
    const int64_t tail = (int64_t)(p.ntiles - nt_main) * p.mtiles;
    const int64_t steps = cols / BK;
    int64_t kmax = steps / MIN_SPLIT_STEPS;
    if (small) kmax = std::min<int64_t>(kmax, MAX_SPLIT_SMALL);
    int64_t ksplit = 1, best = ((tail + slots - 1) / slots) * steps;
    for (int64_t k = 2; k <= kmax; ++k) {
        if (tail * k * p.bm * BN * (int64_t)sizeof(float) > MAX_SPLIT_BYTES) break;
        const int64_t len = ((tail * k + slots - 1) / slots) * ((steps + k - 1) / k);
        if (len < best) best = len, ksplit = k;
    }
    if (ksplit < 2) return p;
    p.nt_main = nt_main;
    p.ksplit = (int)ksplit;
    p.tail = tail;
    p.ws_bytes = (size_t)tail * ksplit * p.bm * BN * sizeof(float);
    return p;
}

template <int BITS, int BM>
hipError_t launch_plan(const fqm_weights& w, const uint16_t* X, uint16_t* Y, int64_t M, void* ws,
                       const GemmPlan& p, hipStream_t s) {
    hipError_t e;
    const int64_t main_tiles = (int64_t)p.nt_main * p.mtiles;
    auto kernel = [](bool partial) {
        if constexpr (BITS == 4 && BM == BM_SMALL)
            return partial ? lut4_gemm_small_kernel<true> : lut4_gemm_small_kernel<false>;
        else if constexpr (BITS == 4)
            return partial ? lut4_gemm_kernel<true> : lut4_gemm_kernel<false>;
        else if constexpr (BM == BM_SMALL)
            return partial ? lut6_gemm_small_kernel<true> : lut6_gemm_small_kernel<false>;
        else
            return partial ? lut6_gemm_kernel<true> : lut6_gemm_kernel<false>;
    };
    const uint8_t* packed = BITS == 4 ? w.lut4.packed : w.lut6.packed;
    const int64_t ld = BITS == 4 ? w.lut4.ld : w.lut6.ld;
    const uint16_t* lut = BITS == 4 ? w.lut4.lut : w.lut6.lut;
    if (main_tiles > 0) {
        hipLaunchKernelGGL(kernel(false), dim3((unsigned)main_tiles), dim3(64 * NWAVE), 0, s, X,
                           packed, ld, lut, Y, nullptr, (int)M, (int)w.rows, (int)w.cols,
                           p.mtiles, 0, 1);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (p.tail > 0) {
        float* part = static_cast<float*>(ws);
        hipLaunchKernelGGL(kernel(true), dim3((unsigned)(p.tail * p.ksplit)), dim3(64 * NWAVE), 0, s,
                           X, packed, ld, lut, Y, part, (int)M, (int)w.rows, (int)w.cols,
                           p.mtiles, p.nt_main, p.ksplit);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        const int64_t groups = p.tail * BM * (BN / 4);
        hipLaunchKernelGGL(lut6_gemm_reduce<BM>, dim3((unsigned)((groups + 255) / 256)), dim3(256), 0, s, part, Y,
                           (int)M, (int)w.rows, p.mtiles, p.nt_main, p.ksplit, groups);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t device_cus(int* cus) {
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e == hipSuccess) e = hipDeviceGetAttribute(cus, hipDeviceAttributeMultiprocessorCount, dev);
    return e;
}

}  // namespace

size_t lut_gemm_workspace(const fqm_weights& w, int64_t M) {
    int cus = 0;
    if (M <= 0 || device_cus(&cus) != hipSuccess) return 0;
    return gemm_plan(w.rows, w.cols, M, cus).ws_bytes;
}

hipError_t launch_lut_gemm(const fqm_weights& w, const uint16_t* X, uint16_t* Y, int64_t M, void* ws,
                           size_t ws_bytes, hipStream_t s) {
    if ((w.format != FQM_LUT6 && w.format != FQM_LUT4) || w.cols % BK || w.rows > 0x7fffffff || M > 0x7fffffff || w.cols > 0x7fffffff ||
        M * w.cols * 2 > 0x7fffffff)
        return hipErrorInvalidValue;
    int cus = 0;
    hipError_t e = device_cus(&cus);
    if (e != hipSuccess) return e;
    const GemmPlan p = gemm_plan(w.rows, w.cols, M, cus);
    if ((int64_t)p.ntiles * p.mtiles > 0x7fffffff) return hipErrorInvalidValue;
    if (p.ws_bytes > ws_bytes || (p.ws_bytes && !ws)) return hipErrorInvalidValue;
    if (w.format == FQM_LUT4)
        return p.bm == BM_SMALL ? launch_plan<4, BM_SMALL>(w, X, Y, M, ws, p, s)
                                : launch_plan<4, BM_BIG>(w, X, Y, M, ws, p, s);
    return p.bm == BM_SMALL ? launch_plan<6, BM_SMALL>(w, X, Y, M, ws, p, s)
                            : launch_plan<6, BM_BIG>(w, X, Y, M, ws, p, s);
}

}  // namespace fqm
