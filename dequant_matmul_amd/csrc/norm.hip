// Residual addition and root-mean-square norm, one pass over the rows:
//   h = sum_t x_t + residual,   y = h * weight / sqrt(mean(h^2) + eps),
// y in bf16, fp32 or 8 bits with one scale per row.
//
// A row is read once into registers (chunks of 8 values, chunk c of the row on
// thread c mod NT), one block reduction gives the row's sum of squares and
// max|h * weight|, and the row is written from the registers.  The 8-bit codes
// need no second reduction: y's row factor r = 1/sqrt(...) is common, so
// max|y| = r * max|h w| and y / scale = h w * 127 / max|h w|.
//
// What binds it, on one MI355X: memory for many rows (8192 x 5120 bf16 59.9 us, 5.6
// TB/s; 4096 x 8 terms x 5120 to 8 bits 92 us, 4.8 TB/s), the launch and two
// dependent memory round trips (loads, then stores) for few (1 x 5120 3.6 us).
// Sums, statistics and scales are fp32; h is rounded only where total is stored.
#include <algorithm>

#include "fqm_layer.h"

namespace fqm {
namespace {

constexpr int kVec = 8;            // values per chunk
constexpr int kMaxThreads = 1024;  // per row

// 16-byte pieces at their element's alignment: rows of odd widths and strides
// start anywhere, and gfx950's global accesses take any alignment.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef u32x2 u32x2_a1 __attribute__((aligned(1)));

__device__ __forceinline__ uint16_t to_bf16(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

// Raw loads and their widening are apart, so that several loads are in flight.
template <bool F32>
struct Raw;
template <>
struct Raw<false> {
    u32x4 v;
    __device__ __forceinline__ void load(const void* p, int64_t e) {
        v = *reinterpret_cast<const u32x4_a2*>(static_cast<const uint16_t*>(p) + e);
    }
    __device__ __forceinline__ void add(float (&h)[kVec]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[2 * i] += bf16lo(v[i]);
            h[2 * i + 1] += bf16hi(v[i]);
        }
    }
    __device__ static float one(const void* p, int64_t e) { return bf16_to_f32(static_cast<const uint16_t*>(p)[e]); }
};
template <>
struct Raw<true> {
    u32x4 a, b;
    __device__ __forceinline__ void load(const void* p, int64_t e) {
        const u32x4_a4* q = reinterpret_cast<const u32x4_a4*>(static_cast<const float*>(p) + e);
        a = q[0];
        b = q[1];
    }
    __device__ __forceinline__ void add(float (&h)[kVec]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[i] += __uint_as_float(a[i]);
            h[4 + i] += __uint_as_float(b[i]);
        }
    }
    __device__ static float one(const void* p, int64_t e) { return static_cast<const float*>(p)[e]; }
};

// 8 values to p[e ...], n of them (8: one or two wide stores).
__device__ __forceinline__ void store_f32(void* p, int64_t e, const float (&h)[kVec], int n) {
    float* q = static_cast<float*>(p) + e;
    if (n == kVec) {
        u32x4 a, b;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = __float_as_uint(h[i]);
            b[i] = __float_as_uint(h[4 + i]);
        }
        reinterpret_cast<u32x4_a4*>(q)[0] = a;
        reinterpret_cast<u32x4_a4*>(q)[1] = b;
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (i < n) q[i] = h[i];
    }
}
__device__ __forceinline__ void store_bf16(void* p, int64_t e, const float (&h)[kVec], int n) {
    uint16_t* q = static_cast<uint16_t*>(p) + e;
    if (n == kVec) {
        u32x4 a;
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = (uint32_t)to_bf16(h[2 * i]) | (uint32_t)to_bf16(h[2 * i + 1]) << 16;
        *reinterpret_cast<u32x4_a2*>(q) = a;
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (i < n) q[i] = to_bf16(h[i]);
    }
}
__device__ __forceinline__ void store_i8(void* p, int64_t e, const int (&c)[kVec], int n) {
    uint8_t* q = static_cast<uint8_t*>(p) + e;
    if (n == kVec) {
        u32x2 a;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            a[i] = (uint32_t)(c[4 * i] & 255) | (uint32_t)(c[4 * i + 1] & 255) << 8 |
                   (uint32_t)(c[4 * i + 2] & 255) << 16 | (uint32_t)c[4 * i + 3] << 24;
        *reinterpret_cast<u32x2_a1*>(q) = a;
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (i < n) q[i] = (uint8_t)c[i];
    }
}

// One row per threadIdx.y; blockDim.x threads per row (16, 32, or a multiple of
// 64: a row's lanes are a part of one wave or whole waves), NV chunks each.  XF32, RF32: the types of x and of
// residual (total has the residual's type, or x's without one).
template <int NV, bool XF32, bool RF32>
__global__ __launch_bounds__(kMaxThreads) void add_rms_norm_kernel(const fqm_norm a) {
    __shared__ float s_sq[kMaxThreads / 64], s_mx[kMaxThreads / 64];
    const int nt = blockDim.x;
    const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = row < a.rows;
    const int cols = (int)a.cols;

    // this thread's chunks: columns [c0, c0 + n), n = 0 past the row's end
    float h[NV][kVec];
    float w[NV][kVec];
    int n[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c0 = kVec * (threadIdx.x + v * nt);
        n[v] = live ? max(0, min(kVec, cols - c0)) : 0;
#pragma unroll
        for (int i = 0; i < kVec; ++i) h[v][i] = 0.f, w[v][i] = 1.f;
    }
    const int64_t xr = row * a.ld_x, rr = row * a.ld_res;

    // whole chunks: every load of a term is out before the first is used
    {
        Raw<RF32> res[NV];
        Raw<XF32> x0[NV];
        u32x4 wa[NV], wb[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (n[v] == kVec) {
                const int c0 = kVec * (threadIdx.x + v * nt);
                x0[v].load(a.x, xr + c0);
                if (a.residual) res[v].load(a.residual, rr + c0);
                if (a.weight) {
                    if (a.weight_dtype == FQM_F32) {
                        const u32x4_a4* q = reinterpret_cast<const u32x4_a4*>(static_cast<const float*>(a.weight) + c0);
                        wa[v] = q[0];
                        wb[v] = q[1];
                    } else {
                        wa[v] = *reinterpret_cast<const u32x4_a2*>(static_cast<const uint16_t*>(a.weight) + c0);
                    }
                }
            }
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (n[v] == kVec) x0[v].add(h[v]);
        // further terms, four chunks' loads at a time
        constexpr int U = NV == 1 ? 4 : NV == 2 ? 2 : 1;
        for (int t = 1; t < a.terms; t += U) {
            Raw<XF32> x[U][NV];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int v = 0; v < NV; ++v)
                    if (t + u < a.terms && n[v] == kVec)
                        x[u][v].load(a.x, xr + (t + u) * a.ld_term + kVec * (threadIdx.x + v * nt));
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int v = 0; v < NV; ++v)
                    if (t + u < a.terms && n[v] == kVec) x[u][v].add(h[v]);
        }
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (n[v] == kVec) {
                if (a.residual) res[v].add(h[v]);
                if (a.weight) {
#pragma unroll
                    for (int i = 0; i < kVec; ++i)
                        w[v][i] = a.weight_dtype == FQM_F32 ? __uint_as_float(i < 4 ? wa[v][i] : wb[v][i - 4])
                                  : (i & 1)                 ? bf16hi(wa[v][i >> 1])
                                                            : bf16lo(wa[v][i >> 1]);
                }
            }
    }
    // the row's last, partial chunk, value by value
#pragma unroll
    for (int v = 0; v < NV; ++v)
        if (n[v] > 0 && n[v] < kVec) {
            const int c0 = kVec * (threadIdx.x + v * nt);
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                if (i < n[v]) {
                    for (int t = 0; t < a.terms; ++t) h[v][i] += Raw<XF32>::one(a.x, xr + t * a.ld_term + c0 + i);
                    if (a.residual) h[v][i] += Raw<RF32>::one(a.residual, rr + c0 + i);
                    if (a.weight)
                        w[v][i] = a.weight_dtype == FQM_F32 ? Raw<true>::one(a.weight, c0 + i)
                                                            : Raw<false>::one(a.weight, c0 + i);
                }
        }

    float sq = 0.f, mx = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            sq = fmaf(h[v][i], h[v][i], sq);
            w[v][i] *= h[v][i];  // from here on w holds h * weight
            mx = fmaxf(mx, fabsf(w[v][i]));
            // fmaxf passes a NaN over: an 8-bit row with one (or an infinity) gets a NaN for its scale here
            if (a.y_dtype == FQM_I8) sq = fmaf(w[v][i], 0.f, sq);
        }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1)
        if (nt > o) {  // over the row's lanes (uniform)
            sq += __shfl_xor(sq, o, 64);
            mx = fmaxf(mx, __shfl_xor(mx, o, 64));
        }
    if (nt > 64) {  // uniform over the grid: then one row per block
        const int wave = threadIdx.x >> 6, waves = nt >> 6;
        if ((threadIdx.x & 63) == 0) s_sq[wave] = sq, s_mx[wave] = mx;
        __syncthreads();
        sq = 0.f, mx = 0.f;
        for (int i = 0; i < waves; ++i) {
            sq += s_sq[i];
            mx = fmaxf(mx, s_mx[i]);
        }
    }
    if (!live) return;
    const float r = 1.f / sqrtf(sq / (float)cols + a.eps);

    if (a.total) {
        const int64_t tr = row * a.ld_total;
        const bool f32 = a.residual ? RF32 : XF32;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c0 = kVec * (threadIdx.x + v * nt);
            if (n[v] > 0) {
                if (f32) store_f32(a.total, tr + c0, h[v], n[v]);
                else store_bf16(a.total, tr + c0, h[v], n[v]);
            }
        }
    }
    const int64_t yr = row * a.ld_y;
    if (a.y_dtype == FQM_I8) {
        // a row of zeros has scale 0 with eps = 0 too, where r is infinite (a NaN in the row is in sq)
        const float scale = sq == 0.f && mx == 0.f ? 0.f : r * mx / 127.f;
        // codes: y / scale; 0 where the scale is 0, infinite or NaN (its own arithmetic decides, so that
        // the codes are 0 exactly where the stored scale cannot be used)
        const bool use = scale > 0.f && scale <= 3.4e38f;
        const float k = mx < 1e-30f ? 0x1p100f : 1.f;  // 127 / mx stays finite
        const float f = use ? 127.f / (mx * k) : 0.f;
        if (threadIdx.x == 0) a.y_scale[row] = scale;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            int c[kVec];
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                c[i] = use ? (int)fminf(127.f, fmaxf(-127.f, rintf(w[v][i] * k * f))) : 0;
            const int c0 = kVec * (threadIdx.x + v * nt);
            if (n[v] > 0) store_i8(a.y, yr + c0, c, n[v]);
        }
    } else {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c0 = kVec * (threadIdx.x + v * nt);
#pragma unroll
            for (int i = 0; i < kVec; ++i) w[v][i] *= r;
            if (n[v] > 0) {
                if (a.y_dtype == FQM_F32) store_f32(a.y, yr + c0, w[v], n[v]);
                else store_bf16(a.y, yr + c0, w[v], n[v]);
            }
        }
    }
}

template <int NV>
hipError_t launch_nv(const fqm_norm& a, dim3 grid, dim3 block, hipStream_t s) {
    const bool xf = a.x_dtype == FQM_F32, rf = a.residual ? a.res_dtype == FQM_F32 : xf;
    if (xf && rf) hipLaunchKernelGGL((add_rms_norm_kernel<NV, true, true>), grid, block, 0, s, a);
    else if (xf) hipLaunchKernelGGL((add_rms_norm_kernel<NV, true, false>), grid, block, 0, s, a);
    else if (rf) hipLaunchKernelGGL((add_rms_norm_kernel<NV, false, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((add_rms_norm_kernel<NV, false, false>), grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace

// Threads per row: a chunk each as far as 1024 threads reach (the fewest
// dependent steps); three chunks each for many rows of a single term (8192 x
// 5120 in bf16, 67.5 -> 59.9 us, 5.6 TB/s; eight terms would lose 9 %).  Rows of one
// wave or less share a 256-thread block.
hipError_t launch_add_rms_norm(const fqm_norm& a, hipStream_t s) {
    const int chunks = (int)((a.cols + kVec - 1) / kVec);
    const int per = a.rows >= 2048 && a.terms == 1 ? 3 : 1;
    const int want = (chunks + per - 1) / per;
    const int nt = chunks <= 16 ? 16 : chunks <= 32 ? 32 : std::min(kMaxThreads, (want + 63) / 64 * 64);
    const int rpb = nt <= 64 ? 256 / nt : 1;
    const int64_t blocks = (a.rows + rpb - 1) / rpb;
    if (blocks > 0x7fffffff) return hipErrorInvalidValue;
    const dim3 grid((unsigned)blocks), block((unsigned)nt, (unsigned)rpb);
    const int nv = (chunks + nt - 1) / nt;
    if (nv <= 1) return launch_nv<1>(a, grid, block, s);
    if (nv <= 2) return launch_nv<2>(a, grid, block, s);
    if (nv <= 3) return launch_nv<3>(a, grid, block, s);
    if (nv <= 4) return launch_nv<4>(a, grid, block, s);
    return hipErrorInvalidValue;
}

}  // namespace fqm
