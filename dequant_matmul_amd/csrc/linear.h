// The product with its epilogue (fqm_linear): what its kernels share.
#pragma once

#include "activation.h"
#include "fqm_layer.h"

namespace fqm {

// What every workgroup needs of a call.
struct Linear {
    fqm_epilogue a;
    const uint8_t* packed;
    int64_t ld;
    const uint16_t* lut;
    int N, K;  // rows and columns of W
    int n;     // columns of Y
};

// Few rows of X on the GEMV kernels with the epilogue in theirs: one to three on the shapes of
// lut6_gemv_rows_path and lut4_gemv_rows_path (a wave per row of W), up to eight on those of
// lut_gemv_mfma_supported (16 rows of W a workgroup, on the matrix cores).
hipError_t launch_lut6_linear(const Linear& p, hipStream_t s);
hipError_t launch_lut4_linear(const Linear& p, hipStream_t s);
size_t lut_linear_mfma_workspace(const Linear& p);
hipError_t launch_lut_linear_mfma(const Linear& p, bool six, float* ws, hipStream_t s);

namespace {

// Rows of W of a run of outputs o0 .. o0 + T - 1: as they lie, or with two stacked matrices T / 2 outputs' rows of
// the first and then the same of the second.  row(r): some row where there is none.
template <int T>
struct OutputRows {
    int n, o0, gated;
    __device__ __forceinline__ int output(int r) const { return o0 + (gated && r >= T / 2 ? r - T / 2 : r); }
    __device__ __forceinline__ int row(int r) const { return min(output(r), n - 1) + (gated && r >= T / 2 ? n : 0); }
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
    if (a.bias) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] += b[i];
    }
    activate<V>(a.act, v);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (GATED) v[i] *= a.bias ? w[i] + wb[i] : w[i];
        if (a.residual) v[i] += r[i];
    }
    store_values<V>(a.Y, a.y_dtype, m * a.ld_y + c, v, n);
}

}  // namespace
}  // namespace fqm
