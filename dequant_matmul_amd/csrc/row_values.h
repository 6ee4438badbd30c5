// Rows of bf16, fp32 and 8-bit values in chunks of 8, at their element's
// alignment: what the norms read and write.
#pragma once

#include "fqm_internal.h"

namespace fqm {
namespace {

constexpr int kVec = 8;            // values per chunk

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

// 8 values to p[e ...], those of [lo, hi) (all: one or two wide stores).
__device__ __forceinline__ void store_f32(void* p, int64_t e, const float (&h)[kVec], int lo, int hi) {
    float* q = static_cast<float*>(p) + e;
    if (lo == 0 && hi == kVec) {
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
            if (i >= lo && i < hi) q[i] = h[i];
    }
}
__device__ __forceinline__ void store_bf16(void* p, int64_t e, const float (&h)[kVec], int lo, int hi) {
    uint16_t* q = static_cast<uint16_t*>(p) + e;
    if (lo == 0 && hi == kVec) {
        u32x4 a;
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = (uint32_t)to_bf16(h[2 * i]) | (uint32_t)to_bf16(h[2 * i + 1]) << 16;
        *reinterpret_cast<u32x4_a2*>(q) = a;
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (i >= lo && i < hi) q[i] = to_bf16(h[i]);
    }
}
__device__ __forceinline__ void store_i8(void* p, int64_t e, const int (&c)[kVec], int lo, int hi) {
    uint8_t* q = static_cast<uint8_t*>(p) + e;
    if (lo == 0 && hi == kVec) {
        u32x2 a;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            a[i] = (uint32_t)(c[4 * i] & 255) | (uint32_t)(c[4 * i + 1] & 255) << 8 |
                   (uint32_t)(c[4 * i + 2] & 255) << 16 | (uint32_t)c[4 * i + 3] << 24;
        *reinterpret_cast<u32x2_a1*>(q) = a;
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (i >= lo && i < hi) q[i] = (uint8_t)c[i];
    }
}

}  // namespace
}  // namespace fqm
