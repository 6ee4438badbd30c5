// The norms on both sides of a block, with what lies between them:
//   u = sum_t x_t,   v = u * w1 / sqrt(mean(u^2) + eps),
//   h = residual_scale * residual + scale * act(gate) * v,
//   y = h * w2 / sqrt(mean(h^2) + eps),
// w1 and w2 the norms' weights plus an offset; y in bf16, fp32 or 8 bits with
// one scale per row.
//
// A row is read once into registers (chunks of 8 values, chunk c on thread c mod NT) and stays there over both
// reductions, so memory is touched once.  Everything a row needs is on its way before the first
// reduction waits.  A reduction is four DPP steps and two exchanges in a wave, then one through LDS
// over the waves.  Sums, statistics and scales are fp32; h is rounded only where total is stored.
//
// What binds it, on one MI355X: memory for many rows (8192 x 5120 bf16 with a gate a row 78 us, 4.3 TB/s of the
// copy's 5.1; with a gate a value 100 us, 4.2 TB/s), the waves that fit beside each other where the
// gate has a value for every column (its registers), the launch, two dependent memory round trips and two
// reductions for few (1 x 5120 4.6 us; 48 x 6 terms x 5120 to 8 bits 6.9 us).
#include <algorithm>

#include "activation.h"
#include "fqm_layer.h"
#include "row_values.h"

namespace fqm {
namespace {

constexpr int kMaxThreads = 1024;  // per row
constexpr int kRuns = 64;          // of 64 chunks, the most in a row

// 8 values of a type known at run time.
struct AnyRaw {
    u32x4 a, b;
    __device__ __forceinline__ void load(int dtype, const void* p, int64_t e) {
        if (dtype == FQM_F32) {
            const u32x4_a4* q = reinterpret_cast<const u32x4_a4*>(static_cast<const float*>(p) + e);
            a = q[0];
            b = q[1];
        } else {
            a = *reinterpret_cast<const u32x4_a2*>(static_cast<const uint16_t*>(p) + e);
        }
    }
    __device__ __forceinline__ void get(int dtype, float (&f)[kVec]) const {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            f[i] = dtype == FQM_F32 ? __uint_as_float(i < 4 ? a[i] : b[i - 4]) : (i & 1) ? bf16hi(a[i >> 1]) : bf16lo(a[i >> 1]);
    }
};
// The same, of bf16 only: half the registers.
struct Bf16Raw {
    Raw<false> r;
    __device__ __forceinline__ void load(int, const void* p, int64_t e) { r.load(p, e); }
    __device__ __forceinline__ void get(int, float (&f)[kVec]) const {
#pragma unroll
        for (int i = 0; i < kVec; ++i) f[i] = 0.f;
        r.add(f);
    }
};
__device__ __forceinline__ float value_of(int dtype, const void* p, int64_t e) {
    return dtype == FQM_F32 ? Raw<true>::one(p, e) : Raw<false>::one(p, e);
}

// Over a row's nt threads (nt > 64: over the workgroup); the same in all of them.
template <int CTRL>
__device__ __forceinline__ float row16(float x) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, false));
}
template <bool MAX>
__device__ __forceinline__ float join(float a, float b) { return MAX ? fmaxf(a, b) : a + b; }
template <bool MAX>
__device__ __forceinline__ float reduce_16(float v) {
    v = join<MAX>(v, row16<0xB1>(v));   // quad_perm [1,0,3,2]
    v = join<MAX>(v, row16<0x4E>(v));   // quad_perm [2,3,0,1]
    v = join<MAX>(v, row16<0x141>(v));  // row_half_mirror
    return join<MAX>(v, row16<0x140>(v));  // row_mirror
}
template <bool MAX>
__device__ __forceinline__ float reduce_across(float v) {
    v = join<MAX>(v, __shfl_xor(v, 16, 64));
    return join<MAX>(v, __shfl_xor(v, 32, 64));
}
template <bool MAX>
__device__ __forceinline__ float reduce_lanes(int nt, float v) {
    v = reduce_16<MAX>(v);
    if (nt > 16) v = join<MAX>(v, __shfl_xor(v, 16, 64));  // uniform, as the next
    if (nt > 32) v = join<MAX>(v, __shfl_xor(v, 32, 64));
    return v;
}
// sum[v], mx[v]: the chunk's.  Chunks are added up 64 neighbours at a time, whatever threads hold them, so that a
// row's bits do not depend on NV.
template <int NV, bool WITH_MAX>
__device__ __forceinline__ void row_reduce(int nt, const float (&sum)[NV], const float (&mx)[NV], float* total, float* largest,
                                           float (*s)[kRuns]) {
    float r[NV], m[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        r[v] = reduce_lanes<false>(nt, sum[v]);
        if (WITH_MAX) m[v] = reduce_lanes<true>(nt, mx[v]);
    }
    *total = r[0];
    if (WITH_MAX) *largest = m[0];
    if (NV > 1 || nt > 64) {  // uniform over the grid: then one row per workgroup
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = nt >> 6;
        if (lane == 0)
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                s[0][v * waves + wave] = r[v];
                if (WITH_MAX) s[1][v * waves + wave] = m[v];
            }
        __syncthreads();
        const int runs = NV * waves, at = runs > 16 ? lane : lane & 15;
        float t = reduce_16<false>(at < runs ? s[0][at] : 0.f);
        if (runs > 16) t = reduce_across<false>(t);
        *total = t;
        if (WITH_MAX) {
            t = reduce_16<true>(at < runs ? s[1][at] : 0.f);
            if (runs > 16) t = reduce_across<true>(t);
            *largest = t;
        }
    }
}

// A thread's chunk of a row: columns [c0, c0 + 8), of which [lo, hi) are its own.  The last chunk of a row that 8 does
// not divide starts early, so that its loads are whole too; a row of less than 8 is read value by value.
struct Chunk {
    int c0, lo, hi;
    Chunk() = default;
    __device__ __forceinline__ Chunk(int c, int cols, bool live) {
        const int n = live ? max(0, min(kVec, cols - c)) : 0;
        lo = cols >= kVec && n > 0 ? kVec - n : 0;
        hi = lo + n;
        c0 = c - lo;
    }
    __device__ __forceinline__ bool any() const { return hi > lo; }
    __device__ __forceinline__ bool has(int i) const { return i >= lo && i < hi; }
};

// h's norm and y: the second half of a row.  w: the weights.
template <int NV>
__device__ __forceinline__ void norm_row(const fqm_block& a, int nt, int64_t row, bool live, const Chunk (&q)[NV], const float (&h)[NV][kVec],
                                         float (&w)[NV][kVec], float (*s_red)[kRuns]) {
    float part[NV], most[NV], sq = 0.f, mx = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        part[v] = most[v] = 0.f;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            part[v] = fmaf(h[v][i], h[v][i], part[v]);
            // from here on w holds h * weight; values that are not the thread's are 0, whatever their weight
            w[v][i] = q[v].has(i) ? w[v][i] * h[v][i] : 0.f;
            most[v] = fmaxf(most[v], fabsf(w[v][i]));
            // fmaxf passes a NaN over: an 8-bit row with one (or an infinity) gets a NaN for its scale here
            if (a.y_dtype == FQM_I8) part[v] = fmaf(w[v][i], 0.f, part[v]);
        }
    }
    if (a.y_dtype == FQM_I8) row_reduce<NV, true>(nt, part, most, &sq, &mx, s_red);
    else row_reduce<NV, false>(nt, part, most, &sq, &mx, s_red);
    if (!live) return;
    const float r = 1.f / sqrtf(sq / (float)(int)a.cols + a.eps);
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
            if (q[v].any()) store_i8(a.y, yr + q[v].c0, c, q[v].lo, q[v].hi);
        }
    } else {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
#pragma unroll
            for (int i = 0; i < kVec; ++i) w[v][i] *= r;
            if (q[v].any()) {
                if (a.y_dtype == FQM_F32) store_f32(a.y, yr + q[v].c0, w[v], q[v].lo, q[v].hi);
                else store_bf16(a.y, yr + q[v].c0, w[v], q[v].lo, q[v].hi);
            }
        }
    }
}
template <bool XF32, bool RF32>
__device__ __forceinline__ void store_total(const fqm_block& a, int64_t row, const Chunk& q, const float (&h)[kVec]) {
    const int64_t e = row * a.ld_total + q.c0;
    if (a.residual ? RF32 : XF32) store_f32(a.total, e, h, q.lo, q.hi);
    else store_bf16(a.total, e, h, q.lo, q.hi);
}
__device__ __forceinline__ float scalar_gate(const fqm_block& a, float value) {
    float one[1] = {value};
    activate<1>(a.gate_act, one);
    return one[0];
}

// One row per threadIdx.y; blockDim.x threads per row (16, 32, or a multiple of
// 64: a row's lanes are a part of one wave or whole waves), NV chunks each.  Every load is out before the first
// reduction.
// MORE: several terms.  GATE: a gate with a value for each column.  W: AnyRaw, or Bf16Raw where the weights and such a gate
// are bf16.
template <int NV, bool XF32, bool RF32, bool MORE, bool GATE, class W>
__global__ __launch_bounds__(kMaxThreads) void block_norm_kernel(const fqm_block a) {
    __shared__ float s_red[2][2][kRuns];
    constexpr int U = NV == 1 ? 7 : 1;  // terms' loads in flight behind the first's
    constexpr bool LATE = NV > 1 && MORE;  // rows of more than 8192 columns: what the sum does not need is loaded at its use
    constexpr int HELD = LATE ? 1 : NV;
    const int nt = blockDim.x;
    const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = row < a.rows;
    const int cols = (int)a.cols;
    const int64_t xr = row * a.ld_x, gr = row * a.ld_gate;
    const bool wide = cols >= kVec, gates = GATE && a.gate && a.step_gate, next = a.y && a.weight;
    Chunk q[NV];
    float h[NV][kVec];
    W w1[HELD], w2[HELD], g[GATE ? HELD : 1];
    Raw<RF32> res[HELD];
    auto load_rest = [&](int v, int to) {
        if (a.residual) res[to].load(a.residual, row * a.ld_res + q[v].c0);
        if (gates) g[GATE ? to : 0].load(a.gate_dtype, a.gate, gr + q[v].c0);
        if (a.post_weight) w1[to].load(a.post_dtype, a.post_weight, q[v].c0);
        if (next) w2[to].load(a.weight_dtype, a.weight, q[v].c0);
    };
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        q[v] = Chunk(kVec * (threadIdx.x + v * nt), cols, live);
#pragma unroll
        for (int i = 0; i < kVec; ++i) h[v][i] = 0.f;
    }
    if (wide) {
        Raw<XF32> x[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (q[v].any()) {
                x[v].load(a.x, xr + q[v].c0);
                if (!LATE) load_rest(v, v);
            }
        if (MORE)
        for (int t = 1; t < a.terms; t += U) {
            Raw<XF32> more[U][NV];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int v = 0; v < NV; ++v)
                    if (t + u < a.terms && q[v].any()) more[u][v].load(a.x, xr + (t + u) * a.ld_term + q[v].c0);
            if (t == 1) {
#pragma unroll
                for (int v = 0; v < NV; ++v) x[v].add(h[v]);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int v = 0; v < NV; ++v)
                    if (t + u < a.terms) more[u][v].add(h[v]);
        }
        if (!MORE || a.terms == 1) {
#pragma unroll
            for (int v = 0; v < NV; ++v) x[v].add(h[v]);
        }
    } else {
        for (int t = 0; t < a.terms; ++t)
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                if (q[0].has(i)) h[0][i] += Raw<XF32>::one(a.x, xr + t * a.ld_term + i);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (!q[v].has(i)) h[v][i] = 0.f;

    float r = 1.f;
    if (a.post) {
        float sq, part[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            part[v] = 0.f;
#pragma unroll
            for (int i = 0; i < kVec; ++i) part[v] = fmaf(h[v][i], h[v][i], part[v]);
        }
        row_reduce<NV, false>(nt, part, part, &sq, nullptr, s_red[0]);
        r = 1.f / sqrtf(sq / (float)cols + a.eps);
    }
    r *= a.scale;
    if (a.gate && !gates && live) r *= scalar_gate(a, value_of(a.gate_dtype, a.gate, gr));
    float w[NV][kVec];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int at = LATE ? 0 : v;
        if (LATE && q[v].any()) load_rest(v, 0);
        float f[kVec], by[kVec];  // by: the first norm's weight times the gate
#pragma unroll
        for (int i = 0; i < kVec; ++i) by[i] = 1.f;
        if (a.post_weight) {
            if (wide) w1[at].get(a.post_dtype, by);
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                if (!wide) by[i] = q[v].has(i) ? value_of(a.post_dtype, a.post_weight, i) : 0.f;
                by[i] += a.weight_offset;
            }
        }
        if (gates) {
            if (wide) g[GATE ? at : 0].get(a.gate_dtype, f);
            else
#pragma unroll
                for (int i = 0; i < kVec; ++i) f[i] = q[v].has(i) ? value_of(a.gate_dtype, a.gate, gr + i) : 0.f;
            activate<kVec>(a.gate_act, f);
#pragma unroll
            for (int i = 0; i < kVec; ++i) by[i] *= f[i];
        }
#pragma unroll
        for (int i = 0; i < kVec; ++i) h[v][i] *= by[i];
#pragma unroll
        for (int i = 0; i < kVec; ++i) f[i] = 0.f;
        if (a.residual) {
            if (wide) res[at].add(f);
            else
#pragma unroll
                for (int i = 0; i < kVec; ++i)
                    if (q[v].has(i)) f[i] = Raw<RF32>::one(a.residual, row * a.ld_res + i);
        }
#pragma unroll
        for (int i = 0; i < kVec; ++i) h[v][i] = q[v].has(i) ? fmaf(h[v][i], r, a.residual ? a.residual_scale * f[i] : 0.f) : 0.f;
        if (a.total && q[v].any()) store_total<XF32, RF32>(a, row, q[v], h[v]);
#pragma unroll
        for (int i = 0; i < kVec; ++i) w[v][i] = 1.f;
        if (next) {
            if (wide) w2[at].get(a.weight_dtype, w[v]);
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                if (!wide) w[v][i] = q[v].has(i) ? value_of(a.weight_dtype, a.weight, i) : 0.f;
                w[v][i] += a.weight_offset;
            }
        }
    }
    if (a.y) norm_row<NV>(a, nt, row, live, q, h, w, s_red[1]);
}

// The kernel for the types, and for what the call has.
template <int NV, bool XF32, bool RF32>
hipError_t launch_as(const fqm_block& a, dim3 grid, dim3 block, hipStream_t s) {
    const bool gate = a.gate && a.step_gate, more = a.terms > 1, wide = a.cols > kVec * kMaxThreads;
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, block, 0, s, a);
        return hipGetLastError();
    };
    if constexpr (NV == 1) {
        if (more) return gate ? go(block_norm_kernel<NV, XF32, RF32, true, true, AnyRaw>) : go(block_norm_kernel<NV, XF32, RF32, true, false, AnyRaw>);
        return gate ? go(block_norm_kernel<NV, XF32, RF32, false, true, AnyRaw>) : go(block_norm_kernel<NV, XF32, RF32, false, false, AnyRaw>);
    } else if constexpr (NV < 4) {
        if (NV == 2 && wide) return go(block_norm_kernel<2, XF32, RF32, true, true, AnyRaw>);
        return go(block_norm_kernel<NV, XF32, RF32, false, NV == 3, Bf16Raw>);
    } else {
        return go(block_norm_kernel<NV, XF32, RF32, true, true, AnyRaw>);
    }
}
template <int NV>
hipError_t launch_nv(const fqm_block& a, dim3 grid, dim3 block, hipStream_t s) {
    const bool xf = a.x_dtype == FQM_F32, rf = a.residual ? a.res_dtype == FQM_F32 : xf;
    if (xf) return rf ? launch_as<NV, true, true>(a, grid, block, s) : launch_as<NV, true, false>(a, grid, block, s);
    return rf ? launch_as<NV, false, true>(a, grid, block, s) : launch_as<NV, false, false>(a, grid, block, s);
}

}  // namespace

// Chunks a thread: one, for the fewest dependent steps, up to 8192 columns; the fewest that 1024 threads can hold
// beyond.  Many rows of one term take two, so that more rows share a compute unit (8192 x 5120 97 -> 78 us, 1024 x
// 5120 14.6 -> 13.1; 8192 x 1088 would lose 6 %), with a gate per column three (119 -> 100 us).  That costs registers,
// so the weights have to be bf16: with fp32 ones, and with several terms, it is one chunk (8192 x 5120 with fp32 weights 99 us
// where bf16 ones take 76; 4096 x 5120 of 2, 6 and 8 terms 76, 96 and 108 us, 2.8 to 4.3 TB/s).
hipError_t launch_block_norm(const fqm_block& a, hipStream_t s) {
    const int chunks = (int)((a.cols + kVec - 1) / kVec);
    const bool bf16 = (!a.post_weight || a.post_dtype == FQM_BF16) && (!a.weight || a.weight_dtype == FQM_BF16) &&
                      (!a.gate || !a.step_gate || a.gate_dtype == FQM_BF16);
    int per = chunks > 2 * kMaxThreads ? 4 : chunks > kMaxThreads ? 2 : 1;
    if (per == 1 && chunks >= 256 && a.rows >= 1024 && a.terms == 1 && bf16) per = a.gate && a.step_gate ? 3 : 2;
    const int threads = (chunks + per - 1) / per;
    const int nt = threads <= 16 ? 16 : threads <= 32 ? 32 : (threads + 63) / 64 * 64;
    const int rpb = nt <= 64 && per == 1 ? 256 / nt : 1;
    const int64_t blocks = (a.rows + rpb - 1) / rpb;
    if (blocks > 0x7fffffff) return hipErrorInvalidValue;
    const dim3 grid((unsigned)blocks), block((unsigned)nt, (unsigned)rpb);
    if (per == 1) return launch_nv<1>(a, grid, block, s);
    if (per == 2) return launch_nv<2>(a, grid, block, s);
    if (per == 3) return launch_nv<3>(a, grid, block, s);
    return launch_nv<4>(a, grid, block, s);
}

}  // namespace fqm
