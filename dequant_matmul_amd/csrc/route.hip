// Routing to experts: a token's k experts from its logits, their weights, and
// the plan of the products grouped by expert (a stable counting sort of the
// T k slots by expert).
//
// Choice.  c = score + bias in fp64 (without a bias the logits themselves, whose
// order is the scores'), the groups of best score, then k times the largest
// that is left; ties to the lowest index.  One wave per token, expert e on
// lane e mod 64.
//
// Plan.  Tiles of kTileSlots slots count their experts; each tile then adds up
// the counts of the tiles in front of it and ranks its slots, wave by wave:
// lanes with the same expert find each other with one ballot per bit of its
// number.  No counter is taken by whoever comes first, so the order of a
// group's rows is the slots' order, whatever the timing.
#include <algorithm>

#include "fqm_layer.h"

namespace fqm {
namespace {

constexpr int kWaves = 4;          // of the choice: a token each
constexpr int kMaxE = 1024;
constexpr int kPlanWaves = 8;
constexpr int kTileSlots = 2048;   // of the plan, per workgroup
constexpr float kLargest = 3.4028234663852886e38f;

__device__ __forceinline__ float logit(const fqm_routing& a, int64_t at) {
    const float l = a.x_dtype == FQM_F32 ? static_cast<const float*>(a.logits)[at]
                                         : bf16_to_f32(static_cast<const uint16_t*>(a.logits)[at]);
    return fminf(l, kLargest) == l || l != l ? l : kLargest;
}
__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}
// The largest value of the wave and the lowest index that has it.
template <class V>
__device__ __forceinline__ void wave_best(V& v, int& i) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
        const V ov = __shfl_xor(v, o, 64);
        const int oi = __shfl_xor(i, o, 64);
        if (ov > v || (ov == v && oi < i)) v = ov, i = oi;
    }
}

// Scores of a lane's NV logits (in fp64) under the call's rule; open: bit v is
// set where expert lane + 64 v is open.
template <int NV>
__device__ __forceinline__ void scores_f64(const fqm_routing& a, const float (&l)[NV], uint32_t open, double (&s)[NV]) {
    if (a.score == FQM_SIGMOID) {
#pragma unroll
        for (int v = 0; v < NV; ++v) s[v] = 1.0 / (1.0 + exp(-(double)l[v]));
        return;
    }
    float m = -kLargest;
#pragma unroll
    for (int v = 0; v < NV; ++v)
        if (open >> v & 1) m = fmaxf(m, l[v]);
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
    double z = 0.0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        s[v] = open >> v & 1 ? exp((double)l[v] - (double)m) : 0.0;
        z += s[v];
    }
    z = wave_sum_f64(z);
#pragma unroll
    for (int v = 0; v < NV; ++v) s[v] = z > 0.0 ? s[v] / z : 0.0;
}

template <int NV>
__global__ __launch_bounds__(64 * kWaves) void route_choose(const fqm_routing a) {
    __shared__ double s_c[kWaves][64 * NV];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * kWaves + wave;
    if (t >= a.T) return;
    const double kClosed = -INFINITY;
    float l[NV];
    double c[NV], s[NV];
    uint32_t open = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int e = lane + 64 * v;
        l[v] = -INFINITY;
        if (e < a.E) {
            l[v] = logit(a, t * a.ld_x + e);
            const float b = a.bias ? a.bias[e] : 0.f;
            if (l[v] > -INFINITY && b > -INFINITY) open |= 1u << v;
        }
    }
    const bool sums = a.groups > 1 && a.group_score == FQM_GROUP_TOP2;
    scores_f64<NV>(a, l, open, s);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int e = lane + 64 * v;
        const double sb = a.bias && e < a.E ? s[v] + (double)a.bias[e] : s[v];
        c[v] = open >> v & 1 ? (a.bias ? sb : (double)l[v]) : kClosed;
        if (a.groups > 1 && e < a.E) s_c[wave][e] = open >> v & 1 ? (sums ? sb : c[v]) : kClosed;
    }
    if (a.groups > 1) {
        wave_lds_order();
        const int per = a.E / a.groups;
        // lane g < groups: its group's score, and how many groups come before it
        double best = kClosed, second = kClosed;
        if (lane < a.groups)
            for (int i = 0; i < per; ++i) {
                const double x = s_c[wave][lane * per + i];
                if (x > best) second = best, best = x;
                else if (x > second) second = x;
            }
        if (sums && second > kClosed) best += second;
        int before = 0;
        for (int g = 0; g < a.groups; ++g) {
            const double o = __shfl(best, g, 64);
            before += o > best || (o == best && g < lane);
        }
        const uint64_t kept = __ballot(lane < a.groups && before < a.top_groups);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int e = lane + 64 * v;
            if (e < a.E && !(kept >> (e / per) & 1)) c[v] = kClosed;
        }
    }
    // lane j keeps the j-th choice
    int mine = -1;
    float ml = 0.f;
    double ms = 0.0;
    for (int j = 0; j < a.k; ++j) {
        double bv = kClosed;
        int be = kMaxE;
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (c[v] > bv) bv = c[v], be = lane + 64 * v;
        wave_best(bv, be);
        if (!(bv > kClosed)) break;  // uniform
        float bl = 0.f;
        double bs = 0.0;
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (be == lane + 64 * v) c[v] = kClosed, bl = l[v], bs = s[v];
        bl = __shfl(bl, be & 63, 64);
        bs = __shfl(bs, be & 63, 64);
        if (lane == j) mine = be, ml = bl, ms = bs;
    }
    float w = (float)ms;
    if (a.renormalise) {
        // scores up to a common factor that keeps the largest away from zero: exp(l), or
        // exp(min(l, 0)) / (1 + exp(-|l|))
        const float e = a.score == FQM_SOFTMAX ? ml : fminf(ml, 0.f);
        float m = mine >= 0 ? e : -INFINITY;
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
        w = mine >= 0 ? expf(e - m) : 0.f;
        if (a.score == FQM_SIGMOID) w /= 1.f + expf(-fabsf(ml));
        const float sum = wave_sum(w);
        w = sum > 0.f ? w / sum : 0.f;
    }
    if (lane < a.k) {
        a.expert[t * a.k + lane] = mine;
        a.weight[t * a.k + lane] = mine >= 0 ? w * a.scale : 0.f;
    }
}

// Slot i's place in the sort: its expert, E for none.
__device__ __forceinline__ int slot_key(const fqm_routing& a, int64_t i) {
    const int e = a.expert[i];
    return e < 0 ? a.E : e;
}
// The lanes (of those in `live`) whose key is this lane's.
__device__ __forceinline__ uint64_t same_key(int key, uint64_t live) {
    uint64_t m = live;
#pragma unroll
    for (int b = 0; b < 11; ++b) {
        const uint64_t has = __ballot(key >> b & 1);
        m &= key >> b & 1 ? has : ~has;
    }
    return m;
}

// hist[tile][0 .. E]: how many slots of the tile go to each expert (and to none).
__global__ __launch_bounds__(64 * kPlanWaves) void route_count(const fqm_routing a, int* __restrict__ hist, int64_t slots) {
    __shared__ int s_n[kMaxE + 1];
    for (int e = threadIdx.x; e <= a.E; e += 64 * kPlanWaves) s_n[e] = 0;
    __syncthreads();
    const int64_t first = (int64_t)blockIdx.x * kTileSlots;
    for (int i = threadIdx.x; i < kTileSlots; i += 64 * kPlanWaves)
        if (first + i < slots) atomicAdd(&s_n[slot_key(a, first + i)], 1);
    __syncthreads();
    for (int e = threadIdx.x; e <= a.E; e += 64 * kPlanWaves) hist[(int64_t)blockIdx.x * (a.E + 1) + e] = s_n[e];
}

// The plan's rows of one tile of slots.
__global__ __launch_bounds__(64 * kPlanWaves) void route_place(const fqm_routing a, const int* __restrict__ hist, int64_t slots) {
    constexpr int NT = 64 * kPlanWaves, PER = kTileSlots / kPlanWaves;
    __shared__ int s_all[kMaxE + 1];                // an expert's slots of all tiles, then its first row
    __shared__ int s_at[kPlanWaves][kMaxE + 1];     // its next row for each wave's slots
    __shared__ int s_sum[kPlanWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int tiles = gridDim.x, tile = blockIdx.x, n = a.E + 1;
    for (int e = lane; e < n; e += 64) s_at[wave][e] = 0;
    wave_lds_order();
    // each wave's own counts
    const int64_t first = (int64_t)tile * kTileSlots + wave * PER;
    for (int i = lane; i < PER; i += 64)
        if (first + i < slots) atomicAdd(&s_at[wave][slot_key(a, first + i)], 1);
    // all tiles' counts, and those of the tiles in front
    int mine[(kMaxE + NT) / NT];
#pragma unroll
    for (int q = 0; q < (kMaxE + NT) / NT; ++q) {
        const int e = tid + NT * q;
        int all = 0;
        mine[q] = 0;
        if (e < n) {
            for (int t = 0; t < tiles; ++t) {
                const int h = hist[(int64_t)t * n + e];
                all += h;
                if (t < tile) mine[q] += h;
            }
            s_all[e] = all;
        }
    }
    __syncthreads();
    // exclusive sum of the counts over the experts: thread i takes a run of them
    const int run = (n + NT - 1) / NT, lo = min(n, tid * run), hi = min(n, lo + run);
    int sum = 0;
    for (int e = lo; e < hi; ++e) sum += s_all[e];
    int upto = sum;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(upto, o, 64);
        if (lane >= o) upto += v;
    }
    if (lane == 63) s_sum[wave] = upto;
    __syncthreads();
    int at = upto - sum;
    for (int w = 0; w < wave; ++w) at += s_sum[w];
    for (int e = lo; e < hi; ++e) {
        const int c = s_all[e];
        s_all[e] = at;
        at += c;
    }
    __syncthreads();
    if (tile == 0)
        for (int e = tid; e <= a.E; e += NT) a.offsets[e] = e < a.E ? s_all[e] : (int)slots;
#pragma unroll
    for (int q = 0; q < (kMaxE + NT) / NT; ++q) {
        const int e = tid + NT * q;
        if (e < n) {
            int next = s_all[e] + mine[q];
            for (int w = 0; w < kPlanWaves; ++w) {
                const int c = s_at[w][e];
                s_at[w][e] = next;
                next += c;
            }
        }
    }
    __syncthreads();
    for (int i0 = 0; i0 < PER; i0 += 64) {
        const int64_t i = first + i0 + lane;
        const bool live = i < slots;
        const int key = live ? slot_key(a, i) : 0;
        const uint64_t peers = same_key(key, __ballot(live));
        const int before = __builtin_amdgcn_mbcnt_hi((uint32_t)(peers >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)peers, 0u));
        if (live) {
            const int to = s_at[wave][key] + before;
            const bool none = key == a.E;
            a.dst[to] = (int)i;
            a.src[to] = none ? -1 : (int)(i / a.k);
            a.row_scale[to] = none ? 0.f : a.weight[i];
        }
        wave_lds_order();
        if (live && before == 0) s_at[wave][key] += __builtin_popcountll(peers);
        wave_lds_order();
    }
}

}  // namespace

size_t route_workspace(const fqm_routing& a) {
    if (!a.offsets) return 0;
    const int64_t tiles = (a.T * a.k + kTileSlots - 1) / kTileSlots;
    return ((size_t)tiles * (a.E + 1) * 4 + 15) / 16 * 16;
}

hipError_t launch_route(const fqm_routing& a, void* ws, hipStream_t s) {
    const int64_t slots = a.T * a.k, tiles = (slots + kTileSlots - 1) / kTileSlots;
    const dim3 grid((unsigned)((a.T + kWaves - 1) / kWaves)), block(64 * kWaves);
    if (a.E <= 64) hipLaunchKernelGGL(route_choose<1>, grid, block, 0, s, a);
    else if (a.E <= 128) hipLaunchKernelGGL(route_choose<2>, grid, block, 0, s, a);
    else if (a.E <= 256) hipLaunchKernelGGL(route_choose<4>, grid, block, 0, s, a);
    else if (a.E <= 512) hipLaunchKernelGGL(route_choose<8>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(route_choose<16>, grid, block, 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.offsets) return e;
    int* hist = static_cast<int*>(ws);
    hipLaunchKernelGGL(route_count, dim3((unsigned)tiles), dim3(64 * kPlanWaves), 0, s, a, hist, slots);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL(route_place, dim3((unsigned)tiles), dim3(64 * kPlanWaves), 0, s, a, hist, slots);
    return hipGetLastError();
}

}  // namespace fqm
