// Routing to experts: a token's k experts from its logits, their weights, and
// the plan of the products grouped by expert (a stable counting sort of the
// T k slots by expert).
//
// Choice: one wave per token, expert e on lane e mod 64.  An expert's score + bias (its logit, without
// a bias) in fp32, as an integer of the same order, is a key; a choice is a maximum over the wave (six DPP
// instructions) and, of the lanes that have it, the lowest expert.  One more than k are chosen with a bias.
// Where fp32's errors leave the order of these open, or which groups stay (one token in some hundreds), the
// token is put off until the wave's others are through, and chosen from scores in fp64: inside the
// loop that path's registers would cost every token its neighbours' waves.
//
// Plan: up to kMostTiles tiles of tokens count their experts as they choose; a second launch
// adds up the counts of the tiles in front of each, and ranks its slots wave by wave: lanes
// with the same expert find each other with one ballot per bit of its number.  No
// counter is taken by whoever comes first, so the order of a group's rows is the slots'
// order, whatever the timing.  The fewest tokens are one workgroup's work, in one launch.
//
// What binds it, on one MI355X: the issue of some 710 vector and 490 scalar instructions a token (256 experts, 8
// groups, k 8) and the waits between dependent ones, for many tokens (16384: 31 us, and 13 us for the
// plan, whose workgroups each read all tiles' counts); launches and the latency of one token's chain of steps
// for few (1 token 5.3 us, 48 tokens 12.6 us in two launches).  A bias of -1e4 or below on one expert opens every
// token's choice to fp64, one at a time (16384 tokens of 256 experts, no groups, 34 -> 51 us; -infinity 33).
#include <algorithm>

#include "activation.h"
#include "fqm_layer.h"

namespace fqm {
namespace {

constexpr int kMaxE = 1024;
constexpr int kFewWaves = 4;         // of a choosing workgroup with a short tile
constexpr int kMostTiles = 512;
constexpr int kPlaceWaves = 16;
constexpr int kSmallTokens = 8;      // one workgroup's work: 8 tokens of 256 experts 10.8 us, 9 in two launches 12.1; on
                                     // one compute unit 16 tokens take 13.1, as in two launches, 48 take 27, in two 13.5
constexpr float kLargest = 3.4028234663852886e38f;

// A logit as the choice takes it: +infinity is the largest number, and -0 is +0 (-0 + 0 = +0), since their order as
// integers would tell the two zeros apart.  A NaN stays one.
__device__ __forceinline__ float held(float l) { return l > kLargest ? kLargest : l + 0.f; }
// The sum over the wave in fp64, the same in every lane.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ double dpp_add_f64(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, CTRL, ROW_MASK, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(u >> 32), CTRL, ROW_MASK, 0xF, false);
    return x + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_sum_f64(double v) {
    v = dpp_add_f64<0xB1, 0xF>(v);
    v = dpp_add_f64<0x4E, 0xF>(v);
    v = dpp_add_f64<0x141, 0xF>(v);
    v = dpp_add_f64<0x140, 0xF>(v);
    v = dpp_add_f64<0x142, 0xA>(v);
    v = dpp_add_f64<0x143, 0xC>(v);
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)u, 63), hi = (uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), 63);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// The largest of the wave's, the same in every lane.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ double dpp_max_f64(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp((int)u, (int)u, CTRL, ROW_MASK, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp((int)(u >> 32), (int)(u >> 32), CTRL, ROW_MASK, 0xF, false);
    const double o = __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
    return o > x ? o : x;
}
__device__ __forceinline__ double wave_max_f64(double v) {
    v = dpp_max_f64<0xB1, 0xF>(v);
    v = dpp_max_f64<0x4E, 0xF>(v);
    v = dpp_max_f64<0x141, 0xF>(v);
    v = dpp_max_f64<0x140, 0xF>(v);
    v = dpp_max_f64<0x142, 0xA>(v);
    v = dpp_max_f64<0x143, 0xC>(v);
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)u, 63), hi = (uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), 63);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// The largest of the wave's values (0 where it has none), the same in every lane.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ uint32_t dpp_max(uint32_t x) {
    return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROW_MASK, 0xF, false));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = dpp_max<0xB1, 0xF>(v);   // quad_perm [1,0,3,2]
    v = dpp_max<0x4E, 0xF>(v);   // quad_perm [2,3,0,1]
    v = dpp_max<0x141, 0xF>(v);  // row_half_mirror
    v = dpp_max<0x140, 0xF>(v);  // row_mirror
    v = dpp_max<0x142, 0xA>(v);  // row_bcast:15
    v = dpp_max<0x143, 0xC>(v);  // row_bcast:31
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
// Floats in the order of unsigned integers, and back.
__device__ __forceinline__ uint32_t ordered(float f) {
    const uint32_t u = __float_as_uint(f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
    return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}
__device__ __forceinline__ float wave_max_f(float v) { return from_ordered(wave_max(ordered(v))); }

__device__ __forceinline__ float wave_total(float v) {  // the sum, the same in every lane
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(wave_sum_lane63(v)), 63));
}
__device__ __forceinline__ float at_lane(float v, int l) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
}
__device__ __forceinline__ double at_lane(double v, int l) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)u, l), hi = (uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), l);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// A wave's token: its logits, and which experts are open (bit v: expert lane + 64 v).
template <int NV>
struct Token {
    float l[NV];
    uint32_t open;
};
// What does not change between tokens: the experts' biases, which experts may be chosen, their groups (8 bits each).
template <int NV>
struct Experts {
    float b[NV];
    uint32_t there, group[(NV + 3) / 4];
};
// What lane j < k has chosen: its expert (-1: none) and its logit.
struct Chosen {
    int expert;
    float l;
};

// One step of joining the best and second best of neighbouring lanes.
template <class V>
__device__ __forceinline__ void join(V& best, V& second, V ob, V os) {
    const V low = ob < best ? ob : best;
    best = ob > best ? ob : best;
    second = os > second ? os : second;
    second = low > second ? low : second;
}
template <int CTRL>
__device__ __forceinline__ float dpp_move(float x) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, false));
}
template <int CTRL>
__device__ __forceinline__ double dpp_move(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, CTRL, 0xF, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(u >> 32), CTRL, 0xF, 0xF, false);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// The groups that stay, as a mask, from the values c[0 .. E) in LDS (-infinity: closed): by their best value, or the
// sum of their two best.  near: whether values that may be off by err leave it open which groups stay.
template <class V>
__device__ __forceinline__ uint64_t keep_groups(const fqm_routing& a, const V* c, bool two, V err, bool* near) {
    const int lane = threadIdx.x & 63, per = a.E / a.groups;
    const int shift = __builtin_clz(a.groups - 1) - 26;  // 2^shift lanes a group: 64 over groups, rounded up to a power of two
    const int g = lane >> shift, at = lane & ((1 << shift) - 1);
    V best = -INFINITY, second = -INFINITY;
    if (g < a.groups)
        for (int i = at; i < per; i += 1 << shift) {
            const V x = c[g * per + i];
            if (x > best) second = best, best = x;
            else if (x > second) second = x;
        }
    if (shift >= 1) join(best, second, dpp_move<0xB1>(best), dpp_move<0xB1>(second));    // quad_perm [1,0,3,2]
    if (shift >= 2) join(best, second, dpp_move<0x4E>(best), dpp_move<0x4E>(second));    // quad_perm [2,3,0,1]
    if (shift >= 3) join(best, second, dpp_move<0x141>(best), dpp_move<0x141>(second));  // row_half_mirror
    if (shift >= 4) join(best, second, dpp_move<0x140>(best), dpp_move<0x140>(second));  // row_mirror
    if (shift >= 5) join(best, second, __shfl_xor(best, 16, 64), __shfl_xor(second, 16, 64));
    if (two && second > -INFINITY) best += second;
    // each group against the others, in every lane of the group
    int before = 0;
    for (int o = 0; o < a.groups; ++o) {
        const V x = at_lane(best, o << shift);
        before += x > best || (x == best && o < g);
    }
    const uint64_t first_lanes = __ballot(at == 0 && g < a.groups);
    uint64_t stay = __ballot(before < a.top_groups) & first_lanes, kept = 0;
    if (err > 0 && a.top_groups < a.groups) {
        // the last that stays against the first that does not (one without an open expert stays last)
        const V x = at_lane(best, __builtin_ctzll(__ballot(before == a.top_groups - 1) & first_lanes));
        const V y = at_lane(best, __builtin_ctzll(__ballot(before == a.top_groups) & first_lanes));
        *near = !(x - y > 2 * err) && !(y == -INFINITY);
    }
    for (; stay; stay &= stay - 1) kept |= 1ull << (__builtin_ctzll(stay) >> shift);
    return kept;
}

// A call: inlined, its constants would be kept in registers through all of the kernel.
__device__ __attribute__((noinline)) double exp_f64(double x) { return exp(x); }

// The choice with scores in fp64, for the few tokens that need it.  s_c: E values of LDS of the wave's own.  top and
// z: the softmax's.
template <int NV>
__device__ __forceinline__ Chosen choose_exactly(const fqm_routing& a, const Token<NV>& t, const Experts<NV>& x, double* s_c,
                                                 float* top_out, float* z_out) {
    const int lane = threadIdx.x & 63;
    const double kClosed = -INFINITY;
    const bool softmax = a.score == FQM_SOFTMAX;
    float top = 0.f;
    if (softmax) {
        top = -kLargest;
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (t.open >> v & 1) top = fmaxf(top, t.l[v]);
        top = wave_max_f(top);
    }
    double c[NV], z = 0.0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        c[v] = exp_f64(softmax ? (double)t.l[v] - (double)top : -(double)t.l[v]);
        if (t.open >> v & 1) z += c[v];
    }
    z = softmax ? wave_sum_f64(z) : 1.0;
    *top_out = top;
    *z_out = (float)z;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        c[v] = a.bias || (a.groups > 1 && a.group_score == FQM_GROUP_TOP2) ? softmax ? c[v] / z : 1.0 / (1.0 + c[v]) : (double)t.l[v];
        c[v] = t.open >> v & 1 ? c[v] + (double)x.b[v] : kClosed;
    }
    if (a.groups > 1) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (lane + 64 * v < a.E) s_c[lane + 64 * v] = c[v];
        wave_lds_order();
        bool near;
        const uint64_t kept = keep_groups<double>(a, s_c, a.group_score == FQM_GROUP_TOP2, 0.0, &near);
        wave_lds_order();
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (!a.bias && t.open >> v & 1) c[v] = t.l[v];
            if (!(kept >> (x.group[v / 4] >> 8 * (v & 3) & 63) & 1)) c[v] = kClosed;
        }
    }
    Chosen mine = {-1, 0.f};
    for (int j = 0; j < a.k; ++j) {
        double best = c[0];
#pragma unroll
        for (int v = 1; v < NV; ++v) best = c[v] > best ? c[v] : best;
        best = wave_max_f64(best);
        if (!(best > kClosed)) break;  // uniform
        int e = kMaxE;
#pragma unroll
        for (int v = NV - 1; v >= 0; --v) {
            const uint64_t at = __ballot(c[v] == best);
            if (at) e = 64 * v + __builtin_ctzll(at);
        }
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (lane + 64 * v == e) c[v] = kClosed;
        if (lane == j) mine.expert = e;
    }
    float* s_l = reinterpret_cast<float*>(s_c);
#pragma unroll
    for (int v = 0; v < NV; ++v) s_l[lane + 64 * v] = t.l[v];
    wave_lds_order();
    if (mine.expert >= 0) mine.l = s_l[mine.expert];
    wave_lds_order();
    return mine;
}

// LDS of a wave: two fp32 values an expert, or one in fp64.
template <int NV>
union WaveLds {
    float f[2][64 * NV];
    double d[64 * NV];
};

// exp(l - top) with what the difference's rounding lost.
__device__ __forceinline__ float exp_below(float l, float top) {
    const float d = l - top, t = d - l;
    const float lost = (l - (d - t)) - (top + t);
    return exp_fast(d) * (1.f + fmaxf(-1.f, fminf(lost, 1.f)));
}
// The weights of what lanes j < k have chosen; top and z: the softmax's largest logit and sum, where all of it counts.
__device__ __forceinline__ float weigh(const fqm_routing& a, Chosen got, float top, float z) {
    const bool softmax = a.score == FQM_SOFTMAX, live = got.expert >= 0 && (int)(threadIdx.x & 63) < a.k;
    float w;
    if (a.renormalise) {
        // scores up to a common factor that keeps the largest away from zero: exp(l), or
        // exp(min(l, 0)) / (1 + exp(-|l|))
        const float e = softmax ? got.l : fminf(got.l, 0.f);
        const float m = wave_max_f(live ? e : -INFINITY);
        w = live ? expf(e - m) : 0.f;
        if (!softmax) w /= 1.f + expf(-fabsf(got.l));
        const float sum = wave_total(w);
        w = sum > 0.f ? w / sum : 0.f;
    } else if (softmax) {
        w = exp_below(got.l, top) / z;
    } else {
        w = logistic(got.l);
    }
    return live ? w * a.scale : 0.f;
}

// A token's experts in lanes j < k; false: fp32 leaves the choice open.
template <int NV>
__device__ __forceinline__ bool choose(const fqm_routing& a, const Token<NV>& t, const Experts<NV>& x, WaveLds<NV>* lds, Chosen* chosen,
                                       float* top_out, float* z_out) {
    const int lane = threadIdx.x & 63;
    const bool sums = a.groups > 1 && a.group_score == FQM_GROUP_TOP2, softmax = a.score == FQM_SOFTMAX;
    const bool scored = a.bias || sums || (softmax && !a.renormalise);  // whether all scores are needed
    float s[NV], c[NV], top = 0.f, z = 1.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) s[v] = 0.f;
    if (scored && softmax) {
        top = -kLargest;
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (t.open >> v & 1) top = fmaxf(top, t.l[v]);
        top = wave_max_f(top);
        double part = 0.0;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            s[v] = t.open >> v & 1 ? exp_below(t.l[v], top) : 0.f;
            part += (double)s[v];
        }
        z = (float)wave_sum_f64(part);
        const float r = z > 0.f ? 1.f / z : 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) s[v] *= r;
    } else if (scored) {
#pragma unroll
        for (int v = 0; v < NV; ++v) s[v] = logistic(t.l[v]);
    }
    // How far s + bias may be off, U = 2^-24: 7 U of a sigmoid and U of the sum; of a softmax 6 U for the exponential,
    // as many and U for z, 4 U for its reciprocal and the product.
    const float unit = softmax ? 0x1p-19f : 0x1p-20f;
    float bmax = 0.f;
    if (a.bias) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (t.open >> v & 1) bmax = fmaxf(bmax, fabsf(x.b[v]));
        bmax = wave_max_f(bmax);
    }
    uint32_t key[NV];  // 0: closed
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        c[v] = a.bias ? s[v] + x.b[v] : t.l[v];
        key[v] = t.open >> v & 1 ? ordered(c[v]) : 0u;
    }
    bool near = false;
    if (a.groups > 1) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int e = lane + 64 * v;
            if (e < a.E) lds->f[0][e] = t.open >> v & 1 ? (sums && !a.bias ? s[v] : c[v]) : -INFINITY;
        }
        wave_lds_order();
        const float off = unit * (1.f + bmax);
        const uint64_t kept = keep_groups<float>(a, lds->f[0], sums, sums ? 2 * off : a.bias ? off : 0.f, &near);
        wave_lds_order();
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (!(kept >> (x.group[v / 4] >> 8 * (v & 3) & 63) & 1)) key[v] = 0u;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        lds->f[0][lane + 64 * v] = t.l[v];
        lds->f[1][lane + 64 * v] = c[v];
    }
    // the k + 1 first, the j-th in lane j; without a bias the keys are the logits, whose order is exact
    const int wanted = a.k + (a.bias ? 1 : 0);
    Chosen got = {-1, 0.f};
    int found = 0;
    for (; found < wanted; ++found) {
        uint32_t m = key[0];
#pragma unroll
        for (int v = 1; v < NV; ++v) m = max(m, key[v]);
        m = wave_max(m);
        if (m == 0u) break;  // uniform
        int e = kMaxE;
#pragma unroll
        for (int v = NV - 1; v >= 0; --v) {
            const uint64_t at = __ballot(key[v] == m);
            if (at) e = 64 * v + __builtin_ctzll(at);
        }
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (lane + 64 * v == e) key[v] = 0u;
        if (lane == found) got.expert = e;
    }
    wave_lds_order();
    float cj = 0.f;
    if (got.expert >= 0) {
        got.l = lds->f[0][got.expert];
        cj = lds->f[1][got.expert];
    }
    wave_lds_order();
    if (a.bias) {
        const float err = unit * (fabsf(at_lane(cj, 0)) + 2 * bmax);  // no score is larger than the first c and bmax
        const float cn = __shfl(cj, min(lane + 1, 63), 64);
        near |= __ballot(lane < min(a.k, found - 1) && !(cj - cn > 2 * err)) != 0;
    }
    *chosen = got;
    *top_out = top;
    *z_out = z;
    return !near;
}

template <int NV>
__device__ __forceinline__ void load_token(const fqm_routing& a, int64_t row, Token<NV>* t) {
    const int lane = threadIdx.x & 63;
    if (a.x_dtype == FQM_F32) {
        const float* l = static_cast<const float*>(a.logits) + row * a.ld_x;
#pragma unroll
        for (int v = 0; v < NV; ++v) t->l[v] = l[min(lane + 64 * v, a.E - 1)];
    } else {
        const uint16_t* l = static_cast<const uint16_t*>(a.logits) + row * a.ld_x;
#pragma unroll
        for (int v = 0; v < NV; ++v) t->l[v] = bf16_to_f32(l[min(lane + 64 * v, a.E - 1)]);
    }
}
// What is left to do once they have come.
template <int NV>
__device__ __forceinline__ void open_token(const Experts<NV>& x, Token<NV>* t) {
    t->open = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        t->l[v] = held(t->l[v]);
        if ((x.there >> v & 1) && t->l[v] > -INFINITY) t->open |= 1u << v;
    }
}
template <int NV>
__device__ __forceinline__ void load_experts(const fqm_routing& a, Experts<NV>* x) {
    const int lane = threadIdx.x & 63, per = a.E / a.groups;
    x->there = 0;
#pragma unroll
    for (int q = 0; q < (NV + 3) / 4; ++q) x->group[q] = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int e = lane + 64 * v;
        x->b[v] = a.bias && e < a.E ? a.bias[e] : 0.f;
        if (e < a.E && x->b[v] > -INFINITY) x->there |= 1u << v;
        if (e < a.E) x->group[v / 4] |= (uint32_t)(e / per) << 8 * (v & 3);
    }
}

// Chooses for the tokens first + wave, first + wave + NW, ... below end.
// done(t, expert, weight): lane j < k has token t's j-th.  Tokens that fp32 leaves open wait until 64 are through.
template <int NV, int NW, class Done>
__device__ __forceinline__ void choose_all(const fqm_routing& a, int64_t first, int64_t end, WaveLds<NV>* lds, Done done) {
    const int lane = threadIdx.x & 63;
    for (int64_t t0 = first + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); t0 < end; t0 += 64 * NW) {
        Experts<NV> x;
        load_experts<NV>(a, &x);
        Token<NV> token;
        Chosen got;
        float top, z;
        uint64_t left = 0;
        int64_t t = t0;
        for (int r = 0; r < 64 && t < end; ++r, t += NW) {
            load_token<NV>(a, t, &token);
            open_token<NV>(x, &token);
            if (choose<NV>(a, token, x, lds, &got, &top, &z)) {
                const float w = weigh(a, got, top, z);
                if (lane < a.k) done(t, got.expert, w);
            } else {
                left |= 1ull << r;
            }
        }
        for (; left; left &= left - 1) {
            t = t0 + NW * __builtin_ctzll(left);
            load_experts<NV>(a, &x);
            load_token<NV>(a, t, &token);
            open_token<NV>(x, &token);
            got = choose_exactly<NV>(a, token, x, lds->d, &top, &z);
            const float w = weigh(a, got, top, z);
            if (lane < a.k) done(t, got.expert, w);
        }
    }
}

// A slot's place in the sort: its expert, E for none.
__device__ __forceinline__ int key_of(const fqm_routing& a, int expert) { return expert < 0 ? a.E : expert; }
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
__device__ __forceinline__ int lanes_before(uint64_t m) {
    return __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0u));
}
__device__ __forceinline__ void place(const fqm_routing& a, int to, int64_t slot, int key, float w) {
    const bool none = key == a.E;
    a.dst[to] = (int)slot;
    a.src[to] = none ? -1 : (int)(slot / a.k);
    a.row_scale[to] = none ? 0.f : w;
}
// Exclusive sums of n counts in LDS over the workgroup's NT threads, in place; s_sum: a value per wave.
template <int NT>
__device__ __forceinline__ void exclusive_sums(int* s_n, int n, int* s_sum) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int run = (n + NT - 1) / NT, lo = min(n, tid * run), hi = min(n, lo + run);
    int sum = 0;
    for (int e = lo; e < hi; ++e) sum += s_n[e];
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
        const int c = s_n[e];
        s_n[e] = at;
        at += c;
    }
    __syncthreads();
}

// Ints of a tile's counts: its slots' experts, those without one, and zeros up to whole uint4.
__host__ __device__ __forceinline__ int counts_of(int E) { return (E + 4) / 4 * 4; }

// Workgroup b: tokens [b * tile, + tile), a wave each in turn.  hist: the tiles' counts; NULL: not counted.
// The waves of a workgroup with a long tile, and what two such workgroups make of them on a SIMD, where registers allow:
// 256 experts need 77, which 16 waves would spill (16384 tokens 36 us, with 12 waves 29).
constexpr int many_waves(int nv) { return nv <= 2 ? 16 : nv <= 4 ? 12 : nv <= 8 ? 16 : 8; }
constexpr int min_waves(int nv) { return nv <= 2 ? 8 : nv <= 4 ? 6 : 2; }
template <int NV, int NW>
__global__ __launch_bounds__(64 * NW, NW == kFewWaves ? 1 : min_waves(NV)) void route_choose(const fqm_routing a, int tile,
                                                                                               int* __restrict__ hist) {
    constexpr int NT = 64 * NW;
    __shared__ WaveLds<NV> s_wave[NW];
    __shared__ int s_n[64 * NV + 4];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = counts_of(a.E);
    if (hist) {
        for (int e = tid; e < n; e += NT) s_n[e] = 0;
        __syncthreads();
    }
    const int64_t first = (int64_t)blockIdx.x * tile, end = min(first + tile, a.T);
    choose_all<NV, NW>(a, first, end, &s_wave[wave], [&](int64_t t, int expert, float weight) {
        a.expert[t * a.k + lane] = expert;
        a.weight[t * a.k + lane] = weight;
        if (hist) atomicAdd(&s_n[key_of(a, expert)], 1);
    });
    if (hist) {
        __syncthreads();
        for (int e = tid; e < n; e += NT) hist[(int64_t)blockIdx.x * n + e] = s_n[e];
    }
}

// The plan's rows of the slots of `span` tiles.
__global__ __launch_bounds__(64 * kPlaceWaves) void route_place(const fqm_routing a, const int* __restrict__ hist, int tile, int tiles,
                                                                int span) {
    constexpr int NW = kPlaceWaves, NT = 64 * NW;
    __shared__ int s_all[kMaxE + 4];          // an expert's slots of all tiles, then its first row
    __shared__ int s_front[kMaxE + 4];        // those of the tiles in front
    __shared__ int s_at[NW][kMaxE + 1];       // its next row for each wave's slots
    __shared__ int s_sum[NW];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int n = counts_of(a.E), here = (int)blockIdx.x * span;
    const int64_t slots = a.T * a.k, first = (int64_t)here * tile * a.k, end = min(first + (int64_t)span * tile * a.k, slots);
    const int64_t per = ((end - first + NW - 1) / NW + 63) / 64 * 64;
    const int64_t lo = min(end, first + wave * per), hi = min(end, lo + per);
    const int key0 = lo + lane < hi ? key_of(a, a.expert[lo + lane]) : 0;  // the first 64 stay here
    const float w0 = lo + lane < hi ? a.weight[lo + lane] : 0.f;
    for (int e = tid; e < n; e += NT) s_all[e] = s_front[e] = 0;
    for (int e = lane; e <= a.E; e += 64) s_at[wave][e] = 0;
    __syncthreads();
    // each wave's own counts, of its run of the slots
    for (int64_t i = lo + lane; i < hi; i += 64) atomicAdd(&s_at[wave][i < lo + 64 ? key0 : key_of(a, a.expert[i])], 1);
    // all tiles' counts, and those in front: four experts a thread, of every step-th tile
    const int quads = n / 4, step = NT / quads, q = tid % quads;
    int all[4] = {}, front[4] = {};
    if (tid < step * quads) {
#pragma unroll 8
        for (int t = tid / quads; t < tiles; t += step) {
            const int4 h = reinterpret_cast<const int4*>(hist)[(int64_t)t * quads + q];
            const int v[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                all[i] += v[i];
                front[i] += t < here ? v[i] : 0;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            atomicAdd(&s_all[4 * q + i], all[i]);
            atomicAdd(&s_front[4 * q + i], front[i]);
        }
    }
    __syncthreads();
    exclusive_sums<NT>(s_all, a.E + 1, s_sum);
    if (blockIdx.x == 0)
        for (int e = tid; e <= a.E; e += NT) a.offsets[e] = e < a.E ? s_all[e] : (int)slots;
    for (int e = tid; e <= a.E; e += NT) {
        int next = s_all[e] + s_front[e], c[NW];
#pragma unroll
        for (int w = 0; w < NW; ++w) c[w] = s_at[w][e];
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            s_at[w][e] = next;
            next += c[w];
        }
    }
    __syncthreads();
    for (int64_t i0 = lo; i0 < hi; i0 += 64) {
        const int64_t i = i0 + lane;
        const bool live = i < hi;
        const int key = i0 == lo ? key0 : live ? key_of(a, a.expert[i]) : 0;
        const float w = i0 == lo ? w0 : live ? a.weight[i] : 0.f;
        const uint64_t peers = same_key(key, __ballot(live));
        const int before = lanes_before(peers);
        if (live) place(a, s_at[wave][key] + before, i, key, w);
        wave_lds_order();
        if (live && before == 0) s_at[wave][key] += __builtin_popcountll(peers);
        wave_lds_order();
    }
}

// All of it for few tokens: at most 64 slots a wave.
template <int NV>
__global__ __launch_bounds__(64 * many_waves(NV)) void route_small(const fqm_routing a) {
    constexpr int NW = many_waves(NV), NT = 64 * NW;
    __shared__ WaveLds<NV> s_wave[NW];
    __shared__ uint16_t s_at[NW][64 * NV + 2];  // a wave's slots of each expert, then those of the waves in front
    __shared__ int s_n[64 * NV + 1], s_sum[NW];
    __shared__ int s_key[NT];
    __shared__ float s_w[NT];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int slots = (int)a.T * a.k, waves = (slots + 63) / 64;
    for (int e = lane; e <= a.E; e += 64) s_at[wave][e] = 0;
    choose_all<NV, NW>(a, 0, a.T, &s_wave[wave], [&](int64_t t, int expert, float weight) {
        const int i = (int)t * a.k + lane;
        a.expert[i] = expert;
        a.weight[i] = weight;
        s_key[i] = key_of(a, expert);
        s_w[i] = weight;
    });
    __syncthreads();
    const bool live = tid < slots;
    const int key = live ? s_key[tid] : 0;
    const uint64_t peers = same_key(key, __ballot(live));
    const int before = lanes_before(peers);
    if (live && before == 0) s_at[wave][key] = (uint16_t)__builtin_popcountll(peers);
    __syncthreads();
    for (int e = tid; e <= a.E; e += NT) {
        int n = 0;
        for (int w = 0; w < waves; ++w) {
            const int c = s_at[w][e];
            s_at[w][e] = (uint16_t)n;
            n += c;
        }
        s_n[e] = n;
    }
    __syncthreads();
    exclusive_sums<NT>(s_n, a.E + 1, s_sum);
    for (int e = tid; e <= a.E; e += NT) a.offsets[e] = e < a.E ? s_n[e] : slots;
    if (live) place(a, s_n[key] + s_at[wave][key] + before, tid, key, s_w[tid]);
}

struct Tiles {
    int64_t tile, n;  // tokens, tiles
};
Tiles tiles_of(const fqm_routing& a) {
    const int64_t most = a.E <= 256 ? kMostTiles : kMostTiles / 2;  // up to 256 experts two workgroups fit a compute unit
    const int64_t tile = std::max<int64_t>(1, (a.T + kFewWaves * most - 1) / (kFewWaves * most)) * kFewWaves;
    return {tile, (a.T + tile - 1) / tile};
}
bool small(const fqm_routing& a) { return a.offsets && a.T <= kSmallTokens; }  // up to 64 * 8 slots

template <int NV>
hipError_t launch_nv(const fqm_routing& a, int* hist, hipStream_t s) {
    constexpr int MW = many_waves(NV);
    if (small(a)) {
        hipLaunchKernelGGL(route_small<NV>, dim3(1), dim3(64 * MW), 0, s, a);
        return hipGetLastError();
    }
    const Tiles t = tiles_of(a);
    // 8192 tokens of 256 experts 39 us with 4 waves, 31 with 12; 48 tokens 13.5 with 4
    if (t.tile >= MW) hipLaunchKernelGGL((route_choose<NV, MW>), dim3((unsigned)t.n), dim3(64 * MW), 0, s, a, (int)t.tile, hist);
    else hipLaunchKernelGGL((route_choose<NV, kFewWaves>), dim3((unsigned)t.n), dim3(64 * kFewWaves), 0, s, a, (int)t.tile, hist);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.offsets) return e;
    const int span = (int)std::max<int64_t>(1, 64 * kPlaceWaves / (t.tile * a.k));
    hipLaunchKernelGGL(route_place, dim3((unsigned)((t.n + span - 1) / span)), dim3(64 * kPlaceWaves), 0, s, a, hist, (int)t.tile, (int)t.n,
                       span);
    return hipGetLastError();
}

}  // namespace

size_t route_workspace(const fqm_routing& a) {
    if (!a.offsets || small(a)) return 0;
    return (size_t)tiles_of(a).n * counts_of(a.E) * 4;
}

hipError_t launch_route(const fqm_routing& a, void* ws, hipStream_t s) {
    int* hist = a.offsets ? static_cast<int*>(ws) : nullptr;
    if (a.E <= 64) return launch_nv<1>(a, hist, s);
    if (a.E <= 128) return launch_nv<2>(a, hist, s);
    if (a.E <= 256) return launch_nv<4>(a, hist, s);
    if (a.E <= 512) return launch_nv<8>(a, hist, s);
    return launch_nv<16>(a, hist, s);
}

}  // namespace fqm
