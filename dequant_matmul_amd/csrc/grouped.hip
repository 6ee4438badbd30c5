// Products grouped by expert, weights in the per-row table formats:
//   Y[dst[i]] = row_scale[i] * (W_e X[src[i]]) for the rows i of group e,
// W_e the e-th of `count` equal matrices stacked in one descriptor.
//
// The group sizes are on the device and the host never waits for them: grids
// are sized for the most work that M rows in `count` groups can make, and each
// workgroup finds its own piece in the offsets (one wave scan).
//
// Two kernels, by the rows a group has on average (M / count):
//  - few: grouped_rows_kernel, waves that own rows of W, every weight decoded
//    once for up to four rows of X (reading the codes is what costs);
//  - more: grouped_tile_kernel, tiles of X rows times W rows on the matrix
//    cores, the tile of the ungrouped GEMM (lut_gemm_tile.h).
// Both handle any group size; the choice is about speed alone.
//
// What binds it, on one MI355X.  Few rows (8 of 64 groups with one row each,
// 6-bit 5120 -> 1024): 14.7 us for 32 MB, 2.2 TB/s; the launch, the search of
// the offsets and a table's load stand before a stream of 4 MB a group.  Tiles
// of 32 rows (96 rows in 32 groups, 4-bit 1024 -> 5120): 29 us for 88 MB, 3.0
// TB/s; of 128 rows (16384 rows in 64 groups, 6-bit 5120 -> 1024): 265-315 us,
// 545-650 TFLOP/s.  No unit of the tiles is busy (LDS 24-37 % of the time, VALU
// 20-42 %, matrix cores 10-24 %), the waves wait 26-48 % of theirs; X three to
// five steps ahead instead of two was 0-15 % slower, though.
#include <algorithm>

#include "fqm_layer.h"
#include "lut_gemm_tile.h"

namespace fqm {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// What every workgroup needs of a call.
struct Grouped {
    fqm_groups g;
    const uint8_t* packed;
    int64_t ld;
    const uint16_t* lut;
    int N, K;  // rows and columns of one matrix
};

__device__ __forceinline__ int clamp_row(int v, int64_t M) { return max(0, min(v, (int)M)); }

// The rows [lo, hi) of group e.
__device__ __forceinline__ void group_rows(const fqm_groups& g, int e, int* lo, int* hi) {
    *lo = clamp_row(g.offsets[e], g.M);
    *hi = clamp_row(g.offsets[e + 1], g.M);
}

// The u-th of the groups that have rows (-1: there are not as many).  Every
// lane gets the same answer; a wave looks at 64 groups a time.
__device__ __forceinline__ int find_group(const fqm_groups& g, int u) {
    const int lane = threadIdx.x & 63;
    for (int e0 = 0; e0 < g.count; e0 += 64) {
        bool has = false;
        if (e0 + lane < g.count) {
            int lo, hi;
            group_rows(g, e0 + lane, &lo, &hi);
            has = hi > lo;
        }
        const uint64_t live = __ballot(has);
        const int before = __builtin_amdgcn_mbcnt_hi((uint32_t)(live >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)live, 0u));
        const uint64_t it = __ballot(has && before == u);
        if (it) return e0 + __builtin_ctzll(it);
        u -= __builtin_popcountll(live);
    }
    return -1;
}

// The pieces of a group of m rows: whole ones of BM rows and, of what is left,
// one of at most BM / 4, BM / 2 or BM rows.  All groups' pieces of class 0
// (BM) come first, then those of class 1 (BM / 2) and 2 (BM / 4): the longest
// work starts first, the shortest fills the end.
__device__ __forceinline__ int pieces_of(int m, int bm, int cls) {
    const int left = m & (bm - 1);  // bm is a power of two
    if (cls == 0) return m / bm + (left > bm / 2);
    if (cls == 1) return left > bm / 4 && left <= bm / 2;
    return left > 0 && left <= bm / 4;
}

// The u-th piece of all: its group (-1: there are not as many), first row and class.
__device__ __forceinline__ int find_piece(const fqm_groups& g, int u, int bm, int* first, int* cls) {
    const int lane = threadIdx.x & 63;
    for (int c = 0; c < 3; ++c)
        for (int e0 = 0; e0 < g.count; e0 += 64) {
            int lo = 0, hi = 0;
            if (e0 + lane < g.count) group_rows(g, e0 + lane, &lo, &hi);
            const int n = pieces_of(max(0, hi - lo), bm, c);
            int upto = n;  // inclusive sum over the lanes
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int t = __shfl_up(upto, o, 64);
                if (lane >= o) upto += t;
            }
            const uint64_t past = __ballot(upto > u);
            if (past) {
                const int l = __builtin_ctzll(past);
                const int at = c == 0 ? (u - __builtin_amdgcn_readlane(upto - n, l)) * bm
                                      : __builtin_amdgcn_readlane(hi - lo, l) & ~(bm - 1);
                *first = __builtin_amdgcn_readlane(lo, l) + at;
                *cls = c;
                return e0 + l;
            }
            u -= __builtin_amdgcn_readlane(upto, 63);
        }
    return -1;
}

__device__ __forceinline__ void store_y(const fqm_groups& g, int64_t at, float v) {
    if (g.y_dtype == FQM_F32) static_cast<float*>(g.Y)[at] = v;
    else static_cast<uint16_t*>(g.Y)[at] = __builtin_bit_cast(uint16_t, (__bf16)v);
}

// Grouped row i's row of X (-1: a row of zeros), row of Y (-1: not stored) and factor.
__device__ __forceinline__ int x_row(const fqm_groups& g, int i) {
    const int r = g.src ? g.src[i] : i;
    return r >= 0 && r < g.x_rows ? r : -1;
}
__device__ __forceinline__ int y_row(const fqm_groups& g, int i) {
    const int r = g.dst ? g.dst[i] : i;
    return r >= 0 && r < g.y_rows ? r : -1;
}
__device__ __forceinline__ float row_factor(const fqm_groups& g, int i, int xr) {
    float f = g.row_scale ? g.row_scale[i] : 1.f;
    if (g.x_scale && xr >= 0) f *= g.x_scale[xr];
    return f;
}

// Two 8-bit values (the low 16 bits) as a bf16 pair, exact.
__device__ __forceinline__ uint32_t bf16_pair_of_i8(uint32_t two) {
    const float f0 = (float)(int8_t)(two & 255), f1 = (float)(int8_t)((two >> 8) & 255);
    return __float_as_uint(f0) >> 16 | (__float_as_uint(f1) & 0xFFFF0000u);
}

// ---- few rows per group --------------------------------------------------------
// A wave owns a row of W, each lane pieces of 16 codes (2 BITS bytes): piece
// 64 c + lane of chunk c, so a load of the wave covers the chunk's bytes in
// order.  Codes are requested kAhead chunks ahead, the first of them before X
// is staged.  A weight's table entry is gathered from LDS (one table per
// wave: no bank conflicts), paired, and meets the pair of every row of X in
// v_dot2_f32_bf16 (fp32 accumulate).
constexpr int kRowWaves = 8;
constexpr int kMaxB = 4;                 // rows of X per pass
constexpr int kMaxR = 4;                 // rows of W per wave
constexpr int kAhead = 4;
constexpr int kChunk = 1024;             // columns per chunk: a piece for every lane
constexpr int64_t kRowsLds = 60 * 1024;  // of X in LDS: two workgroups and more per CU

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) u32x4_t lds_u4;
typedef __attribute__((address_space(3))) const u32x4_t lds_u4c;
typedef __attribute__((address_space(3))) const uint16_t lds_u16c;

// Code J of a piece moved to bits 1 .. BITS (the byte offset of its table
// entry), other bits still to be masked.
template <int BITS, int J>
__device__ __forceinline__ uint32_t code_x2(const uint32_t* d) {
    constexpr int bit = BITS * J, w = bit >> 5, o = bit & 31;
    if constexpr (o == 0) return d[w] << 1;
    else if constexpr (o + BITS <= 32) return d[w] >> (o - 1);
    else return __builtin_amdgcn_alignbit(d[w + 1], d[w], o - 1);
}

template <int BITS, int J = 0>
__device__ __forceinline__ void gather_pairs(const uint32_t* d, uint32_t mask, uint32_t tab, uint32_t (&w)[8]) {
    if constexpr (J < 8) {
        const uint32_t lo = (code_x2<BITS, 2 * J>(d) & mask) | tab, hi = (code_x2<BITS, 2 * J + 1>(d) & mask) | tab;
        w[J] = __builtin_amdgcn_perm(*(lds_u16c*)(uintptr_t)hi, *(lds_u16c*)(uintptr_t)lo, 0x05040100u);
        gather_pairs<BITS, J + 1>(d, mask, tab, w);
    }
}

__device__ __forceinline__ float dot2(uint32_t w, uint32_t x, float acc) {
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w), __builtin_bit_cast(bf16x2, x), acc, false);
}

// This lane's piece of chunk c of a row (past the row's end: its last one).
template <int BITS>
__device__ __forceinline__ void load_piece(const uint8_t* prow, int c, int pieces, uint32_t (&d)[BITS / 2]) {
    const int p = min(64 * c + (int)(threadIdx.x & 63), pieces - 1);
    const uint32_t* q = reinterpret_cast<const uint32_t*>(prow + 2 * BITS * p);
#pragma unroll
    for (int i = 0; i < BITS / 2; ++i) d[i] = __builtin_nontemporal_load(q + i);
}

// This wave's rows of W: the r-th of R is row first + kRowWaves r of the matrix
// (rows past the end repeat the last one; they are not stored).
struct RowsOfW {
    const uint8_t* packed;
    int64_t ld;
    int first, last;
    __device__ __forceinline__ int number(int r) const { return first + kRowWaves * r; }
    __device__ __forceinline__ const uint8_t* row(int r) const { return packed + (int64_t)min(number(r), last) * ld; }
};

// B rows of X in LDS (bytes `stride` apart) against the wave's R rows of W, the
// sums to s_sum[r][b].  The codes of (row, chunk) come kAhead steps ahead,
// across the rows' ends; cr holds the first ones.  Every load is
// unconditional (past the end it repeats the last step's) and nothing else in
// the loop touches global memory, so that a wait is for one step's codes.
template <int BITS, int B>
__device__ __forceinline__ void dot_rows(const RowsOfW& W, int R, uint32_t tab, uint32_t xs, uint32_t stride, int pieces,
                                         uint32_t (&cr)[kAhead][BITS / 2], float (*s_sum)[kMaxB]) {
    const int lane = threadIdx.x & 63, chunks = (pieces + 63) / 64, steps = R * chunks;
    uint32_t mask = (uint32_t)((1 << BITS) - 1) << 1;
    asm volatile("" : "+v"(mask));  // in a VGPR: (code & mask) | tab is one v_and_or_b32
    float acc0[B], acc1[B];
#pragma unroll
    for (int b = 0; b < B; ++b) acc0[b] = acc1[b] = 0.f;
    int c = 0, r = 0;                                                                        // this step's chunk and row
    int cn = min(kAhead, steps - 1) % chunks, rn = min(kAhead, steps - 1) / chunks;  // those of the loads
    for (int s0 = 0; s0 < steps; s0 += kAhead) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            uint32_t d[BITS / 2];
#pragma unroll
            for (int i = 0; i < BITS / 2; ++i) d[i] = cr[u][i];
            load_piece<BITS>(W.row(rn), cn, pieces, cr[u]);
            if (s0 + u + kAhead + 1 < steps && ++cn == chunks) cn = 0, ++rn;
            if (s0 + u < steps) {
                if (64 * c + lane < pieces) {
                    uint32_t w[8];
                    gather_pairs<BITS>(d, mask, tab + 128u * r, w);
#pragma unroll
                    for (int b = 0; b < B; ++b) {
                        const uint32_t at = xs + stride * b + 2048u * c + 16u * lane;
                        const u32x4_t xl = *(lds_u4c*)(uintptr_t)at, xh = *(lds_u4c*)(uintptr_t)(at + 1024u);
                        const uint32_t xv[8] = {xl[0], xl[1], xl[2], xl[3], xh[0], xh[1], xh[2], xh[3]};
#pragma unroll
                        for (int j = 0; j < 8; j += 2) {
                            acc0[b] = dot2(w[j], xv[j], acc0[b]);
                            acc1[b] = dot2(w[j + 1], xv[j + 1], acc1[b]);
                        }
                    }
                }
                if (++c == chunks) {
#pragma unroll
                    for (int b = 0; b < B; ++b) {
                        const float sum = wave_sum_lane63(acc0[b] + acc1[b]);
                        if (lane == 63) s_sum[r][b] = sum;
                        acc0[b] = acc1[b] = 0.f;
                    }
                    c = 0, ++r;
                }
            }
        }
    }
}

// 8 values of a row of X from column k on as bf16 pairs (8-bit values: exact).
__device__ __forceinline__ u32x4_t load_x8(const fqm_groups& g, int64_t at) {
    if (g.x_dtype != FQM_I8) return *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(g.X) + at);
    const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const int8_t*>(g.X) + at);
    u32x4_t o;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = bf16_pair_of_i8((j < 2 ? q.x : q.y) >> (16 * (j & 1)));
    return o;
}

// Workgroup (slot, row block): the slot-th group that has rows, kRowWaves R
// rows of its W, all its rows of X in passes of up to `bmax`.
template <int BITS>
__global__ __launch_bounds__(64 * kRowWaves) void grouped_rows_kernel(const Grouped a, int row_blocks, int bmax, int R) {
    constexpr int ENTRIES = 1 << BITS, NT = 64 * kRowWaves;
    extern __shared__ __attribute__((aligned(16))) uint8_t s_x[];
    __shared__ __attribute__((aligned(128))) uint16_t s_tab[kRowWaves][kMaxR][64];
    __shared__ float s_sum[kRowWaves][kMaxR][kMaxB];
    const fqm_groups& g = a.g;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int slot = blockIdx.x / row_blocks, nb = blockIdx.x - slot * row_blocks;
    const int e = find_group(g, slot);
    if (e < 0) return;
    int lo, hi;
    group_rows(g, e, &lo, &hi);
    const int pieces = a.K / 16, chunks = (pieces + 63) / 64;
    const RowsOfW W = {a.packed + (int64_t)e * a.N * a.ld, a.ld, nb * kRowWaves * R + wave, a.N - 1};
    const uint32_t stride = (uint32_t)(a.K + kChunk - 1) / kChunk * (2 * kChunk);
    const uint32_t xs = (uint32_t)(uintptr_t)(lds8*)s_x;
    const uint32_t tab = (uint32_t)(uintptr_t)(lds8*)s_tab + 128u * kMaxR * wave;
    for (int i0 = lo; i0 < hi; i0 += bmax) {
        const int nrows = min(bmax, hi - i0);
        int xr[kMaxB];
#pragma unroll
        for (int b = 0; b < kMaxB; ++b) xr[b] = b < nrows ? x_row(g, i0 + b) : -1;
        if (i0 == lo && lane < ENTRIES) {
            for (int r = 0; r < R; ++r)
                s_tab[wave][r][lane] = a.lut[((int64_t)e * a.N + min(W.number(r), a.N - 1)) * ENTRIES + lane];
        }
        lds_barrier();  // the last pass is done with s_x
        // 16-byte unit u = 128 c + 2 l + h of a row goes to slot 128 c + 64 h + l: a wave's reads are dense.  The
        // first codes are requested behind the last of X's loads, and only the latter are waited for.
        uint32_t cr[kAhead][BITS / 2];
        for (int u0 = 0; u0 < a.K / 8; u0 += NT) {
            const int u = u0 + tid, units = a.K / 8;
            u32x4_t v[kMaxB];
#pragma unroll
            for (int b = 0; b < kMaxB; ++b) {
                v[b] = u32x4_t{0u, 0u, 0u, 0u};
                if (u < units && xr[b] >= 0) v[b] = load_x8(g, (int64_t)xr[b] * a.K + 8 * u);
            }
            if (u0 + NT >= units) {
#pragma unroll
                for (int s = 0; s < kAhead; ++s) load_piece<BITS>(W.row(min(s / chunks, R - 1)), s % chunks, pieces, cr[s]);
            }
            const int slot16 = (u & ~127) | (u & 1) << 6 | ((u >> 1) & 63);
#pragma unroll
            for (int b = 0; b < kMaxB; ++b)
                if (u < units && b < nrows) *(lds_u4*)(uintptr_t)(xs + stride * b + 16u * slot16) = v[b];
        }
        lds_barrier();
        if (pieces == 0) {  // sums of nothing
            if (lane < kMaxR * kMaxB) s_sum[wave][lane / kMaxB][lane % kMaxB] = 0.f;
        } else if (nrows == 1) dot_rows<BITS, 1>(W, R, tab, xs, stride, pieces, cr, s_sum[wave]);
        else if (nrows == 2) dot_rows<BITS, 2>(W, R, tab, xs, stride, pieces, cr, s_sum[wave]);
        else if (nrows == 3) dot_rows<BITS, 3>(W, R, tab, xs, stride, pieces, cr, s_sum[wave]);
        else dot_rows<BITS, 4>(W, R, tab, xs, stride, pieces, cr, s_sum[wave]);
        wave_lds_order();
        // lane (r, b) of the wave stores row r of W, row b of X
        const int b = lane % kMaxB, r = lane / kMaxB;
        if (r < R && b < nrows) {
            const int i = i0 + b, n = W.number(r), yr = y_row(g, i);
            const int from = x_row(g, i);
            const bool none = from < 0 || pieces == 0;  // zeros, whatever the factors and tables hold
            if (n < a.N && yr >= 0) store_y(g, (int64_t)yr * a.N + n, none ? 0.f : s_sum[wave][r][b] * row_factor(g, i, from));
        }
    }
}

// ---- tiles --------------------------------------------------------------------------
// 8-bit rows of X as bf16 (exact), 16 values a thread.
__global__ __launch_bounds__(256) void widen_rows(const uint4* __restrict__ x, uint4* __restrict__ out, int64_t n16) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n16) return;
    const uint4 v = x[i];
    const uint32_t q[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        o[j] = bf16_pair_of_i8(q[j >> 1] >> (16 * (j & 1)));
    }
    out[2 * i] = uint4{o[0], o[1], o[2], o[3]};
    out[2 * i + 1] = uint4{o[4], o[5], o[6], o[7]};
}

// Tile rows [0, rows) are the grouped rows from lo on; the tile is BM rows
// high and takes the K steps [t0, t0 + steps).  part: the fp32 sums go there,
// [M][N], as they are; NULL: to Y.
template <int BITS, int BM, int NW>
__device__ __forceinline__ void grouped_tile(lds8* tab, lds8* x0, lds8* x1, lds8* x2, const Grouped& a,
                                             const uint16_t* xb, int e, int lo, int rows, int n0, int t0, int steps,
                                             float* part) {
    const fqm_groups& g = a.g;
    // rows without a row of X read X's row 0
    const uint16_t* X = g.src ? xb : xb + (int64_t)lo * a.K;
    auto x_off = [&](int r) {
        const int rr = min(r, rows - 1);
        return (uint32_t)(g.src ? max(0, x_row(g, lo + rr)) : rr) * (uint32_t)a.K * 2u;
    };
    typedef __attribute__((address_space(3))) int ldsi;
    typedef __attribute__((address_space(3))) float ldsf;
    ldsi* s_dst = (ldsi*)x0;
    ldsf* s_f = (ldsf*)(x0 + 4 * BM);
    // each row's place in Y (-1: none; -2 - place: zeros, whatever was multiplied) and factor
    auto before = [&](lds8*) {
        for (int r = threadIdx.x; r < BM; r += 64 * NW) {
            int yr = -1;
            float f = 0.f;
            if (r < rows) {
                const int xr = x_row(g, lo + r);
                yr = y_row(g, lo + r);
                f = row_factor(g, lo + r, xr);
                if (xr < 0 && yr >= 0) yr = -2 - yr;
            }
            s_dst[r] = yr;
            s_f[r] = f;
        }
    };
    const int64_t w0 = (int64_t)e * a.N;
    gemm_tile<BITS, BM, NW>(tab, x0, x1, x2, X, 0, x_off, a.packed + w0 * a.ld, a.ld, a.lut + (w0 << BITS),
                            RunOfRows{a.N, n0}, t0,
                            steps,
                            [&](int row, int col, float v) {
                                const int n = n0 + col;
                                if (n >= a.N) return;
                                if (part) {
                                    if (row < rows) part[(int64_t)(lo + row) * a.N + n] = v;
                                    return;
                                }
                                const int yr = s_dst[row];
                                if (yr >= 0) store_y(g, (int64_t)yr * a.N + n, v * s_f[row]);
                                else if (yr != -1) store_y(g, (int64_t)(-2 - yr) * a.N + n, 0.f);
                            },
                            before);
}

// Workgroup (piece u, block of 32 NW rows of its W, K part): the workgroups of a
// piece are 8 apart, they share an XCD and its X rows in that L2.  Short
// pieces take lower tiles.
template <int BITS, int BM, int NW, int CLASSES>
__global__ __launch_bounds__(64 * NW) void grouped_tile_kernel(const Grouped a, const uint16_t* xb, int ntiles,
                                                               int ksplit, int apart, float* part) {
    FQM_GEMM_TILE_LDS(BITS, BM, NW);
    const int b = blockIdx.x, per = ntiles * ksplit;
    const int j = apart ? b >> 3 : b, in = j % per;
    const int u = apart ? (j / per) * 8 + (b & 7) : j / per, n0 = in / ksplit * (32 * NW), ks = in % ksplit;
    int first, cls;
    const int e = find_piece(a.g, u, BM, &first, &cls);
    if (e < 0) return;  // the whole workgroup
    int lo, hi;
    group_rows(a.g, e, &lo, &hi);
    const int rows = min(BM, hi - first), ksteps = a.K / BK;
    const int t0 = ks * ksteps / ksplit, steps = (ks + 1) * ksteps / ksplit - t0;
    if (ksplit > 1) part += (int64_t)ks * a.g.M * a.N;
    if constexpr (CLASSES > 2) {
        if (cls == 2) {
            grouped_tile<BITS, BM / 4, NW>(FQM_GEMM_TILE_LDS_ARGS, a, xb, e, first, rows, n0, t0, steps, part);
            return;
        }
    }
    if constexpr (CLASSES > 1) {
        if (cls >= 1) {
            grouped_tile<BITS, BM / 2, NW>(FQM_GEMM_TILE_LDS_ARGS, a, xb, e, first, rows, n0, t0, steps, part);
            return;
        }
    }
    grouped_tile<BITS, BM, NW>(FQM_GEMM_TILE_LDS_ARGS, a, xb, e, first, rows, n0, t0, steps, part);
}

// Y from the K parts, added in order.  Workgroup (grouped row, 1024 columns of it).
__global__ __launch_bounds__(256) void grouped_split_sum(const Grouped a, const float* __restrict__ part, int blocks,
                                                         int ksplit) {
    const fqm_groups& g = a.g;
    const int i = blockIdx.x / blocks, n0 = (blockIdx.x - i * blocks) * 1024 + threadIdx.x;
    const int64_t all = g.M * a.N;
    const float* p = part + (int64_t)i * a.N;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < ksplit; ++k)
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (n0 + 256 * c < a.N) v[c] += p[k * all + n0 + 256 * c];
    const int xr = x_row(g, i), yr = y_row(g, i);
    const float f = row_factor(g, i, xr);
    // only rows of some group have parts
    bool mine = false;
    for (int e = threadIdx.x & 63; e < g.count; e += 64) {
        int lo, hi;
        group_rows(g, e, &lo, &hi);
        mine |= lo <= i && i < hi;
    }
    if (!__ballot(mine) || yr < 0) return;
#pragma unroll
    for (int c = 0; c < 4; ++c)
        if (n0 + 256 * c < a.N) store_y(g, (int64_t)yr * a.N + n0 + 256 * c, xr < 0 ? 0.f : v[c] * f);
}

struct TilePlan {
    int bm;               // rows of X per tile: 32, 64 or 128
    int ntiles;           // blocks of 32 kTileWaves rows of W
    int ksplit;           // K parts of a tile
    int64_t pieces;       // at most
    bool apart;           // a piece's workgroups on one XCD
    size_t part_bytes;
};

// Heights by the rows M / count a group has on average (one MI355X, us with
// heights 32 / 64 / 128): 64 groups of 6-bit 5120 -> 1024 at 8 rows 81 / 88 / -,
// 16 rows 114 / 90 / 100, 64 rows 186 / 167 / 158, 256 rows 517 / 377 / 300;
// 8 groups of 4-bit 5120 -> 2176 at 8 rows 28 / 29 / -, 32 rows 35 / 31 / 46,
// 96 rows 57 / 50 / 55, 256 rows 116 / 88 / 84.  At its borders the rule costs up
// to 10 %.  256-row tiles (one workgroup
// per CU, as the ungrouped product has them) were 0-9 % faster on large even
// 6-bit groups, 5-40 % slower on ragged and 4-bit ones, and are not built.
// Splitting K fills the chip when the tiles are few: aimed at 768 workgroups
// of at least 8 steps (8 groups of 4-bit 5120 -> 2176 at 1 row 38 -> 24 us, at 8
// rows 38 -> 28; aiming at 1280 was 0-20 % slower).
// With 64 pieces and more, a piece's workgroups go to one XCD, whose L2 then
// holds its X rows (64 groups, 256 rows: 323 -> 304 us); with fewer the XCDs
// would be loaded unevenly (8 groups, 192 rows: 64 -> 82 us).
constexpr int kTileWaves = 4;
TilePlan tile_plan(const fqm_groups& g, int64_t N, int64_t K) {
    TilePlan p;
    const int64_t avg = g.M / g.count;
    p.bm = avg >= 96 ? 128 : avg >= 16 ? 64 : 32;
    p.ntiles = (int)((N + 32 * kTileWaves - 1) / (32 * kTileWaves));
    // a group of m rows makes ceil(m / bm) pieces: at most M / bm + min(count, M) in all
    const int64_t pieces = g.M / p.bm + std::min<int64_t>(g.count, g.M);
    p.apart = pieces >= 64;
    p.pieces = p.apart ? (pieces + 7) / 8 * 8 : pieces;
    const int64_t parts = std::min<int64_t>({768 / std::max<int64_t>(pieces * p.ntiles, 1), K / BK / 8, (int64_t)8});
    p.ksplit = (int)std::max<int64_t>(parts, 1);
    p.part_bytes = p.ksplit > 1 ? (size_t)p.ksplit * g.M * N * 4 : 0;
    return p;
}

template <int BITS, int BM, int CLASSES>
hipError_t launch_tiles(const Grouped& a, const uint16_t* xb, float* part, const TilePlan& p, hipStream_t s) {
    const int64_t grid = p.pieces * p.ntiles * p.ksplit;
    if (grid > 0x7fffffff) return hipErrorInvalidValue;
    hipLaunchKernelGGL((grouped_tile_kernel<BITS, BM, kTileWaves, CLASSES>), dim3((unsigned)grid), dim3(64 * kTileWaves), 0, s, a, xb,
                       p.ntiles, p.ksplit, p.apart, p.ksplit > 1 ? part : nullptr);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.ksplit == 1) return e;
    const int blocks = (a.N + 1023) / 1024;
    if (a.g.M * blocks > 0x7fffffff) return hipErrorInvalidValue;
    hipLaunchKernelGGL(grouped_split_sum, dim3((unsigned)(a.g.M * blocks)), dim3(256), 0, s, a, part, blocks, p.ksplit);
    return hipGetLastError();
}

// The widened copy of 8-bit rows, where the tiles read them.
size_t widened_bytes(const fqm_groups& g, int64_t K) { return g.x_dtype == FQM_I8 ? (size_t)g.x_rows * (size_t)K * 2 : 0; }

// Rows of X that fit the LDS of the few-rows kernel; 0: none.
int64_t rows_x_bytes(int64_t K) { return (K + kChunk - 1) / kChunk * (2 * kChunk); }
int rows_bmax(int64_t K) { return K == 0 ? kMaxB : (int)std::min<int64_t>(kMaxB, kRowsLds / rows_x_bytes(K)); }

// The few-rows kernel up to K / 4096 rows a group on average.  Measured on one
// MI355X, us against the tiles (with their K parts): 64 groups of 6-bit
// 5120 -> 1024 at 1/8 row 14 / 27, 1/2 row 32 / 42, 1 row 55 / 49, 2 rows 87 /
// 76; 8 groups of 4096 -> 4096 at 1/2 row 14 / 23, 1 row 20 / 26, 2 rows 41 / 32;
// 40 groups of 2048 -> 1000 at 1/2 row 16 / 21, 1 row 23 / 22; 32 groups of 4-bit
// 1024 -> 5120 at 1/8 row 11 / 13, 1/4 row 16 / 14, 1/2 row 29 / 17.  At its border
// the rule costs up to 14 %.
bool rows_path(const fqm_groups& g, int64_t K) {
    return K == 0 || (g.M * 4096 <= g.count * K && rows_bmax(K) >= 1);
}

// Rows of W per wave of it: as many as leave 512 workgroups, so that a
// workgroup's X and its start are shared (8 groups of 6-bit 5120 -> 1024, us
// with 1 / 2 / 4: 18.5 / 14.0 / 15.3; 16 groups 30.5 / 24.2 / 21.1; 1 group 7.7 /
// 9.2 / 13.1).
int rows_per_wave(int64_t groups, int64_t N) {
    const int64_t r = groups * N / (512 * kRowWaves);
    return r >= 4 ? 4 : r >= 2 ? 2 : 1;
}

template <int BITS>
hipError_t launch_bits(const Grouped& a, void* ws, hipStream_t s) {
    const fqm_groups& g = a.g;
    if (rows_path(g, a.K)) {
        const int bmax = rows_bmax(a.K);
        const int64_t groups = std::min<int64_t>(g.count, g.M);
        const int R = rows_per_wave(groups, a.N);
        const int row_blocks = (a.N + kRowWaves * R - 1) / (kRowWaves * R);
        const int64_t grid = groups * row_blocks;
        if (grid > 0x7fffffff) return hipErrorInvalidValue;
        hipLaunchKernelGGL(grouped_rows_kernel<BITS>, dim3((unsigned)grid), dim3(64 * kRowWaves), (size_t)(bmax * rows_x_bytes(a.K)), s,
                           a, row_blocks, bmax, R);
        return hipGetLastError();
    }
    const uint16_t* xb = static_cast<const uint16_t*>(g.X);
    if (g.x_dtype == FQM_I8) {
        const int64_t n16 = g.x_rows * a.K / 16;
        xb = static_cast<const uint16_t*>(ws);
        if (n16 > 0) {
            hipLaunchKernelGGL(widen_rows, dim3((unsigned)((n16 + 255) / 256)), dim3(256), 0, s,
                               static_cast<const uint4*>(g.X), static_cast<uint4*>(ws), n16);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    }
    const TilePlan p = tile_plan(g, a.N, a.K);
    float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + widened_bytes(g, a.K));
    if (p.bm == 32) return launch_tiles<BITS, 32, 1>(a, xb, part, p, s);
    if (p.bm == 64) return launch_tiles<BITS, 64, 2>(a, xb, part, p, s);
    return launch_tiles<BITS, 128, 3>(a, xb, part, p, s);
}

}  // namespace

size_t grouped_workspace(const fqm_weights& w, const fqm_groups& g) {
    const int64_t K = g.x_rows == 0 ? 0 : w.cols;
    if (rows_path(g, K)) return 0;
    return widened_bytes(g, K) + tile_plan(g, w.rows / g.count, K).part_bytes;
}

hipError_t launch_grouped(const fqm_weights& w, const fqm_groups& g, void* ws, hipStream_t s) {
    Grouped a;
    a.g = g;
    a.N = (int)(w.rows / g.count);
    a.K = g.x_rows == 0 ? 0 : (int)w.cols;  // without rows of X: sums of nothing (the tiles read at least one row)
    const bool six = w.format == FQM_LUT6;
    a.packed = six ? w.lut6.packed : w.lut4.packed;
    a.ld = six ? w.lut6.ld : w.lut4.ld;
    a.lut = six ? w.lut6.lut : w.lut4.lut;
    return six ? launch_bits<6>(a, ws, s) : launch_bits<4>(a, ws, s);
}

}  // namespace fqm
