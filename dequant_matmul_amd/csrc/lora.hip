// Low-rank adapters of many requests beside one projection:
//   y[m] = base[m] + scale[i] * B_i (A_i x[m]),  i = index[m].
//
// Two launches: t = A_i x in fp32 into the workspace (K in parts), then the
// parts' sum, scaled, through B_i onto base.  Rows of one adapter need not lie
// together.  With few rows each job collects the rows of one adapter from the
// whole batch; with many (prompts: long runs) a block of 64 rows goes through
// its distinct adapters one after the other.  Rows are columns of the matrix
// products, so a row that is not finite, or another request's adapter,
// touches no other row.
//
// What binds it, on one MI355X: many rows - the second launch's loads and their
// latency (4096 rows, 16 adapters of rank 64, 5120 -> 17408 in bf16: 28 us for the
// first launch, 130-136 us for the second, 151 us among other calls, 373 MB at
// 2.5 TB/s; rank 16 91 us, rank 128 182; 17408 -> 5120 of rank 64 106 us).  It
// reads 308 MB for 180 that it cannot do without: every range of outputs sums the
// K parts of t again, and a block's B comes to several XCDs; from rank 33 on two
// workgroups share a CU, not three.  Few rows - two launches and the latency of
// the loads in them (1 row, rank 16, 5120 -> 17408: 4.2 + 7.2 us; 48 rows over 32
// adapters, 17408 -> 5120: 12.6 + 7.0 us for 29 MB).
#include <algorithm>

#include "fqm_layer.h"
#include "lut_gemm_tile.h"

namespace fqm {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));

constexpr int kWaves = 4;

// The call's arguments.
struct Lora {
    fqm_adapters a;
    const uint16_t* x;
    const int32_t* index;
    const void* base;
    void* y;
    int y_f32;
    int64_t M;
    float* part;  // [ksplit][M][ldt]
    int ldt;      // rank rounded up to 16
    int ksplit;
};

__device__ __forceinline__ int rank_of(const fqm_adapters& a, int i) {
    return a.ranks ? max(0, min(a.ranks[i], a.rank)) : a.rank;
}

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ u32x4 load16(const uint16_t* p) { return *reinterpret_cast<const u32x4*>(p); }

// ---- few rows: which rows go together --------------------------------------------
// Row r's job: if r is the 1st, 17th, 33rd ... row of its adapter, the up to
// 16 rows of that adapter from r on (rows without one count as an adapter of
// their own, -1).  Lane l's row for l % 16; lanes past the last row repeat the
// first.  False: another row's job has r.
struct FewRows {
    int idx;        // the adapter, -1: none
    int n;          // rows
    int64_t m;      // this lane's row
};
__device__ __forceinline__ int adapter_of(const Lora& p, int64_t m) {
    const int i = p.index[m];
    return (unsigned)i < (unsigned)p.a.count ? i : -1;
}
__device__ __forceinline__ bool few_rows(const Lora& p, int64_t r, FewRows* f) {
    const int lane = threadIdx.x & 63, col = lane & 15;
    f->idx = adapter_of(p, r);
    f->n = 0;
    f->m = r;
    int before = 0;  // rows of the adapter ahead of r
    for (int64_t m0 = 0; m0 < p.M; m0 += 64) {
        const int64_t m = m0 + lane;
        uint64_t same = __ballot(m < p.M && adapter_of(p, min(m, p.M - 1)) == f->idx);
        if (r >= m0 + 64) {
            before += __builtin_popcountll(same);
            continue;
        }
        if (r >= m0) {
            const uint64_t ahead = (1ull << (r - m0)) - 1;
            before += __builtin_popcountll(same & ahead);
            if (before & 15) return false;
            same &= ~ahead;
        }
        while (same && f->n < 16) {
            if (col == f->n) f->m = m0 + __builtin_ctzll(same);
            same &= same - 1;
            ++f->n;
        }
        if (f->n == 16) break;
    }
    return true;
}

// ---- t = A x, few rows ------------------------------------------------------------
// A wave: a job's rows of x (matrix columns: lane % 16) times RB blocks of 16
// rows of its adapter's A, 32 columns a step; lane (j, q) holds columns 8 q ..
// 8 q + 7 of a step of row j.  U steps' loads go out together.  The four waves
// of a workgroup have four stretches of its K part and add them up in order.
template <int RB>
__global__ __launch_bounds__(64 * kWaves) void lora_shrink_few(const Lora p) {
    __shared__ f32x4 s_acc[kWaves][RB][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), q = lane >> 4;
    const int chunks = (p.ldt + 16 * RB - 1) / (16 * RB);
    int job = blockIdx.x;
    const int ks = job % p.ksplit;
    job /= p.ksplit;
    const int r0 = 16 * RB * (job % chunks);
    FewRows f;
    if (!few_rows(p, job / chunks, &f) || f.idx < 0) return;  // the whole workgroup
    const int i = f.idx, rank = rank_of(p.a, i);
    if (r0 >= rank) return;
    const int K = (int)p.a.cols, all = (K + 31) / 32, parts = p.ksplit * kWaves, part = ks * kWaves + wave;
    const int t0 = (int)((int64_t)part * all / parts), t1 = (int)((int64_t)(part + 1) * all / parts);
    const uint16_t* xp = p.x + f.m * K + 8 * q;
    const uint16_t* ap[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b)
        ap[b] = p.a.A + ((int64_t)i * p.a.rank + min(r0 + 16 * b + (lane & 15), rank - 1)) * p.a.ld_A + 8 * q;
    f32x4 acc[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
    constexpr int U = 4;
    const int full = min(t1, K / 32);  // steps with all 32 columns
    int t = t0;
    for (; t + U <= full; t += U) {
        u32x4 xv[U], av[U][RB];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            xv[u] = load16(xp + 32 * (t + u));
#pragma unroll
            for (int b = 0; b < RB; ++b) av[u][b] = load16(ap[b] + 32 * (t + u));
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int b = 0; b < RB; ++b) acc[b] = mfma(av[u][b], xv[u], acc[b]);
    }
    if (t < t1) {  // up to U steps, the last one perhaps short: columns past the end count as zeros
        u32x4 xv[U], av[U][RB];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = t + u < t1 && 32 * (t + u) + 8 * q < K;
            xv[u] = u32x4{0u, 0u, 0u, 0u};
            if (in) xv[u] = load16(xp + 32 * (t + u));
#pragma unroll
            for (int b = 0; b < RB; ++b) {
                av[u][b] = u32x4{0u, 0u, 0u, 0u};
                if (in) av[u][b] = load16(ap[b] + 32 * (t + u));
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int b = 0; b < RB; ++b) acc[b] = mfma(av[u][b], xv[u], acc[b]);
    }
#pragma unroll
    for (int b = 0; b < RB; ++b) s_acc[wave][b][lane] = acc[b];
    __syncthreads();
    // D: column lane % 16, rows 4 q .. 4 q + 3; sums past the rank are never read.  Wave b adds up block b.
    if (wave < RB && (lane & 15) < f.n && r0 + 16 * wave < p.ldt) {
        f32x4 v = s_acc[0][wave][lane];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) v += s_acc[w][wave][lane];
        *reinterpret_cast<f32x4*>(p.part + ((int64_t)ks * p.M + f.m) * p.ldt + r0 + 16 * wave + 4 * q) = v;
    }
}

// ---- t = A x, many rows -------------------------------------------------------------
// A workgroup: 64 rows of x times 16 RB rows of an adapter's A over one K part,
// 64 columns a step.  Both tiles come by direct global -> LDS loads (1 KB: 8
// rows of 128 bytes, 16-byte chunks XOR-swizzled by (row / 2) % 8) four steps
// ahead in five buffers; a wave contracts its 16 rows of x.  Columns past the
// last whole step (K is a multiple of 8) go through registers.
constexpr int kRing = 5;
template <int RB>
struct ShrinkTile {
    static constexpr int X_BYTES = 64 * 128, BYTES = X_BYTES + 16 * RB * 128;
    static constexpr int A_KB = 2 * RB;                            // kilobytes of A a step
    static constexpr int A_LOADS = A_KB >= kWaves ? A_KB / kWaves : 1;  // with RB = 1 two waves load each twice
    static constexpr int LOADS = 2 + A_LOADS;                      // per wave and step
};

__device__ __forceinline__ int chunk_at(int row, int chunk) { return 128 * row + 16 * (chunk ^ ((row >> 1) & 7)); }

template <int RB>
__device__ __forceinline__ void shrink_block(lds8* const (&BUF)[kRing], const Lora& p, int tiles) {
    using S = ShrinkTile<RB>;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int q = lane >> 4, col = lane & 15, K = (int)p.a.cols;
    int b = blockIdx.x;
    const int64_t m0 = (int64_t)(b % tiles) * 64;
    b /= tiles;
    const int ks = b % p.ksplit, r0 = b / p.ksplit * (16 * RB);
    const int all = K / 64, t0 = (int)((int64_t)ks * all / p.ksplit), t1 = (int)((int64_t)(ks + 1) * all / p.ksplit);
    const bool tail = ks == p.ksplit - 1 && (K & 63);

    // lane r: row m0 + r of the block
    const int idx = m0 + lane < p.M ? p.index[m0 + lane] : -1;
    const int rows_here = (int)min((int64_t)64, p.M - m0);
    const uint16_t* x = p.x + m0 * K;
    const __amdgpu_buffer_rsrc_t xr = __builtin_amdgcn_make_buffer_rsrc((void*)x, (short)0, 0x7fffffff, 0x00020000);
    uint32_t xo[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int row = 8 * (kWaves * u + wave) + (lane >> 3);
        xo[u] = (uint32_t)min(row, rows_here - 1) * (uint32_t)K * 2u + 16u * ((lane & 7) ^ ((row >> 1) & 7));
    }
    uint64_t left = __ballot((unsigned)idx < (unsigned)p.a.count);
    while (left) {
        const int i = __builtin_amdgcn_readlane(idx, __builtin_ctzll(left));
        const uint64_t rows = __ballot(idx == i);
        left &= ~rows;
        const int rank = rank_of(p.a, i);
        if (r0 >= rank) continue;
        const uint16_t* A = p.a.A + ((int64_t)i * p.a.rank + r0) * p.a.ld_A;
        const int a_last = min(16 * RB, rank - r0) - 1;  // rows of A past it repeat it; their sums are never read
        const __amdgpu_buffer_rsrc_t ar = __builtin_amdgcn_make_buffer_rsrc((void*)A, (short)0, 0x7fffffff, 0x00020000);
        uint32_t ao[S::A_LOADS];
#pragma unroll
        for (int u = 0; u < S::A_LOADS; ++u) {
            const int row = 8 * ((kWaves * u + wave) % S::A_KB) + (lane >> 3);
            ao[u] = (uint32_t)min(row, a_last) * (uint32_t)p.a.ld_A * 2u + 16u * ((lane & 7) ^ ((row >> 1) & 7));
        }
        auto request = [&](int buf, int t) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(xr, (lvoid*)(BUF[buf] + 1024 * (kWaves * u + wave)), 16, xo[u],
                                                         (uint32_t)t * 128u, 0, 0);
#pragma unroll
            for (int u = 0; u < S::A_LOADS; ++u)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    ar, (lvoid*)(BUF[buf] + S::X_BYTES + 1024 * ((kWaves * u + wave) % S::A_KB)), 16, ao[u],
                    (uint32_t)t * 128u, 0, 0);
        };
        f32x4 acc[RB];
#pragma unroll
        for (int r = 0; r < RB; ++r) acc[r] = f32x4{0.f, 0.f, 0.f, 0.f};
        auto contract = [&](int buf) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const u32x4 xv = *(lds128c*)(BUF[buf] + chunk_at(16 * wave + col, 4 * s + q));
#pragma unroll
                for (int r = 0; r < RB; ++r) {
                    const u32x4 av = *(lds128c*)(BUF[buf] + S::X_BYTES + chunk_at(16 * r + col, 4 * s + q));
                    acc[r] = mfma(av, xv, acc[r]);
                }
            }
        };
        if (t0 < t1) {
            // Step t is in buffer (t - t0) % kRing.  Before its barrier each wave waits for its own loads of
            // step t (those of the kAhead - 1 steps after it may be in flight); after it every wave has used
            // step t - 1, whose buffer takes step t + kAhead.  Past the end the last step is loaded again, and
            // not used.
            constexpr int kAhead = kRing - 1;
            __syncthreads();  // the last adapter's steps are used
#pragma unroll
            for (int s = 0; s < kAhead; ++s) request(s, min(t0 + s, t1 - 1));
            auto step = [&](int buf, int t) {
                __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): step t - 1 is read, not just requested
                barrier_after_loads<(kAhead - 1) * S::LOADS>();
                request((buf + kAhead) % kRing, min(t + kAhead, t1 - 1));
                contract(buf);
            };
            int t = t0;
            for (; t + kRing - 1 < t1; t += kRing) {
#pragma unroll
                for (int s = 0; s < kRing; ++s) step(s, t + s);
            }
#pragma unroll
            for (int s = 0; s < kRing - 1; ++s)
                if (t + s < t1) step(s, t + s);
            __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): no load may still be writing LDS
        }
        const bool mine = rows >> (16 * wave + col) & 1;
        if (tail) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int k = 64 * all + 32 * s + 8 * q;
                u32x4 xv = {0u, 0u, 0u, 0u};
                if (k < K) xv = load16(x + (int64_t)min(16 * wave + col, rows_here - 1) * K + k);
#pragma unroll
                for (int r = 0; r < RB; ++r) {
                    u32x4 av = {0u, 0u, 0u, 0u};
                    if (k < K) av = load16(A + (int64_t)min(16 * r + col, a_last) * p.a.ld_A + k);
                    acc[r] = mfma(av, xv, acc[r]);
                }
            }
        }
        if (mine) {  // D: column col, rows 4 q .. 4 q + 3
            float* out = p.part + ((int64_t)ks * p.M + m0 + 16 * wave + col) * p.ldt + r0 + 4 * q;
#pragma unroll
            for (int r = 0; r < RB; ++r)
                if (r0 + 16 * r < p.ldt) *reinterpret_cast<f32x4*>(out + 16 * r) = acc[r];
        }
    }
}

template <int RB>
__global__ __launch_bounds__(64 * kWaves) void lora_shrink_blocks(const Lora p, int tiles) {
    __shared__ __attribute__((aligned(16))) uint8_t s_0[ShrinkTile<RB>::BYTES];
    __shared__ __attribute__((aligned(16))) uint8_t s_1[ShrinkTile<RB>::BYTES];
    __shared__ __attribute__((aligned(16))) uint8_t s_2[ShrinkTile<RB>::BYTES];
    __shared__ __attribute__((aligned(16))) uint8_t s_3[ShrinkTile<RB>::BYTES];
    __shared__ __attribute__((aligned(16))) uint8_t s_4[ShrinkTile<RB>::BYTES];
    lds8* const buf[kRing] = {(lds8*)s_0, (lds8*)s_1, (lds8*)s_2, (lds8*)s_3, (lds8*)s_4};
    shrink_block<RB>(buf, p, tiles);
}

// ---- y = base + B t ---------------------------------------------------------------
// The rows' t = scale * (sum of the K parts) goes to LDS as three bf16 terms, each
// the leading 8 bits of what the ones before it leave, cut off, not rounded (the
// largest fp32 values would round up to infinity): 24 bits, all of t, whatever
// y's type (two terms would leave 2^-16, enough to turn the rounding of some bf16
// outputs).  Each meets the same B, smallest first, and the products are exact
// in fp32; where B is not finite only the leading term meets it (finite_of).  In
// a pass of 128 outputs every distinct adapter's B meets the block's rows and its
// own rows' sums go to a tile in LDS; then base streams through it to y in whole
// lines, the next pass's base already requested.  (Straight from the matrix
// layout, 16 rows a load, the same took 1.5 to 2 times as long with many rows.)
constexpr int kTerms = 3;

enum BaseKind { kNoBase = 0, kBaseBf16 = 1, kBaseF32 = 2 };

// 8 consecutive values of base as loaded, from value `at` on (a pointer that is
// the same for all lanes and 32 bits: one address register); n: how many exist.
template <int BASE>
struct Base8 {
    u32x4 v[BASE == kBaseF32 ? 2 : 1];
    __device__ __forceinline__ void load(const void* base, uint32_t at, int n) {
        if constexpr (BASE == kBaseBf16) {
            const uint16_t* b = reinterpret_cast<const uint16_t*>(static_cast<const char*>(base) + at * 2u);
            if (n >= 8) {
                v[0] = *reinterpret_cast<const u32x4_a2*>(b);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t lo = 2 * e < n ? b[2 * e] : 0, hi = 2 * e + 1 < n ? b[2 * e + 1] : 0;
                    v[0][e] = lo | hi << 16;
                }
            }
        } else if constexpr (BASE == kBaseF32) {
            const uint32_t* b = reinterpret_cast<const uint32_t*>(static_cast<const char*>(base) + at * 4u);
            if (n >= 8) {
                v[0] = reinterpret_cast<const u32x4_a4*>(b)[0];
                v[1] = reinterpret_cast<const u32x4_a4*>(b)[1];
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e >> 2][e & 3] = e < n ? b[e] : 0u;
            }
        }
    }
    __device__ __forceinline__ float at(int e) const {
        if constexpr (BASE == kBaseBf16) return e & 1 ? bf16hi(v[0][e >> 1]) : bf16lo(v[0][e >> 1]);
        else if constexpr (BASE == kBaseF32) return __uint_as_float(v[e >> 2][e & 3]);
        else return 0.f;
    }
};

__device__ __forceinline__ uint32_t bf16_bits(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

__device__ __forceinline__ void store8(void* y, int f32, uint32_t at, const float (&o)[8], int n) {
    if (f32) {
        uint32_t* q = reinterpret_cast<uint32_t*>(static_cast<char*>(y) + at * 4u);
        if (n >= 8) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                u32x4 v;
#pragma unroll
                for (int c = 0; c < 4; ++c) v[c] = __float_as_uint(o[4 * e + c]);
                reinterpret_cast<u32x4_a4*>(q)[e] = v;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n) q[e] = __float_as_uint(o[e]);
        }
    } else {
        uint16_t* q = reinterpret_cast<uint16_t*>(static_cast<char*>(y) + at * 2u);
        if (n >= 8) {
            u32x4 v;
#pragma unroll
            for (int c = 0; c < 4; ++c) v[c] = bf16_bits(o[2 * c]) | bf16_bits(o[2 * c + 1]) << 16;
            *reinterpret_cast<u32x4_a2*>(q) = v;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n) q[e] = (uint16_t)bf16_bits(o[e]);
        }
    }
}

constexpr int kPass = 128;        // outputs per pass

// 8 ranks from 8 r8 on of one row's t to LDS: [ranks / 32][kTerms][`bytes` of rows of 32].
__device__ __forceinline__ void put_t(const Lora& p, int64_t m, int row, int r8, int rank, float scale, uint8_t* s_t,
                                      int bytes) {
    f32x4 v[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    const float* src = p.part + m * p.ldt + 8 * r8;
#pragma unroll 8
    for (int k = 0; k < p.ksplit; ++k) {
        v[0] += *reinterpret_cast<const f32x4*>(src + (int64_t)k * p.M * p.ldt);
        v[1] += *reinterpret_cast<const f32x4*>(src + (int64_t)k * p.M * p.ldt + 4);
    }
    float t[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = 8 * r8 + e < rank ? scale * v[e >> 2][e & 3] : 0.f;
    uint8_t* dst = s_t + (r8 >> 2) * (kTerms * bytes) + row * 64 + 16 * (r8 & 3);
#pragma unroll
    for (int term = 0; term < kTerms; ++term) {
        u32x4 o;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            uint32_t h[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float& left = t[2 * e + c];
                h[c] = __float_as_uint(left) & 0xFFFF0000u;
                // an infinite t has one term (inf - inf is none)
                left = (h[c] & 0x7F800000u) == 0x7F800000u ? 0.f : left - __uint_as_float(h[c]);
            }
            o[e] = h[0] >> 16 | h[1];
        }
        *reinterpret_cast<u32x4*>(dst + term * bytes) = o;
    }
}

// J blocks of 16 outputs' operands of B, 32 ranks from 32 kb on; what lies past
// the rank counts as zero, whatever it holds.
template <int J>
__device__ __forceinline__ void load_b(const uint16_t* B, int64_t ld, int n0, int N, int have, int kb, u32x4 (&b)[J]) {
    const int q = (threadIdx.x & 63) >> 4, col = threadIdx.x & 15;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        b[j] = u32x4{0u, 0u, 0u, 0u};
        if (have > 0) b[j] = load16(B + (int64_t)min(n0 + 16 * j + col, N - 1) * ld + 32 * kb + 8 * q);
    }
}
template <int J>
__device__ __forceinline__ void cut_b(int have, u32x4 (&b)[J]) {
    if (have < 8) {
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                b[j][e] &= (2 * e < have ? 0xFFFFu : 0u) | (2 * e + 1 < have ? 0xFFFF0000u : 0u);
    }
}

// Outputs [n, n + cnt) of a row from its sums in LDS (four each at a and b; NULL: none) and base.
template <int BASE>
__device__ __forceinline__ void finish8(void* y, int y_f32, const f32x4* a_at, const f32x4* b_at, const Base8<BASE>& base,
                                        uint32_t at, int cnt) {
    float o[8];
    if (a_at) {
        const f32x4 a = *a_at, b = *b_at;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = (e < 4 ? a[e & 3] : b[e & 3]) + base.at(e);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = base.at(e);
    }
    store8(y, y_f32, at, o, cnt);
}

// What t's lower terms meet: B without its infinities and NaN.  A lower term may
// be zero or of the other sign, and its product with an infinity would turn the
// leading term's into NaN.  Whether there are any is uniform, and hardly ever true.
template <int J>
__device__ __forceinline__ void finite_of(const u32x4 (&b)[J], u32x4 (&low)[J]) {
    uint32_t any = 0;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) any |= (b[j][e] & 0x7F807F80u) + 0x00800080u;  // bit 15 / 31: the half's exponent is full
#pragma unroll
    for (int j = 0; j < J; ++j) low[j] = b[j];
    if (__builtin_expect(__ballot((any & 0x80008000u) != 0) != 0, 0)) {
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t full = ((b[j][e] & 0x7F807F80u) + 0x00800080u) >> 15 & 0x00010001u;
                low[j][e] &= ~((full << 16) - full);
            }
    }
}

// The tile of sums in LDS: rows of kPass floats, four outputs (`quad`, of kPass / 4) apiece, XOR-swizzled so
// that 16 rows' pieces of one quad lie in 16 different bank groups (without padding: with it two workgroups of
// rank 128 would not fit a CU).
__device__ __forceinline__ f32x4* sums_at(uint8_t* s_d, int row, int quad) {
    return reinterpret_cast<f32x4*>(s_d + kPass * 4 * row + 16 * (quad ^ (row & 15)));
}

// Few rows.  Wave job: (row, pass of outputs), the rows of few_rows.  Waves are
// independent of each other.
constexpr int kFewBytes = 16 * 64;             // of one term of 32 ranks of 16 rows' t
constexpr int kFewTile = 16 * kPass * 4;

template <int BASE>
__global__ __launch_bounds__(64 * kWaves) void lora_expand_few(const Lora p, int passes) {
    extern __shared__ __attribute__((aligned(16))) uint8_t s_all[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int q = lane >> 4, col = lane & 15, N = (int)p.a.rows, t_bytes = (p.ldt + 31) / 32 * kTerms * kFewBytes;
    uint8_t* s_t = s_all + wave * (kFewTile + t_bytes);        // [ranks / 32][kTerms][16][32] bf16
    uint8_t* s_d = s_t + t_bytes;                              // 16 rows of sums
    const int64_t job = (int64_t)blockIdx.x * kWaves + wave;
    if (job >= p.M * passes) return;
    const int n0 = (int)(job % passes) * kPass, n_hi = min(N, n0 + kPass);
    FewRows f;
    if (!few_rows(p, job / passes, &f)) return;

    // base: lane group q, row 4 s + q of the job, 8 outputs from 8 col on
    const int n = n0 + 8 * col, cnt = min(8, n_hi - n);
    int64_t at[4];  // of the rows' first value
    constexpr int64_t kB = BASE == kBaseF32 ? 4 : 2;
    Base8<BASE> base[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        at[s] = __shfl((int)f.m, 4 * s + q, 64) * (int64_t)N;
        if (4 * s + q < f.n && cnt > 0) base[s].load(static_cast<const char*>(p.base) + at[s] * kB, (uint32_t)n, cnt);
    }
    if (f.idx >= 0) {
        const int i = f.idx, rank = rank_of(p.a, i), groups = (rank + 7) / 8;
        const float scale = p.a.scale ? p.a.scale[i] : 1.f;
        const uint16_t* B = p.a.B + (int64_t)i * N * p.a.ld_B;
        for (int w0 = 0; w0 < f.n * groups; w0 += 64) {
            const int w = w0 + lane, r = w / groups, r8 = w - r * groups;
            const int64_t m = __shfl((int)f.m, r & 15, 64);  // ahead of the condition: from lanes that may not meet it
            if (r < f.n) put_t(p, m, r, r8, rank, scale, s_t, kFewBytes);
        }
        wave_lds_order();
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if (n0 + 64 * half >= n_hi) break;
            f32x4 acc[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
            for (int kb = 0; 32 * kb < rank; ++kb) {
                const int have = rank - 32 * kb - 8 * q;  // of this lane's 8 ranks
                u32x4 b[4];
                load_b<4>(B, p.a.ld_B, n0 + 64 * half, N, have, kb, b);
                cut_b<4>(have, b);
                u32x4 low[4];
                finite_of<4>(b, low);
#pragma unroll
                for (int term = kTerms - 1; term >= 0; --term) {
                    u32x4 t = {0u, 0u, 0u, 0u};
                    if (have > 0)
                        t = *reinterpret_cast<const u32x4*>(s_t + (kb * kTerms + term) * kFewBytes + col * 64 + 16 * q);
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[j] = mfma(term ? low[j] : b[j], t, acc[j]);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)  // D: row col of the job, outputs 16 j + 4 q .. + 3
                *sums_at(s_d, col, 16 * half + 4 * j + q) = acc[j];
        }
        wave_lds_order();
    }
#pragma unroll
    for (int s = 0; s < 4; ++s)
        if (4 * s + q < f.n && cnt > 0)
            finish8<BASE>(static_cast<char*>(p.y) + at[s] * (p.y_f32 ? 4 : 2), p.y_f32,
                          f.idx >= 0 ? sums_at(s_d, 4 * s + q, 2 * col) : nullptr, sums_at(s_d, 4 * s + q, 2 * col + 1), base[s],
                          (uint32_t)n, cnt);
}

// Many rows.  A workgroup: 64 rows and a range of outputs; in a pass a wave has
// 32 of the 128 outputs, against all 64 rows.
constexpr int kManyBytes = 64 * 64;            // of one term of 32 ranks of 64 rows' t
constexpr int kManyTile = 64 * kPass * 4;

// Three workgroups a CU (168 registers) where base is bf16: 100 us against 121 with two (4096 rows, rank 16,
// 5120 -> 17408; the compiler now stays below 168 by itself, 92 us with this bound or without).  An fp32 base
// does not fit them, and from rank 33 on the rows' t leaves LDS for two.
template <int BASE>
__global__ __launch_bounds__(64 * kWaves, BASE == kBaseF32 ? 2 : 3) void lora_expand_blocks(const Lora p, int ranges, int range) {
    extern __shared__ __attribute__((aligned(16))) uint8_t s_all[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int q = lane >> 4, col = lane & 15, N = (int)p.a.rows;
    uint8_t* s_d = s_all;              // 64 rows of sums
    uint8_t* s_t = s_all + kManyTile;  // [ranks / 32][kTerms][64][32] bf16
    const int64_t m0 = (int64_t)(blockIdx.x / ranges) * 64;
    const int n_lo = blockIdx.x % ranges * range, n_hi = min(N, n_lo + range);
    const char* base_0 = static_cast<const char*>(p.base) + m0 * N * (BASE == kBaseF32 ? 4 : 2);
    char* y_0 = static_cast<char*>(p.y) + m0 * N * (p.y_f32 ? 4 : 2);
    // lane r of every wave: row m0 + r
    const int idx = m0 + lane < p.M ? p.index[m0 + lane] : -1;
    const bool any = (unsigned)idx < (unsigned)p.a.count;
    const uint64_t with = __ballot(any), there = __ballot(m0 + lane < p.M);

    // base of a pass: thread (16 g + c), rows 16 s + g of the block, 8 outputs from 8 c on
    const int g = tid >> 4;
    auto load_base = [&](int n0, Base8<BASE> (&base)[4]) {
        const int n = n0 + 8 * col;
#pragma unroll
        for (int s = 0; s < 4; ++s)
            if ((there >> (16 * s + g) & 1) && n < n_hi) base[s].load(base_0, (uint32_t)((16 * s + g) * N + n), min(8, n_hi - n));
    };
    Base8<BASE> base[4];
    load_base(n_lo, base);
    const int rank = any ? rank_of(p.a, idx) : 0;
    const float scale = any && p.a.scale ? p.a.scale[idx] : 1.f;
    const int groups = p.ldt / 8;
    for (int w = tid; w < 64 * groups; w += 64 * kWaves) {
        const int r = w / groups, r8 = w - r * groups, rank_r = __shfl(rank, r, 64);
        const float scale_r = __shfl(scale, r, 64);
        if (8 * r8 < rank_r) put_t(p, m0 + r, r, r8, rank_r, scale_r, s_t, kManyBytes);
    }
    int row_idx[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) row_idx[t] = __shfl(any ? idx : -1, 16 * t + col, 64);
    // the first adapter's first 64 ranks of B come a pass ahead
    const int lead = with ? __builtin_amdgcn_readlane(idx, __builtin_ctzll(with)) : 0;
    const int lead_rank = with ? __builtin_amdgcn_readlane(rank, __builtin_ctzll(with)) : 0;
    const uint16_t* lead_B = p.a.B + (int64_t)lead * N * p.a.ld_B;
    u32x4 ahead[2][2];
    auto load_ahead = [&](int nw) {
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) load_b<2>(lead_B, p.a.ld_B, nw, N, lead_rank - 32 * kb - 8 * q, kb, ahead[kb]);
    };
    load_ahead(n_lo + 32 * wave);
    lds_barrier();

    // one pass: `now` holds its base, `next` takes that of the following one (two names, no copies: a copy
    // would wait for the loads)
    auto pass = [&](int n0, Base8<BASE> (&now)[4], Base8<BASE> (&next)[4]) {
        const int nw = n0 + 32 * wave;
        bool first = true;
        for (uint64_t left = nw < n_hi ? with : 0; left; first = false) {
            const int l = __builtin_ctzll(left), i = __builtin_amdgcn_readlane(idx, l), ri = __builtin_amdgcn_readlane(rank, l);
            const uint64_t rows = __ballot(any && idx == i);
            left &= ~rows;
            const uint16_t* B = p.a.B + (int64_t)i * N * p.a.ld_B;
            f32x4 acc[4][2];
#pragma unroll
            for (int t = 0; t < 4; ++t) acc[t][0] = acc[t][1] = f32x4{0.f, 0.f, 0.f, 0.f};
            for (int kb = 0; 32 * kb < ri; ++kb) {
                const int have = ri - 32 * kb - 8 * q;  // of this lane's 8 ranks
                u32x4 b[2];
                if (first && kb < 2) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) b[j] = kb ? ahead[1][j] : ahead[0][j];
                } else {
                    load_b<2>(B, p.a.ld_B, nw, N, have, kb, b);
                }
                cut_b<2>(have, b);
                u32x4 low[2];
                finite_of<2>(b, low);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    if (!(rows >> (16 * t) & 0xFFFFu)) continue;  // uniform
                    const uint8_t* at = s_t + kb * (kTerms * kManyBytes) + (16 * t + col) * 64 + 16 * q;
                    u32x4 tv[kTerms];
#pragma unroll
                    for (int u = 0; u < kTerms; ++u) {
                        tv[u] = u32x4{0u, 0u, 0u, 0u};
                        if (have > 0) tv[u] = *reinterpret_cast<const u32x4*>(at + u * kManyBytes);
                    }
#pragma unroll
                    for (int u = kTerms - 1; u >= 0; --u)
#pragma unroll
                        for (int j = 0; j < 2; ++j) acc[t][j] = mfma(u ? low[j] : b[j], tv[u], acc[t][j]);
                }
            }
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (row_idx[t] == i) {  // D: row 16 t + col of the block, outputs 16 j + 4 q .. + 3
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        *sums_at(s_d, 16 * t + col, 8 * wave + 4 * j + q) = acc[t][j];
                }
        }
        if (n0 + kPass < n_hi) {
            load_ahead(nw + kPass);  // ahead of base: it is waited for first
            load_base(n0 + kPass, next);
        }
        lds_barrier();
        const int n = n0 + 8 * col;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int r = 16 * s + g;
            if ((there >> r & 1) && n < n_hi)
                finish8<BASE>(y_0, p.y_f32, with >> r & 1 ? sums_at(s_d, r, 2 * col) : nullptr, sums_at(s_d, r, 2 * col + 1),
                              now[s], (uint32_t)(r * N + n), min(8, n_hi - n));
        }
        lds_barrier();  // the tile is read
    };
    Base8<BASE> other[4];
    for (int n0 = n_lo; n0 < n_hi; n0 += 2 * kPass) {
        pass(n0, base, other);
        if (n0 + kPass < n_hi) pass(n0 + kPass, other, base);
    }
}

// ---- the plan -----------------------------------------------------------------------
// Up to kFewRows rows each adapter's rows are collected from the batch; more
// rows are taken 64 by 64 as they lie.  One MI355X, us for collected / as they
// lie: 48 rows in any order over 32 adapters (ranks to 32, 17408 -> 5120) 19 /
// 94, 256 rows 29 / 113; runs of 3 adapters (rank 16, 5120 -> 17408) 128 rows
// 20 / 13, 512 rows 70 / 22.  The rule looks at M alone, so that more than 256 rows
// in any order are slow: 5120 -> 5120 in bf16, 32 adapters of rank 16, in any order
// / in runs: 256 rows 18 / 21, 257 rows 70 / 24, 1024 rows 80 / 22; 64 adapters of
// rank 32: 27 / 31, 101 / 46, 109 / 30.
constexpr int64_t kFewRows = 256;

struct LoraPlan {
    bool few;
    int rb, ldt, ksplit, chunks;
    int64_t blocks;  // few: rows, otherwise blocks of 64
};

// K parts: as many as fill the chip (512 workgroups of a job's four stretches
// or 256 of 64-row blocks), each of at least four steps, few enough that adding
// them up again stays small (4096 rows, rank 64, aimed at 256 / 512 / 768
// workgroups: 145 / 147 / 161 us).
LoraPlan lora_plan(const fqm_adapters& a, int64_t M) {
    LoraPlan p;
    p.few = M <= kFewRows;
    p.ldt = (a.rank + 15) / 16 * 16;
    p.rb = p.ldt >= 64 ? 4 : p.ldt >= 32 ? 2 : 1;
    p.chunks = (p.ldt + 16 * p.rb - 1) / (16 * p.rb);
    p.blocks = p.few ? M : (M + 63) / 64;
    const int64_t jobs = (p.few ? std::min<int64_t>(M, a.count + M / 16) : p.blocks) * p.chunks;
    const int64_t parts = p.few ? std::min<int64_t>({512 / std::max<int64_t>(jobs, 1), a.cols / 512, (int64_t)8})
                                : std::min<int64_t>({256 / std::max<int64_t>(jobs, 1), a.cols / 256, (int64_t)16});
    p.ksplit = (int)std::max<int64_t>(parts, 1);
    return p;
}

template <int BASE>
hipError_t launch_base(const Lora& p, const LoraPlan& pl, hipStream_t s) {
    const int kblocks = (p.ldt + 31) / 32, N = (int)p.a.rows, passes = (N + kPass - 1) / kPass;
    if (pl.few) {
        const int64_t grid = (p.M * passes + kWaves - 1) / kWaves;
        if (grid > 0x7fffffff) return hipErrorInvalidValue;
        hipLaunchKernelGGL(lora_expand_few<BASE>, dim3((unsigned)grid), dim3(64 * kWaves),
                           (size_t)(kblocks * kTerms * kFewBytes + kFewTile) * kWaves, s, p, passes);
    } else {
        // up to four passes share the rows' t (4096 rows, rank 64, 8 / 4 / 2 passes: 151 / 144 / 150 us),
        // as long as there are 1024 workgroups
        const int range = (int)std::max<int64_t>(1, std::min<int64_t>(4, pl.blocks * passes / 1024)) * kPass;
        const int ranges = (N + range - 1) / range;
        const int64_t grid = pl.blocks * ranges;
        if (grid > 0x7fffffff) return hipErrorInvalidValue;
        hipLaunchKernelGGL(lora_expand_blocks<BASE>, dim3((unsigned)grid), dim3(64 * kWaves),
                           (size_t)(kblocks * kTerms * kManyBytes + kManyTile), s, p, ranges, range);
    }
    return hipGetLastError();
}

template <int RB>
hipError_t launch_shrink(const Lora& p, const LoraPlan& pl, hipStream_t s) {
    const int64_t grid = pl.blocks * pl.chunks * pl.ksplit;
    if (grid > 0x7fffffff) return hipErrorInvalidValue;
    if (pl.few)
        hipLaunchKernelGGL(lora_shrink_few<RB>, dim3((unsigned)grid), dim3(64 * kWaves), 0, s, p);
    else
        hipLaunchKernelGGL(lora_shrink_blocks<RB>, dim3((unsigned)grid), dim3(64 * kWaves), 0, s, p, (int)pl.blocks);
    return hipGetLastError();
}

}  // namespace

size_t lora_workspace(const fqm_adapters& a, int64_t M) {
    const LoraPlan p = lora_plan(a, M);
    return (size_t)p.ksplit * M * p.ldt * sizeof(float);
}

hipError_t launch_lora(const fqm_adapters& a, const uint16_t* x, const int32_t* index, const void* base,
                       int base_f32, void* y, int y_f32, int64_t M, float* ws, hipStream_t s) {
    const LoraPlan pl = lora_plan(a, M);
    const Lora p = {a, x, index, base, y, y_f32, M, ws, pl.ldt, pl.ksplit};
    const hipError_t e = pl.rb == 1   ? launch_shrink<1>(p, pl, s)
                         : pl.rb == 2 ? launch_shrink<2>(p, pl, s)
                                      : launch_shrink<4>(p, pl, s);
    if (e != hipSuccess) return e;
    return !base ? launch_base<kNoBase>(p, pl, s) : base_f32 ? launch_base<kBaseF32>(p, pl, s) : launch_base<kBaseBf16>(p, pl, s);
}

}  // namespace fqm
