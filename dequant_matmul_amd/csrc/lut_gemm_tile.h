// The tile of the LUT GEMMs (fqm_gemm's and fqm_gemm_grouped's): X rows times
// decoded W rows on the bf16 matrix cores, the weights gathered from their
// rows' tables straight into the operands.  lut6_gemm.hip describes the scheme.
#pragma once

#include <type_traits>

#include "fqm_internal.h"

namespace fqm {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x4 u32x4_a8 __attribute__((aligned(8)));
typedef u32x2 u32x2_a8 __attribute__((aligned(8)));
typedef __attribute__((address_space(3))) uint8_t lds8;
typedef __attribute__((address_space(3))) uint16_t lds16;
typedef __attribute__((address_space(3))) const uint16_t lds16c;
typedef __attribute__((address_space(3))) const u32x4 lds128c;
typedef __attribute__((address_space(3))) void lvoid;

constexpr int BK = 64;
constexpr int NXB = 3;  // X tile buffers (and code slots): the loop is unrolled by 3
// A tile: BM rows of X by 32 NW rows of W, NW waves along W's rows, BM x 32
// outputs each.
template <int BM, int NW>
struct TileShape {
    static constexpr int BN = 32 * NW;
    static constexpr int MB = BM / 32;                 // 32-row blocks of X per wave
    static constexpr int XT_BYTES = BM * BK * 2;       // one X tile, 128-byte rows
    static constexpr int XKB = XT_BYTES / 1024;
    static constexpr int XDMA = XKB > NW ? XKB / NW : 1;  // 1 KB direct-to-LDS X loads per wave per step
    static_assert((XKB >= NW ? XKB % NW : NW % XKB) == 0 && NW % 2 == 0,
                  "every wave loads whole kilobytes of the X tile (with more waves than those, several load the "
                  "same bytes); whole table planes");
};

// Per code width: table entries, a table plane (64 rows' tables, bank-sliced),
// the code bytes a lane reads per K step (32 codes) and a row's bytes per step.
template <int BITS>
struct GemmFmt {
    static constexpr int ENTRIES = 1 << BITS;
    static constexpr int PLANE = 128 * ENTRIES;  // 8 KB (6-bit), 2 KB (4-bit)
    static constexpr int ND = BITS;              // dwords of code per lane per step
    static constexpr int STEP_BYTES = 8 * BITS;  // a row's 64 codes
    static constexpr int CODE_LOADS = ND == 6 ? 2 : 1;  // global loads per lane per step (16 + 8 or 16 bytes)
};

template <int BUF>
using Buf = std::integral_constant<int, BUF>;

// Table offset of code C (0..31) of a lane's code run d[0..ND): the code's
// bits moved to bits 7.. and OR-ed into the lane's row offset.
template <int BITS, int C, int ND>
__device__ __forceinline__ uint32_t code_addr(const uint32_t (&d)[ND], uint32_t mask, uint32_t base) {
    constexpr int bit = BITS * C, w = bit >> 5, o = bit & 31;
    uint32_t v;
    if constexpr (o + BITS <= 32) {
        if constexpr (o >= 7) v = d[w] >> (o - 7);
        else v = d[w] << (7 - o);
    } else {
        v = __builtin_amdgcn_alignbit(d[w + 1], d[w], o - 7);
    }
    return (v & mask) | base;
}

// The 8 gather addresses of slice Q (codes 8 Q .. 8 Q + 7).
template <int BITS, int Q, int ND>
__device__ __forceinline__ void slice_addrs(const uint32_t (&d)[ND], uint32_t mask, uint32_t base, uint32_t (&ad)[8]) {
    ad[0] = code_addr<BITS, 8 * Q + 0>(d, mask, base);
    ad[1] = code_addr<BITS, 8 * Q + 1>(d, mask, base);
    ad[2] = code_addr<BITS, 8 * Q + 2>(d, mask, base);
    ad[3] = code_addr<BITS, 8 * Q + 3>(d, mask, base);
    ad[4] = code_addr<BITS, 8 * Q + 4>(d, mask, base);
    ad[5] = code_addr<BITS, 8 * Q + 5>(d, mask, base);
    ad[6] = code_addr<BITS, 8 * Q + 6>(d, mask, base);
    ad[7] = code_addr<BITS, 8 * Q + 7>(d, mask, base);
}

template <int Q>
using Slice = std::integral_constant<int, Q>;

// Workgroup barrier after all but this wave's last N vector-memory loads have
// completed (loads complete in issue order).  LDS reads may stay in flight:
// the buffers they read are not rewritten before the next barrier.  The wait
// is the waitcnt builtin, so the compiler's own wait bookkeeping sees it; the
// barrier is the bare instruction between two compiler memory barriers (a
// workgroup fence would also wait for the loads left in flight).
template <int N>
__device__ __forceinline__ void barrier_after_loads() {
    static_assert(N >= 0 && N < 16, "vmcnt field");
    __builtin_amdgcn_s_waitcnt(0x0F70 | N);  // vmcnt(N) expcnt(7) lgkmcnt(15)
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

#define FQM_GEMM_TILE_LDS(BITS, BM, NW)                                                        \
    __shared__ __attribute__((aligned(8192))) uint8_t s_tab[(NW / 2) * GemmFmt<BITS>::PLANE];     \
    __shared__ __attribute__((aligned(16))) uint8_t s_x0[TileShape<BM, NW>::XT_BYTES];            \
    __shared__ __attribute__((aligned(16))) uint8_t s_x1[TileShape<BM, NW>::XT_BYTES];            \
    __shared__ __attribute__((aligned(16))) uint8_t s_x2[TileShape<BM, NW>::XT_BYTES]
#define FQM_GEMM_TILE_LDS_ARGS (lds8*)s_tab, (lds8*)s_x0, (lds8*)s_x1, (lds8*)s_x2

// Rows n0 .. n0 + 32 NW - 1 of W as a tile's columns (rows past N - 1 repeat it).
struct RunOfRows {
    int N, n0;
    __device__ __forceinline__ bool has(int r) const { return n0 + r < N; }
    __device__ __forceinline__ int row(int r) const { return min(n0 + r, N - 1); }
};

// The tile of BM rows of X and the 32 NW rows of W that `wr` names: wr.row(r) is
// tile column r's row of W, some row of it where there is none (wr.has(r)), over
// the K steps [t0, t0 + steps), steps >= 1.  x_off(row) is the byte offset
// of tile row `row` of X below X + xtile (32 bits in all; callers keep X below
// 2 GiB from X on, and rows past the end at some valid row); out(row, col, v)
// takes the fp32 sum of tile row `row` and tile column `col`, every one of
// them, in a fixed order; an `out` of (sums) takes a wave's 32 x 32 blocks of sums
// as the matrix instruction leaves them, behind a barrier after which the tile
// touches the LDS no more.  Where before is not NoPrep, before(scratch) runs ahead of
// the first out between two barriers, with at least 4 KB of LDS.
// tab, x0, x1, x2: LDS objects of their own (FQM_GEMM_TILE_LDS), so that the
// compiler sees that the table gathers do not wait for the direct loads of X.
struct NoPrep {};
template <int BITS, int BM, int NW, class XOff, class WRows, class Out, class Prep = NoPrep>
__device__ __forceinline__ void gemm_tile(lds8* tab, lds8* x0, lds8* x1, lds8* x2,
                                          const uint16_t* __restrict__ X, uint32_t xtile, XOff x_off,
                                          const uint8_t* __restrict__ packed, int64_t ld,
                                          const uint16_t* __restrict__ lut, WRows wr, int t0, int steps,
                                          Out out, Prep before = Prep()) {
    using S = TileShape<BM, NW>;
    constexpr int MB = S::MB, XDMA = S::XDMA, BN = S::BN;
    using F = GemmFmt<BITS>;
    constexpr int PLANE = F::PLANE, ND = F::ND, EPT = F::ENTRIES / 8;
    lds8* const XS[NXB] = {x0, x1, x2};
    lds8* const TAB = tab;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave;  // W rows 32 wn .. 32 wn + 31 of the tile
    const int g = lane >> 5, j = lane & 31;

    // ---- row tables, bank-sliced (resident for the whole K loop) ------------------
    for (int i = tid; i < BN * 8; i += 64 * NW) {
        const int r = i >> 3, part = i & 7;  // entries EPT part .. + EPT - 1 of tile row r
        uint32_t v[4] = {0u, 0u, 0u, 0u};
        if (wr.has(r)) {
            const uint16_t* src = lut + (int64_t)wr.row(r) * F::ENTRIES + part * EPT;
            if constexpr (EPT == 8) {
                const u32x4 q = *reinterpret_cast<const u32x4*>(src);
                v[0] = q[0]; v[1] = q[1]; v[2] = q[2]; v[3] = q[3];
            } else {
                v[0] = *reinterpret_cast<const uint32_t*>(src);
            }
        }
        lds8* dst = TAB + PLANE * (r >> 6) + 4 * (r & 31) + 2 * ((r >> 5) & 1) + 128 * EPT * part;
#pragma unroll
        for (int e = 0; e < EPT; ++e) *(lds16*)(dst + 128 * e) = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
    }
    // this lane's row 32 wn + j: plane wn / 2, half wn % 2 (bits below the code's and above them only)
    const uint32_t tbase = (uint32_t)PLANE * (wn >> 1) + 4u * j + 2u * (wn & 1);
    uint32_t cmask = (uint32_t)(F::ENTRIES - 1) << 7;
    asm volatile("" : "+v"(cmask));  // in a VGPR: (v & mask) | base is one v_and_or_b32

    // ---- X: direct global -> LDS, 1 KB (8 rows) per wave instruction -----------
    // Buffer loads with an LDS destination from the tile's X panel (the
    // compiler tracks these exactly; the flat-address form makes it wait for
    // every LDS read while one is in flight).  Load u of wave w fills rows
    // 8 (NW u + w) .. + 7 (modulo BM); lane l lands at byte 16 l of that kilobyte (row +
    // l / 8, stored chunk l % 8) and fetches the logical chunk that the
    // swizzle puts there, (l % 8) ^ ((row / 2) % 8).
    // X as one buffer; the tile's part of the offset goes into the scalar one.
    const __amdgpu_buffer_rsrc_t xrsrc = __builtin_amdgcn_make_buffer_rsrc((void*)X, (short)0, 0x7fffffff, 0x00020000);
    uint32_t xoff[XDMA];
#pragma unroll
    for (int u = 0; u < XDMA; ++u) {
        const int row = 8 * ((NW * u + wave) % S::XKB) + (lane >> 3);
        const int chunk = (lane & 7) ^ ((row >> 1) & 7);
        xoff[u] = x_off(row) + 16u * chunk;
    }
    auto dma_x = [&](int buf, int t) {
#pragma unroll
        for (int u = 0; u < XDMA; ++u)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(xrsrc, (lvoid*)(XS[buf] + 1024 * ((NW * u + wave) % S::XKB)), 16, xoff[u],
                                                     xtile + (uint32_t)t * (BK * 2), 0, 0);
    };

    // ---- codes: 24 bytes of row 32 wn + j per lane per step ------------------------
    const uint8_t* csrc = packed + (int64_t)wr.row(32 * wn + j) * ld + 4 * ND * g;
    uint32_t cw[NXB][ND];
    auto load_codes = [&](int slot, int t) {
        const uint8_t* p = csrc + F::STEP_BYTES * t;
        const u32x4 lo = *reinterpret_cast<const u32x4_a8*>(p);
        cw[slot][0] = lo[0]; cw[slot][1] = lo[1]; cw[slot][2] = lo[2]; cw[slot][3] = lo[3];
        if constexpr (ND == 6) {
            const u32x2 hi = *reinterpret_cast<const u32x2_a8*>(p + 16);
            cw[slot][4] = hi[0]; cw[slot][5] = hi[1];
        }
    };

    // ---- X operand offsets ------------------------------------------------------
    // A of block i, slice q: X tile row 32 i + j, logical chunk 4 g + q.
    int aoff[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) aoff[q] = 128 * j + 16 * ((4 * g + q) ^ ((j >> 1) & 7));

    f32x16 acc[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][r] = 0.f;

    __builtin_assume(steps > 0);

    // ---- operands: A one slice ahead, table gathers two slices ahead ----------------
    // a[i] and bop hold the operands of the slice whose MFMAs issue next, wv
    // the gathered table entries of the slice after it.  A slice first packs
    // wv into the next B operand; while its MFMAs run, the wave reads the next
    // slice's A operands (a[i] right after the MFMA that consumes it) and
    // gathers the entries of the slice after that.  The order is pinned with
    // scheduling groups, one MFMA at a time.
    bf16x8 a[MB];
    bf16x8 bop;
    uint32_t wv[8];
    auto pack_b = [&]() {
        u32x4 bw;
#pragma unroll
        for (int e = 0; e < 4; ++e) bw[e] = __builtin_amdgcn_perm(wv[2 * e + 1], wv[2 * e], 0x05040100u);
        return __builtin_bit_cast(bf16x8, bw);
    };
    auto read_a = [&](int buf, auto qc) {
        constexpr int q = decltype(qc)::value;
#pragma unroll
        for (int i = 0; i < MB; ++i) a[i] = __builtin_bit_cast(bf16x8, *(lds128c*)(XS[buf] + aoff[q] + 4096 * i));
    };
    auto gather = [&](auto qc, int slot) {
        constexpr int q = decltype(qc)::value;
        uint32_t ad[8];
        slice_addrs<BITS, q>(cw[slot], cmask, tbase, ad);
#pragma unroll
        for (int e = 0; e < 8; ++e) wv[e] = *(lds16c*)(TAB + ad[e]);
    };
    // Gathers ride with the first half of the slice's MFMAs (GPM per MFMA), so
    // that the perms at the start of the next slice wait only for LDS reads
    // issued half a slice earlier.
    constexpr int HALF = MB > 1 ? MB / 2 : 1, GPM = 8 / HALF;
    static_assert(GPM * HALF == 8, "8 gathers per slice");
    // The MFMAs of the current slice; A of slice AQ from X buffer AB, gathers of
    // slice GQ from code slot GS.
    auto slice = [&](auto aqc, int ab, auto gqc, int gs) {
        constexpr int aq = decltype(aqc)::value, gq = decltype(gqc)::value;
        __builtin_amdgcn_sched_barrier(0);
        const bf16x8 bnext = pack_b();
        uint32_t ad[8];
        slice_addrs<BITS, gq>(cw[gs], cmask, tbase, ad);
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], bop, acc[i], 0, 0, 0);
            a[i] = __builtin_bit_cast(bf16x8, *(lds128c*)(XS[ab] + aoff[aq] + 4096 * i));
            if (i < HALF) {
#pragma unroll
                for (int e = GPM * i; e < GPM * (i + 1); ++e) wv[e] = *(lds16c*)(TAB + ad[e]);
            }
        }
        bop = bnext;
        // perms and the first addresses; per MFMA: the MFMA, its A read (and in
        // the first half its gathers), then the next gathers' addresses
        __builtin_amdgcn_sched_group_barrier(0x0002, 4 + 2 * GPM, 0);
#pragma unroll
        for (int i = 0; i < HALF; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x0008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x0100, 1 + GPM, 0);
            __builtin_amdgcn_sched_group_barrier(0x0002, 2 * GPM, 0);
        }
#pragma unroll
        for (int i = HALF; i < MB; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x0008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x0100, 1, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    };

    // ---- prologue: X(t0) and the codes of steps t0, t0 + 1 in place; then, as
    // after every barrier, the next X tile and codes requested; operands of
    // slice 0 read and entries of slices 0 and 1 gathered
    dma_x(0, t0);
    load_codes(0, t0);
    load_codes(1, t0 + min(1, steps - 1));
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
    __syncthreads();                     // tables and X(t0) visible
    dma_x(1, t0 + min(1, steps - 1));
    __builtin_amdgcn_sched_barrier(0);  // the X loads go out before the code loads
    load_codes(2, t0 + min(2, steps - 1));
    gather(Slice<0>{}, 0);
    read_a(0, Slice<0>{});
    bop = pack_b();
    gather(Slice<1>{}, 0);

    // ---- main loop -----------------------------------------------------------------
    // Step t0 + t uses X buffer and code slot P = t % 3.  Its slices 0..2 issue
    // their MFMAs while reading A of slices 1..3 and gathering for slices 2, 3
    // and slice 0 of step t+1; then the wave waits until X(t+1) (requested one
    // step earlier) has landed, the workgroup barrier publishes it, and slice 3
    // reads A of slice 0 of step t+1 from it and gathers for that step's slice
    // 1.  After the barrier every wave has consumed X(t-1) (its MFMAs read those
    // operands), so that buffer takes X(t+2); the codes of step t+3 go into
    // slot P (its last gathers were issued in slice 1).  Memory loads complete
    // in issue order: after the barrier a step issues X(t+2) and then
    // codes(t+3), so at the next barrier only this step's code loads may still
    // be in flight.  Past the end the indices are clamped; the extra reads land
    // in buffers and registers that are never used.
    auto step = [&](auto pc, int t) {
        constexpr int P = decltype(pc)::value, P1 = (P + 1) % NXB, P2 = (P + 2) % NXB;
        slice(Slice<1>{}, P, Slice<2>{}, P);
        slice(Slice<2>{}, P, Slice<3>{}, P);
        slice(Slice<3>{}, P, Slice<0>{}, P1);
        barrier_after_loads<F::CODE_LOADS>();
        dma_x(P2, t0 + min(t + 2, steps - 1));
        __builtin_amdgcn_sched_barrier(0);  // the X loads go out before the code loads
        load_codes(P, t0 + min(t + 3, steps - 1));
        slice(Slice<0>{}, P1, Slice<1>{}, P1);
    };
    int t = 0;
    for (; t + 2 < steps; t += 3) {
        step(Buf<0>{}, t);
        step(Buf<1>{}, t + 1);
        step(Buf<2>{}, t + 2);
    }
    if (t < steps) step(Buf<0>{}, t);
    if (t + 1 < steps) step(Buf<1>{}, t + 1);
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): no X load may still be writing this workgroup's LDS

    if constexpr (!std::is_same<Prep, NoPrep>::value) {
        __syncthreads();  // every wave is done with the buffers
        before(x0);
        __syncthreads();
    }
    // D layout of a 32x32 block: lane l, item r -> row (r % 4) + 8 * (r / 4) + 4 * (l / 32), column l % 32.
    if constexpr (std::is_invocable<Out, const f32x16(&)[MB]>::value) {
        __syncthreads();
        out(acc);
    } else {
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) out(32 * i + (r & 3) + 8 * (r >> 2) + 4 * g, 32 * wn + j, acc[i][r]);
    }
}

}  // namespace
}  // namespace fqm
