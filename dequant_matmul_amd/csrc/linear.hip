// The product with its epilogue, weights in the per-row table formats:
//   v = W x + bias,   y = residual + act(v)   or   residual + act(v[0..n)) v[n..2n).
//
// Tiles of X rows times W rows on the matrix cores (lut_gemm_tile.h).  Where W
// is two stacked matrices, a wave's 32 rows of W are 16 of the first and the same
// 16 of the second, so that both factors of an output are in the same wave.
// Few tiles are split along K; the parts' sums go through the workspace and a
// second launch adds them in order and applies the epilogue.  Up to 32 rows the weights' stream is the
// work, and other kernels do it: a wave a row of W for one to three rows, 16-row blocks up to eight (the
// gemv kernels with this epilogue), the stream kernel below beyond.
//
// What binds it, on one MI355X: the matrix cores and the tables' gathers beside them for many rows (2048 rows 5120 ->
// 8704 gated 358 to 381 us by the card, 0.96 to 1.02 PFLOP/s, of which the epilogue and the partial round's two
// launches are 60), the weights' stream for few (1 row 17408 -> 5120 15.6 us, 4.3 TB/s of codes and tables; 16 rows 5120 ->
// 17408 gated 43 us and 5 for the sums), launches and the parts' way through memory between (77 rows 4160 -> 1000 9.0 +
// 5.0 us).
#include <algorithm>

#include "linear.h"
#include "lut_gemm_tile.h"

namespace fqm {
namespace {

typedef __attribute__((address_space(3))) float lds_f;

// The epilogue of V neighbouring columns c .. of many rows, what belongs to the columns loaded once.
template <bool GATED, int V>
struct Columns {
    const fqm_epilogue& a;
    int c, n;  // n of the columns are there
    float b[V], wb[V];
    __device__ __forceinline__ Columns(const Linear& p, int first) : a(p.a), c(first), n(max(0, min(V, p.n - first))) {
#pragma unroll
        for (int i = 0; i < V; ++i) b[i] = wb[i] = 0.f;
        if (a.bias && n > 0) {
            load_values<V>(a.bias, a.bias_dtype, c, n, b);
            if (GATED) load_values<V>(a.bias, a.bias_dtype, p.n + c, n, wb);
        }
    }
    __device__ __forceinline__ void row(int64_t m, float (&v)[V], float (&w)[V]) const {
        if (n <= 0) return;
        float r[V];
        if (a.residual) load_values<V>(a.residual, a.res_dtype, m * a.ld_res + c, n, r);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            v[i] += b[i];
            if (GATED) w[i] += wb[i];
        }
        activate<V>(a.act, v);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (GATED) v[i] *= w[i];
            if (a.residual) v[i] += r[i];
        }
        store_values<V>(a.Y, a.y_dtype, m * a.ld_y + c, v, n);
    }
};

// A wave's 32 x 32 blocks of sums, as the matrix instruction leaves them (lane l, item r: row (r % 4) + 8 (r / 4) + 4
// (l / 32), column l % 32), go through LDS of the wave's own to neighbouring outputs on a lane, 8 rows (1 KB) at a time.
template <int R>
__device__ __forceinline__ void put_8_rows(lds8* own, const f32x16& acc) {  // items 4 R .. 4 R + 3
    lds_f* put = (lds_f*)own + 128 * ((threadIdx.x >> 5) & 1) + (threadIdx.x & 31);
#pragma unroll
    for (int r = 0; r < 4; ++r) put[32 * r] = acc[4 * R + r];
}
template <bool GATED, int V>
__device__ __forceinline__ void finish_8_rows(const Columns<GATED, V>& cols, const lds8* own, int64_t m, int rows) {
    const int row = (threadIdx.x & 63) >> 3;
    const lds_f* get = (const lds_f*)own + 32 * row + V * (threadIdx.x & 7);
    float v[V], w[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = get[i], w[i] = GATED ? get[16 + i] : 0.f;
    if (row < rows) cols.row(m + row, v, w);
}

// All MB blocks of a wave, of its own 1024 KB bytes (a multiple of 1 KB) of each of two buffers: as many rows at once
// as these hold, so that the epilogue's code is there few times (it runs once a tile: what it costs is fetching it,
// and choosing the sums by a loop's counter cost 112 selections a block).  m, c: Y's row and the wave's first column;
// rows: how many rows there are from m on.
template <bool GATED, int MB, int KB>
__device__ __forceinline__ void finish_blocks(const Linear& p, lds8* x0, lds8* x1, const f32x16 (&acc)[MB], int64_t m, int c, int rows) {
    constexpr int V = GATED ? 2 : 4, EACH = KB >= 4 ? 4 : KB, ALL = 4 * MB, AT_ONCE = 2 * EACH < ALL ? 2 * EACH : ALL;
    const Columns<GATED, V> cols(p, c + V * (threadIdx.x & 7));
#pragma unroll
    for (int r0 = 0; r0 < ALL; r0 += AT_ONCE) {
#pragma unroll
        for (int r = 0; r < AT_ONCE; ++r) {
            lds8* to = (r < EACH ? x0 : x1) + 1024 * (r % EACH);
            const f32x16& from = acc[(r0 + r) / 4];
            switch ((r0 + r) % 4) {
                case 0: put_8_rows<0>(to, from); break;
                case 1: put_8_rows<1>(to, from); break;
                case 2: put_8_rows<2>(to, from); break;
                default: put_8_rows<3>(to, from); break;
            }
        }
        wave_lds_order();
#pragma unroll 1
        for (int r = 0; r < AT_ONCE; ++r)
            finish_8_rows(cols, (r < EACH ? x0 : x1) + 1024 * (r % EACH), m + 8 * (r0 + r), rows - 8 * (r0 + r));
        wave_lds_order();
    }
}

// Workgroup b: M tile tt % mtiles and N tile nt0 + tt / mtiles, tt = b / ksplit, over the
// K steps of its part b % ksplit.  PARTIAL: the fp32 tile goes to part[b].
template <int BITS, int BM, int NW, bool GATED, bool PARTIAL>
__global__ __launch_bounds__(64 * NW) void linear_tile_kernel(const Linear p, int mtiles, int nt0, int ksplit,
                                                              float* __restrict__ part) {
    constexpr int BN = 32 * NW, OUT = GATED ? BN / 2 : BN;
    constexpr int OWN = BM * 128 / NW;  // of an X buffer, a wave's in the epilogue
    FQM_GEMM_TILE_LDS(BITS, BM, NW);
    const fqm_epilogue& a = p.a;
    const int b = blockIdx.x, tt = b / ksplit, ks = b - tt * ksplit;
    const int mt = tt % mtiles, nt = nt0 + tt / mtiles;
    const int64_t m0 = (int64_t)mt * BM;
    const int rows = (int)min((int64_t)BM, a.M - m0), ksteps = p.K / BK;
    const int t0 = (int)((int64_t)ks * ksteps / ksplit), t1 = (int)((int64_t)(ks + 1) * ksteps / ksplit);
    auto x_off = [&](int row) { return (uint32_t)min(row, rows - 1) * (uint32_t)a.ld_x * 2u; };
    auto tile = [&](auto wr) {
        const uint16_t* X = a.X + m0 * a.ld_x;
        if constexpr (PARTIAL)
            gemm_tile<BITS, BM, NW>(FQM_GEMM_TILE_LDS_ARGS, X, 0, x_off, p.packed, p.ld, p.lut, wr, t0, t1 - t0,
                                    [&](int row, int col, float v) { part[(size_t)b * (BM * BN) + row * BN + col] = v; });
        else
            gemm_tile<BITS, BM, NW>(FQM_GEMM_TILE_LDS_ARGS, X, 0, x_off, p.packed, p.ld, p.lut, wr, t0, t1 - t0,
                                    [&](const f32x16(&acc)[BM / 32]) {
                                        const int wn = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
                                        finish_blocks<GATED, BM / 32, OWN / 1024>(p, (lds8*)s_x0 + OWN * wn, (lds8*)s_x1 + OWN * wn, acc, m0,
                                                                                  nt * OUT + OUT / NW * wn, rows);
                                    });
    };
    if constexpr (GATED) tile(StackedRows{p.n, nt * OUT});
    else tile(RunOfRows{p.N, nt * OUT});
}

// Y of the split tiles: the parts' sums in order, then the epilogue.  4 outputs a thread.
template <int BM, int NW, bool GATED>
__global__ __launch_bounds__(256) void linear_reduce(const Linear p, const float* __restrict__ part, int mtiles, int nt0,
                                                     int ksplit, int64_t groups) {
    constexpr int BN = 32 * NW, OUT = GATED ? BN / 2 : BN;
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (e >= groups) return;
    const int64_t tt = e / (BM * OUT / 4);
    const int rem = (int)(e - tt * (BM * OUT / 4)), row = rem / (OUT / 4), o = 4 * (rem - row * (OUT / 4));
    const int64_t m = (tt % mtiles) * BM + row;
    const int c = (int)(nt0 + tt / mtiles) * OUT + o;
    if (m >= p.a.M || c >= p.n) return;
    typedef float f32x4 __attribute__((ext_vector_type(4)));
    const float* q = part + (size_t)tt * ksplit * (BM * BN) + row * BN + (GATED ? 32 * (o >> 4) + (o & 15) : o);
    float v[4] = {0.f, 0.f, 0.f, 0.f}, w[4] = {0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < ksplit; ++k) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(q + (size_t)k * (BM * BN));
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += x[i];
        if (GATED) {
            const f32x4 y = *reinterpret_cast<const f32x4*>(q + (size_t)k * (BM * BN) + 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] += y[i];
        }
    }
    finish<GATED, 4>(p, m, c, v, w, min(4, p.n - c));
}

// ---- up to 32 rows -----------------------------------------------------------------------
// Here the weights' stream is the work.  A workgroup's 4 waves own 32 rows of W each and share the
// rows of X; K goes by in stages of 128.  Codes and X come by direct global -> LDS loads, a stage
// ahead (a third buffer gained nothing: two workgroups a compute unit cover each other's waits), in whole 64-byte
// pieces of a row: read straight into the operands' layout (24 bytes a lane, a row of W on every second lane) the
// codes cost the address unit 128 accesses for 2 KB and bound the kernel at 28 us for 69 MB; this way they cost 24.
//
// All tiles' stages are one range, cut evenly over the workgroups (two a compute unit): each has the same
// work whatever the shape, and at most two tiles that it shares with others.  Their sums go through the
// workspace, and a second launch adds them in order and applies the epilogue.
//
// LDS layouts, chunks of 16 bytes.  Codes: 6 (6-bit) or 4 chunks a row, a row's chunks turned (6) or XORed (4)
// by its number so that the 64 lanes' reads (row j, half g) meet every bank equally.  X: 16 chunks a row, XORed
// by row % 16.
constexpr int kStreamRows = 32;
constexpr int kStreamWaves = 4;

// Byte of a stage's X (16 MX rows) at which lane j of 32 finds its operand's chunk.  The matrix instruction takes 32 rows:
// with 16, lanes 16 .. 31 read rows 0 .. 15 again, whose sums in their places are never stored.
template <int MX>
constexpr int stream_x_at(int j, int chunk) {
    const int row = j & (16 * MX - 1);
    return 256 * row + 16 * (chunk ^ (row & 15));
}
template <int MX>
constexpr bool stream_x_inside() {
    for (int j = 0; j < 32; ++j)
        for (int chunk = 0; chunk < 16; ++chunk)
            if (stream_x_at<MX>(j, chunk) < 0 || stream_x_at<MX>(j, chunk) + 16 > MX * 4096) return false;
    return true;
}
static_assert(stream_x_inside<1>() && stream_x_inside<2>(), "every lane's operand lies in the stage's X");

// Workgroup g's first stage of all tiles' `total`, and the workgroup that has stage u (32 bits hold total * groups).
__device__ __forceinline__ uint32_t stream_first(uint32_t g, uint32_t total, uint32_t groups) { return g * total / groups; }
__device__ __forceinline__ uint32_t stream_owner(uint32_t u, uint32_t total, uint32_t groups) {
    return ((u + 1) * groups - 1) / total;
}

template <int BITS, int MX, bool GATED>
__device__ __forceinline__ void stream_tiles(const Linear& p, int tiles, float* __restrict__ part) {
    using F = GemmFmt<BITS>;
    constexpr int NW = kStreamWaves, ND = F::ND, OUT = GATED ? 16 : 32, BN = 32 * NW;
    constexpr int MB = (MX + 1) / 2;                  // 32-row blocks of X
    constexpr int CH = BITS == 6 ? 6 : 4;             // chunks of a row's codes per stage
    constexpr int CD = CH / 2;                        // 1 KB loads of a wave's codes per stage
    __shared__ __attribute__((aligned(8192))) uint8_t s_tab[(NW / 2) * F::PLANE];
    __shared__ __attribute__((aligned(16))) uint8_t s_zero[16];
    // objects of their own, so that the compiler sees which reads a load under way does not concern
    __shared__ __attribute__((aligned(16))) uint8_t s_c0[NW * 1024 * CD];
    __shared__ __attribute__((aligned(16))) uint8_t s_c1[NW * 1024 * CD];
    __shared__ __attribute__((aligned(16))) uint8_t s_x0[MX * 4096];
    __shared__ __attribute__((aligned(16))) uint8_t s_x1[MX * 4096];
    lds8* const CS[2] = {(lds8*)s_c0, (lds8*)s_c1};
    lds8* const XS[2] = {(lds8*)s_x0, (lds8*)s_x1};
    const fqm_epilogue& a = p.a;
    const int tid = threadIdx.x, lane = tid & 63, j = lane & 31, g = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int M = (int)a.M, ksteps = p.K / BK, stages = (ksteps + 1) / 2;
    const int total = tiles * stages;
    const int u0 = (int)stream_first(blockIdx.x, total, gridDim.x), u1 = (int)stream_first(blockIdx.x + 1, total, gridDim.x);

    // X: load u of wave w fills rows 4 (MX w + u) .. + 3, lane l the place l % 16 of row l / 16
    const __amdgpu_buffer_rsrc_t xrsrc = __builtin_amdgcn_make_buffer_rsrc((void*)a.X, (short)0, 0x7fffffff, 0x00020000);
    uint32_t xrow[MX], xin[MX];
#pragma unroll
    for (int u = 0; u < MX; ++u) {
        const int row = 4 * (MX * wave + u) + (lane >> 4);
        xrow[u] = (uint32_t)min(row, M - 1) * (uint32_t)a.ld_x * 2u;
        xin[u] = 16u * ((lane & 15) ^ (row & 15));
    }
    // operand reads: row j, logical chunk 8 h + 4 g + q
    int aoff[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) aoff[c] = stream_x_at<MX>(j, 8 * (c >> 2) + 4 * g + (c & 3));
    // code reads of lane (j, g): its 24 (16) bytes of both steps of a stage
    constexpr int CR = BITS == 6 ? 6 : 2;
    int coff[CR];
#pragma unroll
    for (int i = 0; i < CR; ++i) {
        if constexpr (BITS == 6) {
            const int at = 48 * (i / 3) + 24 * g + 8 * (i % 3);  // byte of the row's 96
            coff[i] = 96 * j + 16 * ((at / 16 + (j >> 3)) % 6) + (at & 15);
        } else {
            coff[i] = 64 * j + 16 * ((2 * i + g) ^ ((j >> 2) & 3));
        }
    }
    uint32_t cmask = (uint32_t)(F::ENTRIES - 1) << 7;
    asm volatile("" : "+v"(cmask));  // in a VGPR: (v & mask) | base is one v_and_or_b32
    const uint32_t tbase = (uint32_t)F::PLANE * (wave >> 1) + 4u * j + 2u * (wave & 1);
    lds8* const TAB = (lds8*)s_tab;

    for (int u = u0; u < u1;) {
        const int nt = u / stages, s0 = u - nt * stages, s1 = min(stages, s0 + (u1 - u));
        const auto wr = [&] {
            if constexpr (GATED) return StackedRows{p.n, OUT * NW * nt};
            else return RunOfRows{p.N, BN * nt};
        }();
        __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): from here on only the loads below are counted
        __syncthreads();                     // every wave is done with the last tile's LDS
        // codes: load u of a wave fills 64 chunks, in order of (row, place)
        const uint8_t* base = p.packed + (int64_t)wr.row(32 * wave) * p.ld;
        const __amdgpu_buffer_rsrc_t crsrc = __builtin_amdgcn_make_buffer_rsrc((void*)base, (short)0, 0x7fffffff, 0x00020000);
        uint32_t crow[CD], cin[CD];
#pragma unroll
        for (int v = 0; v < CD; ++v) {
            const int e = 64 * v + lane, row = e / CH, place = e - row * CH;
            crow[v] = (uint32_t)((int64_t)(wr.row(32 * wave + row) - wr.row(32 * wave)) * p.ld);
            cin[v] = 16u * (BITS == 6 ? (place + 6 - (row >> 3)) % 6 : place ^ ((row >> 2) & 3));
        }
        // past a row's end (the second half of a last stage, where K is an odd number of steps): a chunk of codes
        // again, and for X an offset past the buffer, which loads zeros
        const uint32_t clast = (uint32_t)(F::STEP_BYTES * ksteps - 16), xend = 2u * (uint32_t)p.K;
        auto load_stage = [&](int ring, int s) {
#pragma unroll
            for (int v = 0; v < CD; ++v)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(crsrc, (lvoid*)(CS[ring] + 1024 * (CD * wave + v)), 16,
                                                         crow[v] + min(cin[v] + (uint32_t)s * (16u * CH), clast), 0, 0, 0);
#pragma unroll
            for (int v = 0; v < MX; ++v) {
                const uint32_t at = xin[v] + (uint32_t)s * 256u;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(xrsrc, (lvoid*)(XS[ring] + 1024 * (MX * wave + v)), 16,
                                                         at < xend ? xrow[v] + at : 0xffffff00u, 0, 0, 0);
            }
        };
        // tables, bank-sliced as in the tiles
        {
            constexpr int EPT = F::ENTRIES / 8;
            uint32_t tv[BN * 8 / (64 * NW)][EPT / 2];
#pragma unroll
            for (int v = 0; v < BN * 8 / (64 * NW); ++v) {
                const int i = tid + 64 * NW * v;
                const uint32_t* src = reinterpret_cast<const uint32_t*>(p.lut + (int64_t)wr.row(i >> 3) * F::ENTRIES + EPT * (i & 7));
                if constexpr (EPT == 8) {
                    const u32x4 q = *reinterpret_cast<const u32x4*>(src);
                    tv[v][0] = q[0], tv[v][1] = q[1], tv[v][2] = q[2], tv[v][3] = q[3];
                } else {
                    tv[v][0] = *src;
                }
            }
            load_stage(0, s0);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int v = 0; v < BN * 8 / (64 * NW); ++v) {
                const int i = tid + 64 * NW * v, r = i >> 3;
                lds8* dst = TAB + F::PLANE * (r >> 6) + 4 * (r & 31) + 2 * ((r >> 5) & 1) + 128 * EPT * (i & 7);
#pragma unroll
                for (int e = 0; e < EPT; ++e) *(lds16*)(dst + 128 * e) = (uint16_t)(tv[v][e >> 1] >> (16 * (e & 1)));
            }
        }
        if (tid == 0) *(__attribute__((address_space(3))) uint32_t*)s_zero = 0u;

        f32x16 acc[MB];
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][r] = 0.f;
        uint32_t mask1 = cmask, base1 = tbase;
        auto step = [&](auto rc, auto hc) {
            constexpr int ring = decltype(rc)::value, h = decltype(hc)::value;
            uint32_t cw[ND];
            lds8* from = CS[ring] + 1024 * CD * wave;
#pragma unroll
            for (int i = 0; i < ND / 2; ++i) {
                if constexpr (BITS == 6) {
                    const u32x2 d = *(__attribute__((address_space(3))) const u32x2*)(from + coff[3 * h + i]);
                    cw[2 * i] = d[0], cw[2 * i + 1] = d[1];
                } else if (i == 0) {
                    const u32x4 d = *(lds128c*)(from + coff[h]);
                    cw[0] = d[0], cw[1] = d[1], cw[2] = d[2], cw[3] = d[3];
                }
            }
            auto slice = [&](auto qc) {
                constexpr int q = decltype(qc)::value;
                uint32_t ad[8], wv[8];
                if constexpr (h == 0) slice_addrs<BITS, q>(cw, cmask, tbase, ad);
                else slice_addrs<BITS, q>(cw, mask1, base1, ad);
#pragma unroll
                for (int e = 0; e < 8; ++e) wv[e] = *(lds16c*)(TAB + ad[e]);
                u32x4 bw;
#pragma unroll
                for (int e = 0; e < 4; ++e) bw[e] = __builtin_amdgcn_perm(wv[2 * e + 1], wv[2 * e], 0x05040100u);
#pragma unroll
                for (int i = 0; i < MB; ++i) {
                    const bf16x8 x = __builtin_bit_cast(bf16x8, *(lds128c*)(XS[ring] + aoff[4 * h + q] + 8192 * i));
                    acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, __builtin_bit_cast(bf16x8, bw), acc[i], 0, 0, 0);
                }
            };
            slice(Slice<0>{});
            slice(Slice<1>{});
            slice(Slice<2>{});
            slice(Slice<3>{});
        };
        auto stage = [&](auto rc, int s) {
            constexpr int R = decltype(rc)::value;
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            load_stage(1 - R, min(s + 1, s1 - 1));
            const bool none = 2 * s + 1 >= ksteps;  // no second half: its weights are the zero
            mask1 = none ? 0u : cmask;
            base1 = none ? (uint32_t)(uintptr_t)(lds8*)s_zero - (uint32_t)(uintptr_t)TAB : tbase;
            step(rc, Slice<0>{});
            step(rc, Slice<1>{});
        };
        int s = s0;
        for (; s + 1 < s1; s += 2) {
            stage(Buf<0>{}, s);
            stage(Buf<1>{}, s + 1);
        }
        if (s < s1) stage(Buf<0>{}, s);
        __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): no load may still be writing this workgroup's LDS
        if (s0 == 0 && s1 == stages) {
            __syncthreads();
            finish_blocks<GATED, MB, MX>(p, XS[0] + 1024 * MX * wave, XS[1] + 1024 * MX * wave, acc, 0, OUT * (NW * nt + wave), M);
        } else {
            float* q = part + ((size_t)2 * blockIdx.x + (u != u0)) * M * BN + 32 * wave + j;
#pragma unroll
            for (int i = 0; i < MB; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int row = 32 * i + (r & 3) + 8 * (r >> 2) + 4 * g;
                    if (row < M) q[(size_t)row * BN] = acc[i][r];
                }
        }
        u += s1 - s0;
    }
}

template <int BITS, int MX, bool GATED>
__global__ __launch_bounds__(64 * kStreamWaves) void linear_stream_kernel(const Linear p, int tiles, float* __restrict__ part) {
    stream_tiles<BITS, MX, GATED>(p, tiles, part);
}

// Y of the tiles that workgroups share: their sums in order, then the epilogue.  Workgroup: 1024 outputs of a tile
// at most, 4 a thread.
template <bool GATED>
__global__ __launch_bounds__(256) void linear_stream_sum(const Linear p, const float* __restrict__ part, int tiles, int groups,
                                                         int per_tile) {
    constexpr int BN = 32 * kStreamWaves, OUT = GATED ? BN / 2 : BN, AT_ONCE = 4;
    typedef float f32x4 __attribute__((ext_vector_type(4)));
    const int nt = blockIdx.x / per_tile, e = (blockIdx.x - nt * per_tile) * 256 + threadIdx.x;
    const int M = (int)p.a.M, m = e / (OUT / 4), o = 4 * (e % (OUT / 4)), c = OUT * nt + o;
    const uint32_t stages = (uint32_t)(p.K / BK + 1) / 2, total = tiles * stages, lo = nt * stages;
    const int g0 = (int)stream_owner(lo, total, groups), g1 = (int)stream_owner(lo + stages - 1, total, groups);
    if (g0 == g1 || m >= M || c >= p.n) return;  // g0 == g1: that workgroup has finished the tile
    const bool later = stream_first(g0, total, groups) < lo;  // g0's second place: its last tile
    const float* q = part + (size_t)m * BN + (GATED ? 32 * (o >> 4) + (o & 15) : o);
    const size_t each = (size_t)M * BN;
    float v[4] = {0.f, 0.f, 0.f, 0.f}, w[4] = {0.f, 0.f, 0.f, 0.f};
    for (int g = g0; g <= g1; g += AT_ONCE) {
        f32x4 x[AT_ONCE], y[AT_ONCE];
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            const float* from = q + each * (2 * min(g + k, g1) + (g + k == g0 && later));
            x[k] = *reinterpret_cast<const f32x4*>(from);
            if (GATED) y[k] = *reinterpret_cast<const f32x4*>(from + 16);
        }
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] += g + k <= g1 ? x[k][i] : 0.f;
                if (GATED) w[i] += g + k <= g1 ? y[k][i] : 0.f;
            }
    }
    finish<GATED, 4>(p, m, c, v, w, min(4, p.n - c));
}

// Of the current device (without one, an MI355X's).
int compute_units() {
    int dev = 0, cus = 0;
    if (hipGetDevice(&dev) != hipSuccess || hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess) {
        (void)hipGetLastError();
        return 256;
    }
    return std::max(cus, 1);
}

struct StreamPlan {
    int tiles, groups;
    bool shared;  // whether some tile is
    size_t part_bytes;
};

StreamPlan stream_plan(int64_t N, int64_t K, int64_t M, bool gated) {
    StreamPlan p;
    const int64_t n = gated ? N / 2 : N, per = (gated ? 16 : 32) * kStreamWaves, stages = (K / BK + 1) / 2;
    p.tiles = (int)((n + per - 1) / per);
    const int64_t total = p.tiles * stages;
    p.groups = (int)std::min<int64_t>(2 * compute_units(), (total + 3) / 4);
    p.shared = total % p.groups || total / p.groups % stages;
    p.part_bytes = p.shared ? (size_t)2 * p.groups * M * 32 * kStreamWaves * 4 : 0;
    return p;
}

template <int BITS, int MX, bool GATED>
hipError_t launch_stream(const Linear& p, float* part, hipStream_t s) {
    const StreamPlan plan = stream_plan(p.N, p.K, p.a.M, GATED);
    hipLaunchKernelGGL((linear_stream_kernel<BITS, MX, GATED>), dim3((unsigned)plan.groups), dim3(64 * kStreamWaves), 0, s, p,
                       plan.tiles, part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !plan.shared) return e;
    const int per_tile = ((int)p.a.M * (GATED ? 4 : 8) * kStreamWaves + 255) / 256;
    hipLaunchKernelGGL(linear_stream_sum<GATED>, dim3((unsigned)(plan.tiles * per_tile)), dim3(256), 0, s, p, part, plan.tiles,
                       plan.groups, per_tile);
    return hipGetLastError();
}

// The loads' 32-bit offsets reach both matrices of a tile, and the stages are counted in 32 bits.
bool stream_path(const Linear& p) {
    const StreamPlan plan = stream_plan(p.N, p.K, p.a.M, p.a.gated);
    return p.a.M <= kStreamRows && (p.a.gated ? (int64_t)(p.n + 32) * p.ld : 32 * p.ld) < 0x7fffffff &&
           (int64_t)plan.tiles * ((p.K / BK + 1) / 2 + 1) * plan.groups <= 0x7fffffff;
}

// cols == 0: the sums are of nothing.
__global__ __launch_bounds__(256) void linear_of_nothing(const Linear p, int64_t outputs) {
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (e >= outputs) return;
    const int64_t m = e / p.n;
    const int c = (int)(e - m * p.n);
    float v[2] = {0.f, 0.f};
    const float w[2] = {0.f, 0.f};
    if (p.a.gated) finish<true, 2>(p, m, c, v, w, 1);
    else finish<false, 2>(p, m, c, v, w, 1);
}

// Tiles and what is split.  64- and 128-row tiles (4 waves; several a compute unit) are all split along K alike; of
// 256-row tiles (8 waves, one a compute unit) whole rounds run as one launch, and the N tiles that are left for a
// partial round are split into as many parts as make that round shortest.
struct LinearPlan {
    int bm, nw, mtiles, ntiles;
    int nt_main;      // N tiles [0, nt_main) are not split
    int ksplit;       // K parts of the others
    int64_t tail;     // the others
    double us;        // what it should take
    size_t part_bytes;
};

// The time is that of the compute unit with the most workgroups: its K steps (and 6 for each workgroup's start) at
// what one takes there, more than its share where a workgroup is alone, and the parts' way through memory with a
// second launch.
LinearPlan tile_plan(int bm, int64_t N, int64_t K, int64_t M, bool gated) {
    LinearPlan p;
    p.bm = bm;
    p.nw = bm == 256 ? 8 : 4;
    const int64_t per = gated ? 16 * p.nw : 32 * p.nw, n = gated ? N / 2 : N, steps = K / BK, cus = compute_units();
    const double step_us = bm == 64 ? 0.42 : bm == 128 ? 0.5 : 1.7, alone_us = bm == 64 ? 0.5 : bm == 128 ? 0.6 : 1.7, start = 6;
    auto steps_us = [&](int64_t groups, int64_t of) {
        const int64_t each = (groups + cus - 1) / cus;
        return (each == 1 ? alone_us : each * step_us) * (of + start);
    };
    p.mtiles = (int)((M + bm - 1) / bm);
    p.ntiles = (int)((n + per - 1) / per);
    const int64_t tiles = (int64_t)p.mtiles * p.ntiles;
    p.nt_main = bm == 256 ? (int)(tiles / cus * cus / p.mtiles) : 0;
    p.tail = (int64_t)(p.ntiles - p.nt_main) * p.mtiles;
    p.us = 1e30;
    const double tile_bytes = 4.0 * bm * 32 * p.nw;
    for (int64_t k = 1; k <= std::max<int64_t>(1, std::min<int64_t>(steps / 4, bm == 256 ? steps / 8 : 8)); ++k) {
        const double parts = k == 1 ? 0 : 2 * k * p.tail * tile_bytes;
        if (k > 1 && parts > 2 * (256 << 20)) break;
        const double us = p.tail == 0 ? 0 : steps_us(p.tail * k, (steps + k - 1) / k) + (k > 1 ? 3 + parts / 8e6 : 0);
        if (us < p.us) p.us = us, p.ksplit = (int)k;
    }
    if (tiles > p.tail) p.us += steps_us(tiles - p.tail, steps);
    if (p.ksplit == 1) p.nt_main = p.ntiles, p.tail = 0;
    p.part_bytes = p.ksplit > 1 ? (size_t)(p.tail * p.ksplit * tile_bytes) : 0;
    return p;
}

// The height whose time should be the least.  Measured on one MI355X, us with 64 / 128 / 256 rows (no epilogue but SiLU
// where gated, three sets of weights in turn): 6-bit 5120 -> 17408 at 64 rows 35 / - / -, 96 rows 59 / 44 / 60, 128 rows 61 /
// 47 / -, 192 rows 68 / 82 / 65, 256 rows 100 / 88 / 68, 320 rows 105 / 94 / 124, 512 rows 165 / 142 / 133; its gated form
// with twice the rows of W at 128 rows 114 / 95 / -, 256 rows 177 / 152 / 134, 512 rows 311 / 245 / 200; 6-bit 17408 -> 5120
// at 128 rows 47 / 39 / -, 256 rows 85 / 68 / 67, 512 rows 161 / 123 / 106; 4-bit 4160 -> 1000 at 96 rows 12.8 / 14.0 / 22,
// 512 rows 19.5 / 21.4 / 29.  Of these the rule takes the best or one within 5 %, but for 256 rows gated (128: 14 % more), 512
// rows 5120 -> 17408 (128: 6 %) and 512 rows 4160 -> 1000 (128: 10 %).
LinearPlan linear_plan(int64_t N, int64_t K, int64_t M, bool gated) {
    LinearPlan best = tile_plan(64, N, K, M, gated);
    for (const int bm : {128, 256}) {
        if (M <= bm / 2) break;
        const LinearPlan p = tile_plan(bm, N, K, M, gated);
        if (p.us < best.us) best = p;
    }
    return best;
}

template <int BITS, int BM, int NW, bool GATED>
hipError_t launch_tiles(const Linear& p, const LinearPlan& plan, float* part, hipStream_t s) {
    const int64_t main_tiles = (int64_t)plan.nt_main * plan.mtiles, grid = plan.tail * plan.ksplit;
    if (main_tiles > 0x7fffffff || grid > 0x7fffffff) return hipErrorInvalidValue;
    hipError_t e = hipSuccess;
    if (main_tiles > 0) {
        hipLaunchKernelGGL((linear_tile_kernel<BITS, BM, NW, GATED, false>), dim3((unsigned)main_tiles), dim3(64 * NW), 0, s, p,
                           plan.mtiles, 0, 1, nullptr);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (plan.tail == 0) return e;
    hipLaunchKernelGGL((linear_tile_kernel<BITS, BM, NW, GATED, true>), dim3((unsigned)grid), dim3(64 * NW), 0, s, p,
                       plan.mtiles, plan.nt_main, plan.ksplit, part);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const int64_t groups = plan.tail * BM * (GATED ? 4 * NW : 8 * NW);
    if ((groups + 255) / 256 > 0x7fffffff) return hipErrorInvalidValue;
    hipLaunchKernelGGL((linear_reduce<BM, NW, GATED>), dim3((unsigned)((groups + 255) / 256)), dim3(256), 0, s, p, part,
                       plan.mtiles, plan.nt_main, plan.ksplit, groups);
    return hipGetLastError();
}

template <int BITS, bool GATED>
hipError_t launch_tile_bits(const Linear& p, void* ws, hipStream_t s) {
    float* part = static_cast<float*>(ws);
    const LinearPlan plan = linear_plan(p.N, p.K, p.a.M, GATED);
    if (plan.bm == 64) return launch_tiles<BITS, 64, 4, GATED>(p, plan, part, s);
    if (plan.bm == 128) return launch_tiles<BITS, 128, 4, GATED>(p, plan, part, s);
    return launch_tiles<BITS, 256, 8, GATED>(p, plan, part, s);
}

template <int BITS, bool GATED>
hipError_t launch_stream_bits(const Linear& p, void* ws, hipStream_t s) {
    float* part = static_cast<float*>(ws);
    return p.a.M <= 16 ? launch_stream<BITS, 1, GATED>(p, part, s) : launch_stream<BITS, 2, GATED>(p, part, s);
}

Linear linear_of(const fqm_weights& w, const fqm_epilogue& a) {
    Linear p;
    p.a = a;
    const bool six = w.format == FQM_LUT6;
    p.packed = six ? w.lut6.packed : w.lut4.packed;
    p.ld = six ? w.lut6.ld : w.lut4.ld;
    p.lut = six ? w.lut6.lut : w.lut4.lut;
    p.N = (int)w.rows;
    p.K = (int)w.cols;
    p.n = a.gated ? p.N / 2 : p.N;
    return p;
}

// Measured: 1 row 17408 -> 5120 15.6 us on a wave a row and 31 on the tiles; 8 rows 5120 -> 17408 24 us in 16-row blocks,
// 27 on the stream kernel; 16 rows 5120 -> 17408 gated 46 us on the stream kernel, 66 on the tiles.
// Three rows, a wave a row of W / 16-row blocks, 6-bit (4-bit): below 2^26 weights the waves win, 2048 -> 4096 5.0 / 11.0 (4.6 /
// 9.7), 5120 -> 5120 8.8 / 14.1 (8.4 / 13.1), 5120 -> 12288 17.6 / 20.2 (16.2 / 18.4); from about 10^8 on the blocks do, 12288 ->
// 8192 30 / 25 (29 / 22), 9216 -> 17297 41 / 36 (40 / 32).  Between them it goes by how the blocks' K parts fill the card:
// 8192 -> 8192 18.9 / 20.2 (18.2 / 18.0), 5120 -> 14336 19.4 / 22.8 (18.4 / 20.7), 12288 -> 6144 23.8 / 22.6 (23.1 / 20.3), 9216 ->
// 8192 24.1 / 22.3 (23.3 / 19.1), 5120 -> 16384 22.6 / 19.8 (20.2 / 17.9), 5120 -> 17408 23.3 / 23.0 (21.4 / 20.1).  Two
// rows 9216 -> 17297 27 / 32 (6-bit 32 / 38).
enum class Path { rows, mfma, stream, tiles };
Path path_of(const fqm_weights& w, const Linear& p) {
    const bool blocks = p.a.M <= 8 && lut_gemv_mfma_supported(w, (int)std::max<int64_t>(p.a.M, 2));
    if (blocks && p.a.M >= 3 && w.rows * w.cols >= 1 << 26) return Path::mfma;
    if (p.a.M <= 3 && (w.format == FQM_LUT6 ? lut6_gemv_rows_path(w, (int)p.a.M) : lut4_gemv_rows_path(w, (int)p.a.M))) return Path::rows;
    if (blocks) return Path::mfma;
    return stream_path(p) ? Path::stream : Path::tiles;
}
}  // namespace

size_t linear_workspace(const fqm_weights& w, const fqm_epilogue& a) {
    if (w.cols == 0) return 0;
    const Linear p = linear_of(w, a);
    switch (path_of(w, p)) {
        case Path::rows: return 0;
        case Path::mfma: return lut_linear_mfma_workspace(p);
        case Path::stream: return stream_plan(p.N, p.K, a.M, a.gated).part_bytes;
        default: return linear_plan(p.N, p.K, a.M, a.gated).part_bytes;
    }
}

hipError_t launch_linear(const fqm_weights& w, const fqm_epilogue& a, void* ws, hipStream_t s) {
    const Linear p = linear_of(w, a);
    if (p.K == 0) {
        const int64_t outputs = a.M * p.n, grid = (outputs + 255) / 256;
        if (grid > 0x7fffffff) return hipErrorInvalidValue;
        hipLaunchKernelGGL(linear_of_nothing, dim3((unsigned)grid), dim3(256), 0, s, p, outputs);
        return hipGetLastError();
    }
    const bool six = w.format == FQM_LUT6;
    switch (path_of(w, p)) {
        case Path::rows: return six ? launch_lut6_linear(p, s) : launch_lut4_linear(p, s);
        case Path::mfma: return launch_lut_linear_mfma(p, six, static_cast<float*>(ws), s);
        case Path::stream:
            if (six) return a.gated ? launch_stream_bits<6, true>(p, ws, s) : launch_stream_bits<6, false>(p, ws, s);
            return a.gated ? launch_stream_bits<4, true>(p, ws, s) : launch_stream_bits<4, false>(p, ws, s);
        default:
            if (six) return a.gated ? launch_tile_bits<6, true>(p, ws, s) : launch_tile_bits<6, false>(p, ws, s);
            return a.gated ? launch_tile_bits<4, true>(p, ws, s) : launch_tile_bits<4, false>(p, ws, s);
    }
}

}  // namespace fqm
