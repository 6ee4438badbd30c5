// C ABI: argument checks on the host, then stream-ordered launches.
// Nothing here allocates, synchronises or keeps state between calls.
#include <stdlib.h>
#include <string.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <mutex>

#include "fqm_layer.h"

using namespace fqm;

namespace {

// ---- the static scratch of fqm_gemv_static ----------------------------------
// One array per GPU the library runs on, held until the process ends.  Host
// code never uses the array's name as an address (on the host it is only a
// stand-in): each device's address is looked up once, with that device
// current, and kept in scratch_addr.
__device__ __align__(256) uint8_t scratch[FQM_STATIC_SCRATCH_BYTES];

constexpr int kMaxDevices = 64;
std::atomic<void*> scratch_addr[kMaxDevices];
std::mutex scratch_mu;

// The current device's copy of `scratch`.
hipError_t scratch_for_current_device(void** out) {
    int dev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return hipErrorInvalidDevice;
    void* p = scratch_addr[dev].load(std::memory_order_acquire);
    if (!p) {
        std::lock_guard<std::mutex> lock(scratch_mu);
        p = scratch_addr[dev].load(std::memory_order_relaxed);
        if (!p) {
            e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
            if (e != hipSuccess) return e;
            if (!p) return hipErrorInvalidSymbol;
            scratch_addr[dev].store(p, std::memory_order_release);
        }
    }
    *out = p;
    return hipSuccess;
}

// ---- debug checks --------------------------------------------------------------
// -1 until the first call reads FQM_DEBUG; then 0 (off) or 1 (on).
std::atomic<int> debug_state{-1};

bool debug_on() {
    int v = debug_state.load(std::memory_order_relaxed);
    if (v < 0) {
        const char* e = getenv("FQM_DEBUG");
        const int from_env = (e && *e && strcmp(e, "0") != 0) ? 1 : 0;
        int expected = -1;
        debug_state.compare_exchange_strong(expected, from_env);
        v = debug_state.load(std::memory_order_relaxed);
    }
    return v > 0;
}

// [p, p + bytes) lies inside one device allocation (nothing to check when
// bytes <= 0).
bool in_allocation(const void* p, int64_t bytes) {
    if (bytes <= 0) return true;
    if (!p) return false;
    hipDeviceptr_t base = nullptr;
    size_t size = 0;
    if (hipMemGetAddressRange(&base, &size, const_cast<void*>(p)) != hipSuccess) {
        (void)hipGetLastError();  // not device memory: clear the sticky error
        return false;
    }
    const uintptr_t b = reinterpret_cast<uintptr_t>(base), q = reinterpret_cast<uintptr_t>(p);
    return q >= b && (uint64_t)(q - b) + (uint64_t)bytes <= (uint64_t)size;
}

// Bytes that `rows` rows `ld` apart span when the last one needs `last` bytes.
inline int64_t span(int64_t rows, int64_t ld, int64_t last) { return rows > 0 ? (rows - 1) * ld + last : 0; }

// Every buffer of a descriptor (already checked by check_weights) at the
// extent the kernels may touch.
fqm_status check_weight_buffers(const fqm_weights& w) {
    const int64_t R = w.rows, C = w.cols;
    if (R == 0) return FQM_OK;
    bool ok = true;
    switch (w.format) {
        case FQM_LUT6:
            ok = in_allocation(w.lut6.packed, span(R, w.lut6.ld, C * 3 / 4)) && in_allocation(w.lut6.lut, R * 128);
            break;
        case FQM_LUT4:
            ok = in_allocation(w.lut4.packed, span(R, w.lut4.ld, C / 2)) && in_allocation(w.lut4.lut, R * 32);
            break;
        case FQM_FABQ: {
            const fqm_fabq& f = w.fabq;
            const int64_t n_lo = R - f.n_hi, nb = C / f.blocksize;
            const int hb = f.hi_bits ? f.hi_bits : 4;
            ok = in_allocation(f.row_of, R * 4);
            if (f.n_hi > 0)
                ok = ok && in_allocation(f.q4, span(f.n_hi, f.ld_q4, C * hb / 8)) && in_allocation(f.s_hi, f.n_hi * 2);
            if (n_lo > 0) {
                ok = ok && in_allocation(f.signs, span(n_lo, f.ld_signs, C / 8)) &&
                     in_allocation(f.s_blk, n_lo * nb * 2) && in_allocation(f.idx, span(n_lo, f.ld_idx, (nb + 1) / 2));
                if (f.cb_mode == FQM_CB_SCALAR16) ok = ok && in_allocation(f.codebook, 16 * 2);
                if (f.cb_mode == FQM_CB_TIERED) ok = ok && in_allocation(f.codebook, 4 * 64 * 2);
                if (f.cb_mode == FQM_CB_VECTOR) ok = ok && in_allocation(f.vcodebook, 4 * 64 * 128 * 4);
                if (f.cb_mode != FQM_CB_SCALAR16) ok = ok && in_allocation(f.tier, n_lo);
            }
            break;
        }
        case FQM_MDBF: {
            const fqm_mdbf& f = w.mdbf;
            for (int p = 0; p < f.P && ok; ++p) {
                const fqm_mdbf_path& q = f.path[p];
                ok = in_allocation(q.S_A, span(R, q.ld_A, ((f.r + 7) / 8 + 15) & ~15)) &&
                     in_allocation(q.S_B, span(f.r, q.ld_B, (C / 8 + 15) & ~15)) &&
                     in_allocation(q.A_amp, R * f.l * 2) && in_allocation(q.B_amp, C * f.l * 2) &&
                     in_allocation(q.Q_U, (int64_t)f.r * f.l * 2) && in_allocation(q.Q_V, (int64_t)f.r * f.l * 2);
            }
            break;
        }
        default:
            break;
    }
    return ok ? FQM_OK : FQM_E_BOUNDS;
}

// After a call's launches: with the checks on (and the stream not being
// captured), wait for the stream and turn a kernel failure into FQM_E_HIP.
fqm_status debug_finish(fqm_status st, hipStream_t s) {
    if (st != FQM_OK || !debug_on()) return st;
    hipStreamCaptureStatus cs = hipStreamCaptureStatusNone;
    if (hipStreamIsCapturing(s, &cs) != hipSuccess) return FQM_E_HIP;
    if (cs != hipStreamCaptureStatusNone) return st;
    if (hipStreamSynchronize(s) != hipSuccess || hipGetLastError() != hipSuccess) return FQM_E_HIP;
    return st;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool ld_ok(int64_t ld, int64_t need) { return ld >= need && (ld & 15) == 0; }
inline hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }
inline fqm_status hip_status(hipError_t e) { return e == hipSuccess ? FQM_OK : FQM_E_HIP; }

// Checks a descriptor; on success returns FQM_OK.  Only host memory is read.
fqm_status check_weights(const fqm_weights* w) {
    if (!w) return FQM_E_NULL;
    if (w->rows < 0 || w->cols < 0) return FQM_E_SHAPE;
    switch (w->format) {
        case FQM_LUT6: {
            const fqm_lut6& f = w->lut6;
            if (w->cols % 64) return FQM_E_SHAPE;
            if (w->rows == 0) return FQM_OK;
            if (!f.packed || !f.lut) return FQM_E_NULL;
            if (!aligned16(f.packed) || !aligned16(f.lut)) return FQM_E_ALIGN;
            if (f.ld < w->cols * 3 / 4) return FQM_E_SHAPE;
            if (f.ld & 15) return FQM_E_ALIGN;
            return FQM_OK;
        }
        case FQM_LUT4: {
            const fqm_lut4& f = w->lut4;
            if (w->cols % 64) return FQM_E_SHAPE;
            if (w->rows == 0) return FQM_OK;
            if (!f.packed || !f.lut) return FQM_E_NULL;
            if (!aligned16(f.packed) || !aligned16(f.lut)) return FQM_E_ALIGN;
            if (f.ld < w->cols / 2) return FQM_E_SHAPE;
            if (f.ld & 15) return FQM_E_ALIGN;
            return FQM_OK;
        }
        case FQM_FABQ: {
            const fqm_fabq& f = w->fabq;
            const int bs = f.blocksize;
            if (bs != 16 && bs != 32 && bs != 64 && bs != 128 && bs != 256 && bs != 512) return FQM_E_FORMAT;
            if (f.hi_bits != 0 && f.hi_bits != 4 && f.hi_bits != 8) return FQM_E_FORMAT;
            if (f.cb_mode < FQM_CB_SCALAR16 || f.cb_mode > FQM_CB_VECTOR) return FQM_E_FORMAT;
            if (f.cb_mode != FQM_CB_SCALAR16 && (f.cb_base < 0 || f.cb_base > 48 || (f.cb_base & 15)))
                return FQM_E_FORMAT;
            if (w->cols % bs) return FQM_E_SHAPE;
            if (f.n_hi < 0 || f.n_hi > w->rows) return FQM_E_SHAPE;
            if (w->rows == 0) return FQM_OK;
            const int64_t n_lo = w->rows - f.n_hi;
            const int64_t nb = w->cols / bs;
            const int hb = f.hi_bits ? f.hi_bits : 4;
            if (!f.row_of) return FQM_E_NULL;
            if (!aligned16(f.row_of)) return FQM_E_ALIGN;
            if (f.n_hi > 0) {
                if (!f.q4 || !f.s_hi) return FQM_E_NULL;
                if (!aligned16(f.q4) || !aligned16(f.s_hi)) return FQM_E_ALIGN;
                if (f.ld_q4 < w->cols * hb / 8) return FQM_E_SHAPE;
                if (f.ld_q4 & 15) return FQM_E_ALIGN;
            }
            if (n_lo > 0) {
                if (!f.signs || !f.s_blk || !f.idx) return FQM_E_NULL;
                if (f.cb_mode == FQM_CB_VECTOR ? !f.vcodebook : !f.codebook) return FQM_E_NULL;
                if (f.cb_mode != FQM_CB_SCALAR16 && !f.tier) return FQM_E_NULL;
                if (!aligned16(f.signs) || !aligned16(f.s_blk) || !aligned16(f.idx) ||
                    (f.codebook && !aligned16(f.codebook)) || (f.tier && !aligned16(f.tier)) ||
                    (f.vcodebook && !aligned16(f.vcodebook)))
                    return FQM_E_ALIGN;
                if (f.ld_signs < w->cols / 8 || f.ld_idx < (nb + 1) / 2) return FQM_E_SHAPE;
                if ((f.ld_signs & 15) || (f.ld_idx & 15)) return FQM_E_ALIGN;
            }
            return FQM_OK;
        }
        case FQM_MDBF: {
            const fqm_mdbf& f = w->mdbf;
            if (f.l < 1 || f.l > 16 || (f.P != 1 && f.P != 2)) return FQM_E_FORMAT;
            if (f.r < 1 || f.r > 65536) return FQM_E_FORMAT;
            if (w->cols % 32) return FQM_E_SHAPE;
            if (w->rows == 0) return FQM_OK;
            for (int p = 0; p < f.P; ++p) {
                const fqm_mdbf_path& q = f.path[p];
                if (!q.S_A || !q.S_B || !q.A_amp || !q.B_amp || !q.Q_U || !q.Q_V) return FQM_E_NULL;
                if (!aligned16(q.S_A) || !aligned16(q.S_B) || !aligned16(q.A_amp) ||
                    !aligned16(q.B_amp) || !aligned16(q.Q_U) || !aligned16(q.Q_V))
                    return FQM_E_ALIGN;
                if (q.ld_A < (f.r + 7) / 8 || q.ld_B < w->cols / 8) return FQM_E_SHAPE;
                if ((q.ld_A & 15) || (q.ld_B & 15)) return FQM_E_ALIGN;
            }
            return FQM_OK;
        }
        default:
            return FQM_E_FORMAT;
    }
}

}  // namespace

extern "C" {

int32_t fqm_version(void) { return FQM_VERSION; }

int32_t fqm_set_debug(int32_t on) {
    const int prev = debug_on() ? 1 : 0;
    debug_state.store(on ? 1 : 0, std::memory_order_relaxed);
    return prev;
}

const char* fqm_status_str(int32_t status) {
    switch (status) {
        case FQM_OK: return "ok";
        case FQM_E_NULL: return "a required pointer is NULL";
        case FQM_E_ALIGN: return "a base pointer or row stride is not 16-byte aligned";
        case FQM_E_SHAPE: return "sizes negative, out of range or inconsistent";
        case FQM_E_FORMAT: return "unknown format or format parameter out of range";
        case FQM_E_WORKSPACE: return "workspace missing or too small";
        case FQM_E_UNSUPPORTED: return "combination not supported";
        case FQM_E_HIP: return "HIP launch failed";
        case FQM_E_SCRATCH: return "needs more scratch than fqm_gemv_static's static maximum";
        case FQM_E_BOUNDS: return "debug checks: a buffer is not inside one device allocation of its size";
        default: return "unknown status";
    }
}

fqm_status fqm_pack_bits(const uint8_t* vals, uint8_t* out, int64_t rows, int64_t cols,
                         int32_t bits, int64_t ld, int32_t* d_err, void* stream) {
    if (bits != 1 && bits != 4 && bits != 6 && bits != 8) return FQM_E_FORMAT;
    if (rows < 0 || cols < 0) return FQM_E_SHAPE;
    if (rows == 0) return FQM_OK;
    if (!out || (cols > 0 && !vals)) return FQM_E_NULL;
    if (!aligned16(out)) return FQM_E_ALIGN;
    if (ld < (cols * bits + 7) / 8) return FQM_E_SHAPE;
    if (ld & 15) return FQM_E_ALIGN;
    if (debug_on() && !(in_allocation(vals, rows * cols) && in_allocation(out, span(rows, ld, (cols * bits + 7) / 8)) &&
                        (!d_err || in_allocation(d_err, 4))))
        return FQM_E_BOUNDS;
    return debug_finish(hip_status(launch_pack_bits(vals, out, rows, cols, bits, ld, d_err, as_stream(stream))),
                        as_stream(stream));
}

fqm_status fqm_pack(const uint8_t* codes, uint8_t* packed, int64_t rows, int64_t cols, int64_t ld,
                    int32_t* d_err, void* stream) {
    return fqm_pack_bits(codes, packed, rows, cols, 6, ld, d_err, stream);
}

fqm_status fqm_unpack(const uint8_t* packed, uint8_t* codes, int64_t rows, int64_t cols, int64_t ld,
                      void* stream) {
    if (rows < 0 || cols < 0 || (cols & 3)) return FQM_E_SHAPE;
    if (rows == 0 || cols == 0) return FQM_OK;
    if (!packed || !codes) return FQM_E_NULL;
    if (!aligned16(packed)) return FQM_E_ALIGN;
    if (ld < cols * 3 / 4) return FQM_E_SHAPE;
    if (ld & 15) return FQM_E_ALIGN;
    if (debug_on() && !(in_allocation(packed, span(rows, ld, cols * 3 / 4)) && in_allocation(codes, rows * cols)))
        return FQM_E_BOUNDS;
    return debug_finish(hip_status(launch_unpack6(packed, codes, rows, cols, ld, as_stream(stream))), as_stream(stream));
}

fqm_status fqm_dequant(const fqm_weights* w, uint16_t* W, void* stream) {
    const fqm_status st = check_weights(w);
    if (st != FQM_OK) return st;
    if (w->format == FQM_MDBF) return FQM_E_UNSUPPORTED;
    if (w->rows == 0 || w->cols == 0) return FQM_OK;
    if (!W) return FQM_E_NULL;
    if (!aligned16(W)) return FQM_E_ALIGN;
    if (debug_on() && (check_weight_buffers(*w) != FQM_OK || !in_allocation(W, w->rows * w->cols * 2)))
        return FQM_E_BOUNDS;
    hipStream_t s = as_stream(stream);
    if (w->format == FQM_LUT6) return debug_finish(hip_status(launch_dequant_lut6(*w, W, s)), s);
    if (w->format == FQM_LUT4) return debug_finish(hip_status(launch_dequant_lut4(*w, W, s)), s);
    return debug_finish(hip_status(launch_dequant_fabq(*w, W, s)), s);
}

size_t fqm_workspace_size(const fqm_weights* w, int32_t batch) {
    if (check_weights(w) != FQM_OK || batch < 1 || batch > 16) return 0;
    if (w->format == FQM_LUT6 || w->format == FQM_LUT4) return fqm::lut_gemv_mfma_workspace(*w, batch);
    if (w->format == FQM_FABQ) return fqm::fabq_workspace_bytes(*w, batch);
    if (w->format != FQM_MDBF) return 0;
    return fqm::mdbf_workspace_bytes(*w, batch);
}

}  // extern "C"

namespace {

// The launches of fqm_gemv once its arguments have passed the checks.
fqm_status gemv_launch(const fqm_weights* w, const uint16_t* x, void* y, int y_f32, int32_t batch,
                       void* workspace, size_t ws_bytes, hipStream_t s) {
    if (w->cols == 0)  // an empty sum: y = 0 whatever the format (x is not read)
        return hip_status(launch_zero_fill(y, (int64_t)batch * w->rows, y_f32 ? 4 : 2, s));
    switch (w->format) {
        case FQM_LUT6: {
            const size_t need = fqm_workspace_size(w, batch);
            if (need && (!workspace || ws_bytes < need)) return FQM_E_WORKSPACE;
            if (need && !aligned16(workspace)) return FQM_E_ALIGN;
            return hip_status(
                launch_lut6_gemv(*w, x, y, y_f32, batch, static_cast<float*>(workspace), s));
        }
        case FQM_LUT4: {
            const size_t need = fqm_workspace_size(w, batch);
            if (need && (!workspace || ws_bytes < need)) return FQM_E_WORKSPACE;
            if (need && !aligned16(workspace)) return FQM_E_ALIGN;
            return hip_status(
                launch_lut4_gemv(*w, x, y, y_f32, batch, static_cast<float*>(workspace), s));
        }
        case FQM_FABQ: {
            const size_t need = fqm_workspace_size(w, batch);
            if (need && (!workspace || ws_bytes < need)) return FQM_E_WORKSPACE;
            if (need && !aligned16(workspace)) return FQM_E_ALIGN;
            return hip_status(launch_fabq_gemv(*w, x, y, y_f32, batch, static_cast<float*>(workspace), s));
        }
        case FQM_MDBF: {
            const size_t need = fqm_workspace_size(w, batch);
            if (!workspace || ws_bytes < need) return FQM_E_WORKSPACE;
            if (!aligned16(workspace)) return FQM_E_ALIGN;
            return hip_status(
                launch_mdbf_gemv(*w, x, y, y_f32, batch, workspace, s));
        }
    }
    return FQM_E_FORMAT;
}

// fqm_gemv; static_ws: the workspace is fqm_gemv_static's scratch array (a
// device symbol, not an allocation the debug checks can look up).
fqm_status gemv_impl(const fqm_weights* w, const uint16_t* x, void* y, int32_t y_dtype, int32_t batch,
                     void* workspace, size_t ws_bytes, void* stream, bool static_ws) {
    const fqm_status st = check_weights(w);
    if (st != FQM_OK) return st;
    if (batch < 1 || batch > 16) return FQM_E_SHAPE;
    if (y_dtype != FQM_BF16 && y_dtype != FQM_F32) return FQM_E_FORMAT;
    if (w->rows == 0) return FQM_OK;
    if (!y || (w->cols > 0 && !x)) return FQM_E_NULL;
    if (!aligned16(y) || (x && !aligned16(x))) return FQM_E_ALIGN;
    const int y_f32 = y_dtype == FQM_F32;
    hipStream_t s = as_stream(stream);
    if (!debug_on()) return gemv_launch(w, x, y, y_f32, batch, workspace, ws_bytes, s);
    const size_t need = w->cols > 0 ? fqm_workspace_size(w, batch) : 0;
    if (check_weight_buffers(*w) != FQM_OK || !in_allocation(x, (int64_t)batch * w->cols * 2) ||
        !in_allocation(y, (int64_t)batch * w->rows * (y_f32 ? 4 : 2)) ||
        (!static_ws && workspace && !in_allocation(workspace, (int64_t)need)))
        return FQM_E_BOUNDS;
    return debug_finish(gemv_launch(w, x, y, y_f32, batch, workspace, ws_bytes, s), s);
}

}  // namespace

extern "C" {

fqm_status fqm_gemv(const fqm_weights* w, const uint16_t* x, void* y, int32_t y_dtype,
                    int32_t batch, void* workspace, size_t ws_bytes, void* stream) {
    return gemv_impl(w, x, y, y_dtype, batch, workspace, ws_bytes, stream, false);
}

fqm_status fqm_gemv_static(const fqm_weights* w, const uint16_t* x, void* y, int32_t y_dtype,
                           int32_t batch, void* stream) {
    const fqm_status st = check_weights(w);
    if (st != FQM_OK) return st;
    if (batch < 1 || batch > 16) return FQM_E_SHAPE;
    const size_t need = fqm_workspace_size(w, batch);
    if (need > FQM_STATIC_SCRATCH_BYTES) return FQM_E_SCRATCH;
    void* ws = nullptr;
    if (need && scratch_for_current_device(&ws) != hipSuccess) return FQM_E_HIP;
    return gemv_impl(w, x, y, y_dtype, batch, ws, need, stream, true);
}

// Up to 16 rows of X go to the GEMV kernels when they have a tuned kernel
// for the shape: the prefill tiles are 256 rows tall, so below that the
// matrix cores would mostly multiply padding (measured on the 17408 x 5120
// layer: 14-31 us through the GEMV path against 68-71 us as a GEMM).
static bool gemm_as_gemv(const fqm_weights& w, int64_t M) {
    if (M < 1 || M > 16) return false;
    return w.format == FQM_LUT4 ? fqm::lut4_gemv_fast_path(w, (int)M) : fqm::lut6_gemv_fast_path(w, (int)M);
}

static bool lut_format(const fqm_weights& w) { return w.format == FQM_LUT6 || w.format == FQM_LUT4; }

size_t fqm_gemm_workspace_size(const fqm_weights* w, int64_t M) {
    if (check_weights(w) != FQM_OK || !lut_format(*w) || M <= 0 || w->rows == 0) return 0;
    if (w->cols % 64 || M * w->cols * 2 > INT32_MAX) return 0;
    if (w->cols == 0) return 0;  // Y is zero-filled, no K parts
    if (gemm_as_gemv(*w, M)) return fqm::lut_gemv_mfma_workspace(*w, (int)M);
    return fqm::lut_gemm_workspace(*w, M);
}

fqm_status fqm_gemm(const fqm_weights* w, const uint16_t* X, uint16_t* Y, int64_t M, void* workspace,
                    size_t ws_bytes, void* stream) {
    const fqm_status st = check_weights(w);
    if (st != FQM_OK) return st;
    if (!lut_format(*w)) return FQM_E_UNSUPPORTED;
    if (M < 0) return FQM_E_SHAPE;
    if (M > (int64_t)65535 * 128) return FQM_E_SHAPE;
    if (M == 0 || w->rows == 0) return FQM_OK;
    if (w->cols % 64 || M * w->cols * 2 > INT32_MAX) return FQM_E_SHAPE;
    if (!Y || (w->cols > 0 && !X)) return FQM_E_NULL;
    if (!aligned16(Y) || (X && !aligned16(X))) return FQM_E_ALIGN;
    const size_t need = fqm_gemm_workspace_size(w, M);
    if (need && (!workspace || ws_bytes < need)) return FQM_E_WORKSPACE;
    if (need && !aligned16(workspace)) return FQM_E_ALIGN;
    hipStream_t s = as_stream(stream);
    if (debug_on() && (check_weight_buffers(*w) != FQM_OK || !in_allocation(X, M * w->cols * 2) ||
                       !in_allocation(Y, M * w->rows * 2) || (need && !in_allocation(workspace, (int64_t)need))))
        return FQM_E_BOUNDS;
    fqm_status r;
    if (w->cols == 0)  // an empty sum: Y = 0 (the tile kernels assume at least one K step)
        r = hip_status(launch_zero_fill(Y, M * w->rows, 2, s));
    else if (gemm_as_gemv(*w, M))  // Y[M][rows] bf16 is the GEMV's y[batch][rows]
        r = hip_status(w->format == FQM_LUT4
                           ? launch_lut4_gemv(*w, X, Y, 0, (int)M, static_cast<float*>(workspace), s)
                           : launch_lut6_gemv(*w, X, Y, 0, (int)M, static_cast<float*>(workspace), s));
    else
        r = hip_status(launch_lut_gemm(*w, X, Y, M, workspace, ws_bytes, s));
    return debug_finish(r, s);
}

}  // extern "C"

// ---- the operators around the products ---------------------------------------

namespace {

inline bool value_dtype(int32_t t) { return t == FQM_BF16 || t == FQM_F32; }
inline int64_t dtype_bytes(int32_t t) { return t == FQM_F32 ? 4 : t == FQM_BF16 ? 2 : 1; }
inline bool aligned_to(const void* p, int64_t bytes) {
    return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) == 0;
}
// `rows` rows of `need` elements `ld` apart: the stride holds a row and the
// extent in bytes stays far inside int64.
inline bool rows_ok(int64_t rows, int64_t ld, int64_t need) {
    return ld >= need && ld <= ((int64_t)1 << 40) && rows <= ((int64_t)1 << 58) / std::max<int64_t>(ld, 1);
}

fqm_status check_norm(const fqm_norm* a) {
    if (!a) return FQM_E_NULL;
    if (a->rows < 0 || a->rows > 0x7fffffff || a->cols < 0 || a->cols > 32768 || a->terms < 1 || a->terms > 64)
        return FQM_E_SHAPE;
    if (!value_dtype(a->x_dtype) || (a->residual && !value_dtype(a->res_dtype)) ||
        (a->weight && !value_dtype(a->weight_dtype)) || !(value_dtype(a->y_dtype) || a->y_dtype == FQM_I8) ||
        !(a->eps >= 0.f && a->eps <= 3.4e38f))
        return FQM_E_FORMAT;
    if (a->rows == 0) return FQM_OK;
    if (a->y_dtype == FQM_I8 && !a->y_scale) return FQM_E_NULL;
    if (a->y_dtype == FQM_I8 && !aligned_to(a->y_scale, 4)) return FQM_E_ALIGN;
    if (a->cols == 0) return FQM_OK;
    if (!a->x || !a->y) return FQM_E_NULL;
    if (!rows_ok(a->rows, a->ld_x, a->cols) || (a->terms > 1 && !rows_ok(a->terms, a->ld_term, a->cols)) ||
        (a->residual && !rows_ok(a->rows, a->ld_res, a->cols)) ||
        (a->total && !rows_ok(a->rows, a->ld_total, a->cols)) || !rows_ok(a->rows, a->ld_y, a->cols))
        return FQM_E_SHAPE;
    const int32_t total_dtype = a->residual ? a->res_dtype : a->x_dtype;
    if (!aligned_to(a->x, dtype_bytes(a->x_dtype)) || !aligned_to(a->y, dtype_bytes(a->y_dtype)) ||
        (a->residual && !aligned_to(a->residual, dtype_bytes(a->res_dtype))) ||
        (a->weight && !aligned_to(a->weight, dtype_bytes(a->weight_dtype))) ||
        (a->total && !aligned_to(a->total, dtype_bytes(total_dtype))))
        return FQM_E_ALIGN;
    return FQM_OK;
}

bool norm_buffers_ok(const fqm_norm& a) {
    const int64_t xb = dtype_bytes(a.x_dtype), rb = dtype_bytes(a.res_dtype), yb = dtype_bytes(a.y_dtype);
    const int64_t tb = a.residual ? rb : xb;
    const int64_t term = a.terms > 1 ? (a.terms - 1) * a.ld_term : 0;
    return in_allocation(a.x, (span(a.rows, a.ld_x, a.cols) + term) * xb) &&
           (!a.residual || in_allocation(a.residual, span(a.rows, a.ld_res, a.cols) * rb)) &&
           (!a.weight || in_allocation(a.weight, a.cols * dtype_bytes(a.weight_dtype))) &&
           (!a.total || in_allocation(a.total, span(a.rows, a.ld_total, a.cols) * tb)) &&
           in_allocation(a.y, span(a.rows, a.ld_y, a.cols) * yb) &&
           (a.y_dtype != FQM_I8 || in_allocation(a.y_scale, a.rows * 4));
}

constexpr int64_t kMaxRows = (int64_t)1 << 24;  // rows of one lora or grouped call

fqm_status check_adapters(const fqm_adapters* a) {
    if (!a) return FQM_E_NULL;
    if (a->count < 1 || a->count > 65536 || a->rank < 1 || a->rank > 256) return FQM_E_FORMAT;
    if (a->rows < 0 || a->rows > (1 << 22) || a->cols < 0 || a->cols > (1 << 21) || a->cols % 8) return FQM_E_SHAPE;
    if (a->rows == 0) return FQM_OK;
    if ((a->cols > 0 && !a->A) || !a->B) return FQM_E_NULL;
    if (!rows_ok((int64_t)a->count * a->rank, a->ld_A, a->cols) || a->ld_A > (1 << 22) ||
        !rows_ok((int64_t)a->count * a->rows, a->ld_B, a->rank))
        return FQM_E_SHAPE;
    if (!aligned16(a->A) || !aligned16(a->B) || (a->ld_A & 7) || (a->ld_B & 7) || !aligned_to(a->scale, 4) ||
        !aligned_to(a->ranks, 4))
        return FQM_E_ALIGN;
    return FQM_OK;
}

// What the workspace depends on: sizes and types, no pointer of g.
fqm_status check_group_sizes(const fqm_weights* w, const fqm_groups* g) {
    const fqm_status st = check_weights(w);
    if (st != FQM_OK) return st;
    if (!lut_format(*w)) return FQM_E_UNSUPPORTED;
    if (!g) return FQM_E_NULL;
    if (g->count < 1 || g->count > 4096) return FQM_E_FORMAT;
    if (!(g->x_dtype == FQM_BF16 || g->x_dtype == FQM_I8) || !value_dtype(g->y_dtype)) return FQM_E_FORMAT;
    if (g->M < 0 || g->M > kMaxRows || g->x_rows < 0 || g->x_rows > 0x7fffffff || g->y_rows < 0 ||
        g->y_rows > 0x7fffffff || w->rows % g->count || w->rows / g->count > kMaxRows || w->cols > (1 << 21))
        return FQM_E_SHAPE;
    if (g->M == 0 || w->rows == 0) return FQM_OK;
    if ((!g->src && g->x_rows < g->M) || (!g->dst && g->y_rows < g->M)) return FQM_E_SHAPE;
    if (g->src && g->x_rows * w->cols * 2 > INT32_MAX) return FQM_E_SHAPE;
    return FQM_OK;
}

fqm_status check_groups(const fqm_weights* w, const fqm_groups* g) {
    const fqm_status st = check_group_sizes(w, g);
    if (st != FQM_OK || g->M == 0 || w->rows == 0) return st;
    const bool has_x = g->x_rows > 0 && w->cols > 0;
    if (!g->offsets || (g->y_rows > 0 && !g->Y) || (has_x && !g->X) ||
        (g->x_dtype == FQM_I8 && has_x && !g->x_scale))
        return FQM_E_NULL;
    if (!aligned16(g->X) || !aligned16(g->Y) || !aligned_to(g->offsets, 4) || !aligned_to(g->src, 4) ||
        !aligned_to(g->dst, 4) || !aligned_to(g->x_scale, 4) || !aligned_to(g->row_scale, 4))
        return FQM_E_ALIGN;
    return FQM_OK;
}

bool groups_buffers_ok(const fqm_weights& w, const fqm_groups& g) {
    return check_weight_buffers(w) == FQM_OK && in_allocation(g.offsets, ((int64_t)g.count + 1) * 4) &&
           in_allocation(g.X, g.x_rows * w.cols * dtype_bytes(g.x_dtype)) &&
           (g.x_dtype != FQM_I8 || in_allocation(g.x_scale, g.x_rows * 4)) && (!g.src || in_allocation(g.src, g.M * 4)) &&
           in_allocation(g.Y, g.y_rows * (w.rows / g.count) * dtype_bytes(g.y_dtype)) &&
           (!g.dst || in_allocation(g.dst, g.M * 4)) && (!g.row_scale || in_allocation(g.row_scale, g.M * 4));
}

}  // namespace

extern "C" {

fqm_status fqm_add_rms_norm(const fqm_norm* a, void* stream) {
    const fqm_status st = check_norm(a);
    if (st != FQM_OK || a->rows == 0) return st;
    hipStream_t s = as_stream(stream);
    if (a->cols == 0) {
        if (a->y_dtype != FQM_I8) return FQM_OK;
        if (debug_on() && !in_allocation(a->y_scale, a->rows * 4)) return FQM_E_BOUNDS;
        return debug_finish(hip_status(launch_zero_fill(a->y_scale, a->rows, 4, s)), s);
    }
    if (debug_on() && !norm_buffers_ok(*a)) return FQM_E_BOUNDS;
    return debug_finish(hip_status(launch_add_rms_norm(*a, s)), s);
}

size_t fqm_lora_workspace_size(const fqm_adapters* a, int64_t M) {
    if (check_adapters(a) != FQM_OK || M <= 0 || M > kMaxRows || a->rows == 0) return 0;
    return fqm::lora_workspace(*a, M);
}

fqm_status fqm_lora(const fqm_adapters* a, const uint16_t* x, const int32_t* index, const void* base,
                    int32_t base_dtype, void* y, int32_t y_dtype, int64_t M, void* workspace, size_t ws_bytes,
                    void* stream) {
    const fqm_status st = check_adapters(a);
    if (st != FQM_OK) return st;
    if (M < 0 || M > kMaxRows) return FQM_E_SHAPE;
    if (!value_dtype(y_dtype) || (base && !value_dtype(base_dtype))) return FQM_E_FORMAT;
    if (M == 0 || a->rows == 0) return FQM_OK;
    if ((a->cols > 0 && !x) || !index || !y) return FQM_E_NULL;
    if (base == y && base_dtype != y_dtype) return FQM_E_FORMAT;
    if (!aligned16(x) || !aligned_to(index, 4) || !aligned_to(y, dtype_bytes(y_dtype)) ||
        (base && !aligned_to(base, dtype_bytes(base_dtype))))
        return FQM_E_ALIGN;
    const size_t need = fqm_lora_workspace_size(a, M);
    if (need && (!workspace || ws_bytes < need)) return FQM_E_WORKSPACE;
    if (need && !aligned16(workspace)) return FQM_E_ALIGN;
    hipStream_t s = as_stream(stream);
    if (debug_on() &&
        !(in_allocation(a->A, span((int64_t)a->count * a->rank, a->ld_A, a->cols) * 2) &&
          in_allocation(a->B, span((int64_t)a->count * a->rows, a->ld_B, a->rank) * 2) &&
          (!a->scale || in_allocation(a->scale, a->count * 4ll)) &&
          (!a->ranks || in_allocation(a->ranks, a->count * 4ll)) && in_allocation(x, M * a->cols * 2) &&
          in_allocation(index, M * 4) && (!base || in_allocation(base, M * a->rows * dtype_bytes(base_dtype))) &&
          in_allocation(y, M * a->rows * dtype_bytes(y_dtype)) && in_allocation(workspace, (int64_t)need)))
        return FQM_E_BOUNDS;
    return debug_finish(hip_status(launch_lora(*a, x, index, base, base_dtype == FQM_F32, y, y_dtype == FQM_F32, M,
                                               static_cast<float*>(workspace), s)),
                        s);
}

size_t fqm_gemm_grouped_workspace_size(const fqm_weights* w, const fqm_groups* g) {
    if (check_group_sizes(w, g) != FQM_OK || g->M == 0 || w->rows == 0) return 0;
    return fqm::grouped_workspace(*w, *g);
}

fqm_status fqm_gemm_grouped(const fqm_weights* w, const fqm_groups* g, void* workspace, size_t ws_bytes,
                            void* stream) {
    const fqm_status st = check_groups(w, g);
    if (st != FQM_OK || g->M == 0 || w->rows == 0) return st;
    const size_t need = fqm::grouped_workspace(*w, *g);
    if (need && (!workspace || ws_bytes < need)) return FQM_E_WORKSPACE;
    if (need && !aligned16(workspace)) return FQM_E_ALIGN;
    hipStream_t s = as_stream(stream);
    if (debug_on() && (!groups_buffers_ok(*w, *g) || (need && !in_allocation(workspace, (int64_t)need))))
        return FQM_E_BOUNDS;
    return debug_finish(hip_status(launch_grouped(*w, *g, workspace, s)), s);
}

}  // extern "C"
