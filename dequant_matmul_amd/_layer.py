"""The operators around the quantized products: the residual norm, the
low-rank adapters and the products grouped by expert.

Argument marshalling only, as in the package's other calls: shapes, types,
layouts and devices are checked here (the C ABI sees only pointers), the
computation runs in the HIP kernels behind ``fqm_add_rms_norm``, ``fqm_lora``
and ``fqm_gemm_grouped`` (include/fqm.h has their definitions).  With ``stream``
given, what a call allocates belongs to that stream.  There are no gradients, as
in the package's other calls: outputs are detached from the inputs.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import (FQM_BF16, FQM_F32, FQM_I8, FQM_LUT4, FQM_LUT6, _Adapters, _check, _check_workspace, _Groups, _Norm,
               _stream, _WeightsBase, load)

# The current stream's handle without a Stream object around it (2.9 us a call on the host, as much as a launch).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)

_CODE = {torch.bfloat16: FQM_BF16, torch.float32: FQM_F32, torch.int8: FQM_I8}
_VALUE = (torch.bfloat16, torch.float32)


def _need(t, name: str, dtypes, device=None, dim: int | None = None):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}; expected one of {dtypes}")
    if not t.is_cuda:
        raise ValueError(f"{name} is on {t.device}; the library takes GPU tensors")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if dim is not None and t.dim() != dim:
        raise ValueError(f"{name} has shape {tuple(t.shape)}; expected {dim} dimensions")


def _elsewhere(stream, device):
    """Whether the call is for another stream or device than the current ones.  It is then
    made again inside them: what it allocates (outputs, workspace) belongs to that stream,
    so that its memory is not handed out again under the running kernels."""
    if stream is not None and stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the operands on {device}")
    return stream is not None or device.index != torch.cuda.current_device()


class _inside:
    """The device and stream of a call as the current ones."""

    def __init__(self, stream, device):
        self.device = torch.cuda.device(device)
        self.stream = torch.cuda.stream(stream)

    def __enter__(self):
        self.device.__enter__()
        self.stream.__enter__()

    def __exit__(self, *exc):
        self.stream.__exit__(*exc)
        self.device.__exit__(*exc)


def _handle(device):
    return _raw_stream(device.index) if _raw_stream is not None else _stream()


def _vector(t, name: str, n: int, dtypes, device):
    """An optional contiguous vector of n values."""
    if t is None:
        return None
    _need(t, name, dtypes, device)
    if tuple(t.shape) != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of {n} values; got shape {tuple(t.shape)}")
    return t.data_ptr()


def _row_stride(t, name: str, shape) -> int:
    """The row stride of a [rows][cols] tensor whose rows are dense and do not overlap."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}; expected {tuple(shape)}")
    rows, cols = shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have dense rows (stride 1 in the last dimension)")
    if rows <= 1:
        return cols
    if t.stride(0) < cols:
        raise ValueError(f"{name} has overlapping rows (row stride {t.stride(0)}, width {cols})")
    return t.stride(0)


# ---------------------------------------------------------------------------
# residual norm
# ---------------------------------------------------------------------------
class NormOut(NamedTuple):
    """y [rows][cols]; scale [rows] of an int8 y, else None; total, the sum
    that was normed, where it was asked for."""
    y: torch.Tensor
    scale: Optional[torch.Tensor]
    total: Optional[torch.Tensor]


def add_rms_norm(x: torch.Tensor, weight: torch.Tensor | None = None, eps: float = 1e-6,
                 residual: torch.Tensor | None = None, out_dtype: torch.dtype = torch.bfloat16,
                 y: torch.Tensor | None = None, scale: torch.Tensor | None = None,
                 total: torch.Tensor | None = None, keep_total: bool | None = None, stream=None) -> NormOut:
    """The residual's addition and the root-mean-square norm in one pass:
    ``h = x + residual`` (fp32), ``y = h * weight / sqrt(mean(h^2) + eps)``.

    x: [rows][cols], or [rows][terms][cols] whose terms are added up (the rows
    that a token's experts return); bf16 or fp32, rows of any stride.
    residual: [rows][cols] or None.  ``total`` gets h in the residual's dtype
    (x's without one); it is returned where there is something to add up,
    unless ``keep_total`` says otherwise, and may be ``residual`` itself.
    out_dtype: bfloat16, float32, or int8 with one scale a row:
    ``scale = max|y| / 127``, ``y`` the nearest codes."""
    _need(x, "x", _VALUE)
    if _elsewhere(stream, x.device):
        with _inside(stream, x.device):
            return add_rms_norm(x, weight, eps, residual, out_dtype, y, scale, total, keep_total)
    if x.dim() not in (2, 3):
        raise ValueError(f"x must be [rows][cols] or [rows][terms][cols]; got shape {tuple(x.shape)}")
    dev, rows, cols = x.device, x.shape[0], x.shape[-1]
    terms = x.shape[1] if x.dim() == 3 else 1
    if not 1 <= terms <= 64:
        raise ValueError(f"x has {terms} terms; 1 to 64 can be added up")
    if cols > 1 and x.stride(-1) != 1:
        raise ValueError("x must have dense rows (stride 1 in the last dimension)")
    ld_x = x.stride(0) if rows > 1 else cols
    ld_term = x.stride(1) if terms > 1 else cols
    if ld_x < cols or ld_term < cols:
        raise ValueError("x has overlapping rows")
    total_dtype = x.dtype
    a = _Norm(rows, cols, terms, _CODE[x.dtype], 0, 0, 0, eps, x.data_ptr(), ld_x, ld_term)
    if residual is not None:
        _need(residual, "residual", _VALUE, dev)
        a.ld_res = _row_stride(residual, "residual", (rows, cols))
        total_dtype = residual.dtype
        a.residual, a.res_dtype = residual.data_ptr(), _CODE[total_dtype]
    if weight is not None:
        a.weight = _vector(weight, "weight", cols, _VALUE, dev)
        a.weight_dtype = _CODE[weight.dtype]
    if keep_total is None:
        keep_total = residual is not None or terms > 1
    if total is not None:
        _need(total, "total", (total_dtype,), dev)
        a.ld_total, a.total = _row_stride(total, "total", (rows, cols)), total.data_ptr()
    elif keep_total:
        total = torch.empty((rows, cols), dtype=total_dtype, device=dev)
        a.ld_total, a.total = cols, total.data_ptr()
    if y is None:
        if out_dtype not in _CODE:
            raise ValueError(f"out_dtype must be bfloat16, float32 or int8, not {out_dtype}")
        y = torch.empty((rows, cols), dtype=out_dtype, device=dev)
        a.ld_y = cols
    else:
        _need(y, "y", tuple(_CODE), dev)
        a.ld_y, out_dtype = _row_stride(y, "y", (rows, cols)), y.dtype
    a.y, a.y_dtype = y.data_ptr(), _CODE[out_dtype]
    if out_dtype == torch.int8:
        if scale is None:
            scale = torch.empty(rows, dtype=torch.float32, device=dev)
        a.y_scale = _vector(scale, "scale", rows, (torch.float32,), dev)
    else:
        scale = None
    _check(load().fqm_add_rms_norm(ctypes.byref(a), _handle(dev)), "fqm_add_rms_norm")
    return NormOut(y, scale, total)


# ---------------------------------------------------------------------------
# low-rank adapters
# ---------------------------------------------------------------------------
class Adapters:
    """The low-rank adapters of one projection: A [count][rank][cols] and
    B [count][rows][rank] in bf16, adapter a adding ``scale[a] * B_a (A_a x)``.

    scale: [count] fp32 (ones if None).  ranks: [count] int32 where adapters
    have ranks below the layout's; what A and B hold past them is not used.
    A and B are read in place where their last dimension is dense with row
    strides that are multiples of 8 values, their matrices lie back to back and
    they start at a multiple of 16 bytes; others (a rank that is no multiple of
    8, for one) are copied into padded rows, and what is written to them later
    does not reach the copy."""

    def __init__(self, A: torch.Tensor, B: torch.Tensor, scale: torch.Tensor | None = None,
                 ranks: torch.Tensor | None = None):
        _need(A, "A", (torch.bfloat16,), dim=3)
        _need(B, "B", (torch.bfloat16,), A.device, dim=3)
        self.device = A.device
        self.count, self.rank, self.cols = A.shape
        self.rows = B.shape[1]
        if B.shape[0] != self.count or B.shape[2] != self.rank:
            raise ValueError(f"B has shape {tuple(B.shape)}; expected ({self.count}, rows, {self.rank})")
        if not (1 <= self.count <= 65536 and 1 <= self.rank <= 256):
            raise ValueError(f"{self.count} adapters of rank {self.rank}: 1 to 65536, ranks 1 to 256")
        if self.cols % 8:
            raise ValueError(f"{self.cols} inputs: a multiple of 8 is needed")
        self.A, self.B = (t if self._rows_fit(t) else self._padded(t) for t in (A, B))
        self.scale, self.ranks = scale, ranks
        self.desc = _Adapters(self.count, self.rank, self.rows, self.cols, self.A.data_ptr(), self._ld(self.A),
                              self.B.data_ptr(), self._ld(self.B),
                              _vector(scale, "scale", self.count, (torch.float32,), self.device),
                              _vector(ranks, "ranks", self.count, (torch.int32,), self.device))

    @staticmethod
    def _ld(t):
        if t.shape[2] == 0:  # no values: any stride, and torch's own is 1
            return 0
        return t.stride(1) if t.shape[1] > 1 else t.stride(0) if t.shape[0] > 1 else (t.shape[2] + 7) // 8 * 8

    @classmethod
    def _rows_fit(cls, t):
        n, rows, cols = t.shape
        ld = cls._ld(t)
        return ((cols == 1 or t.stride(2) == 1) and ld >= cols and ld % 8 == 0 and t.data_ptr() % 16 == 0
                and (n == 1 or t.stride(0) == rows * ld))

    @staticmethod
    def _padded(t):
        n, rows, cols = t.shape
        out = torch.zeros((n, rows, (cols + 7) // 8 * 8), dtype=t.dtype, device=t.device)
        out[:, :, :cols] = t
        return out[:, :, :cols]

    @property
    def ref(self):
        return ctypes.byref(self.desc)

    def nbytes(self) -> int:
        """Bytes of all adapters at their layout's rank (unpadded)."""
        return self.count * self.rank * (self.cols + self.rows) * 2


def lora_workspace_size(adapters: Adapters, M: int) -> int:
    return int(load().fqm_lora_workspace_size(adapters.ref, M))


def lora(adapters: Adapters, x: torch.Tensor, index: torch.Tensor, base: torch.Tensor | None = None,
         y: torch.Tensor | None = None, out_dtype: torch.dtype = torch.bfloat16,
         workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[m] = base[m] + scale[i] * B_i (A_i x[m]), i = index[m]: the adapters of
    many requests on the rows of one batch, beside the shared projection whose
    output is ``base`` (None: zeros).

    x [M][cols] bf16; index [M] int32, rows in any order, a value outside
    0..count-1 for a row without an adapter; base [M][rows] bf16 or fp32.
    ``y`` may be ``base`` (the addition in place).  Any M: single tokens and
    prompts, mixed; above 256 rows the call is 2 to 4 times as fast where each
    adapter's rows lie together."""
    _need(x, "x", (torch.bfloat16,), adapters.device, dim=2)
    if _elsewhere(stream, x.device):
        with _inside(stream, x.device):
            return lora(adapters, x, index, base, y, out_dtype, workspace)
    M = x.shape[0]
    dev = x.device
    if x.shape[1] != adapters.cols or not x.is_contiguous():
        raise ValueError(f"x has shape {tuple(x.shape)}; expected contiguous (M, {adapters.cols})")
    ip = _vector(index, "index", M, (torch.int32,), dev)
    if ip is None:
        raise ValueError("index must be a torch.Tensor")
    shape = (M, adapters.rows)
    bp, bdt = None, FQM_BF16
    if base is not None:
        _need(base, "base", _VALUE, dev)
        if tuple(base.shape) != shape or not base.is_contiguous():
            raise ValueError(f"base has shape {tuple(base.shape)}; expected contiguous {shape}")
        bp, bdt = base.data_ptr(), _CODE[base.dtype]
    if y is None:
        if out_dtype not in _VALUE:
            raise ValueError(f"out_dtype must be bfloat16 or float32, not {out_dtype}")
        y = torch.empty(shape, dtype=out_dtype, device=dev)
    else:
        _need(y, "y", _VALUE, dev)
        if tuple(y.shape) != shape or not y.is_contiguous():
            raise ValueError(f"y has shape {tuple(y.shape)}; expected contiguous {shape}")
    _check_workspace(workspace, dev)
    lib = load()
    if workspace is None:
        need = lib.fqm_lora_workspace_size(adapters.ref, M)
        workspace = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib.fqm_lora(adapters.ref, x.data_ptr(), ip, bp, bdt, y.data_ptr(), _CODE[y.dtype], M,
                        workspace.data_ptr() if workspace is not None else None, ws_bytes, _handle(dev)),
           "fqm_lora")
    return y


# ---------------------------------------------------------------------------
# products grouped by expert
# ---------------------------------------------------------------------------
def _groups(w: _WeightsBase, X, offsets, src, x_scale, dst, row_scale, Y, out_dtype, y_rows, sizes_only=False):
    """Checks the operands; returns the descriptor and Y (sizes_only: a descriptor without Y)."""
    if getattr(w, "fmt", None) not in (FQM_LUT6, FQM_LUT4):
        raise ValueError("grouped products take Lut6Weights or Lut4Weights")
    dev = w.packed.device
    _need(offsets, "offsets", (torch.int32,), dev, dim=1)
    count = offsets.shape[0] - 1
    if count < 1 or not offsets.is_contiguous():
        raise ValueError("offsets must be a contiguous vector of one more value than there are groups")
    if w.rows % count:
        raise ValueError(f"{w.rows} stacked rows are not {count} matrices of equal size")
    rows = w.rows // count
    _need(X, "X", (torch.bfloat16, torch.int8), dev, dim=2)
    if X.shape[1] != w.cols or not X.is_contiguous():
        raise ValueError(f"X has shape {tuple(X.shape)}; expected contiguous (rows, {w.cols})")
    if (X.dtype == torch.int8) != (x_scale is not None):
        raise ValueError("int8 rows need x_scale, one value per row of X, and bf16 rows take none")
    M = X.shape[0]
    if src is not None:
        _need(src, "src", (torch.int32,), dev, dim=1)
        M = src.shape[0]
    if Y is not None:
        _need(Y, "Y", _VALUE, dev, dim=2)
    if y_rows is None:
        y_rows = M if Y is None else Y.shape[0]
    if Y is None:
        if out_dtype not in _VALUE:
            raise ValueError(f"out_dtype must be bfloat16 or float32, not {out_dtype}")
        if not sizes_only:
            Y = torch.empty((y_rows, rows), dtype=out_dtype, device=dev)
    else:
        out_dtype = Y.dtype
        if tuple(Y.shape) != (y_rows, rows) or not Y.is_contiguous():
            raise ValueError(f"Y has shape {tuple(Y.shape)}; expected contiguous ({y_rows}, {rows})")
    if dst is None and y_rows < M:
        raise ValueError(f"Y has {y_rows} rows for {M} grouped rows")
    g = _Groups(count, offsets.data_ptr(), M, X.data_ptr(), _CODE[X.dtype], X.shape[0],
                _vector(x_scale, "x_scale", X.shape[0], (torch.float32,), dev),
                _vector(src, "src", M, (torch.int32,), dev), None if Y is None else Y.data_ptr(), _CODE[out_dtype], y_rows,
                _vector(dst, "dst", M, (torch.int32,), dev),
                _vector(row_scale, "row_scale", M, (torch.float32,), dev))
    return g, Y


def gemm_grouped_workspace_size(w: _WeightsBase, X: torch.Tensor, offsets: torch.Tensor,
                                src: torch.Tensor | None = None, x_scale: torch.Tensor | None = None,
                                out_dtype: torch.dtype = torch.bfloat16) -> int:
    """Bytes of workspace that gemm_grouped needs for such operands on this device."""
    g, _ = _groups(w, X, offsets, src, x_scale, None, None, None, out_dtype, None, sizes_only=True)
    return int(load().fqm_gemm_grouped_workspace_size(w.ref, ctypes.byref(g)))


def gemm_grouped(w: _WeightsBase, X: torch.Tensor, offsets: torch.Tensor, src: torch.Tensor | None = None,
                 x_scale: torch.Tensor | None = None, dst: torch.Tensor | None = None,
                 row_scale: torch.Tensor | None = None, Y: torch.Tensor | None = None,
                 out_dtype: torch.dtype = torch.bfloat16, y_rows: int | None = None,
                 workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Products grouped by expert: grouped rows offsets[e] .. offsets[e+1]-1 meet
    expert e's matrix, ``Y[dst[i]] = row_scale[i] * (W_e X[src[i]])``.

    w: Lut6Weights or Lut4Weights of the experts' matrices stacked row-wise
    (rows = experts * rows of one).  offsets: [experts + 1] int32.  X: [x_rows][cols]
    bf16, or int8 with x_scale (as add_rms_norm gives them).  src: the row of X that
    a grouped row reads (None: its own number; outside X: a row of zeros).  dst: the
    row of Y that it is stored to (None: its own number; outside Y: not stored).
    row_scale: a factor of each grouped row, such as the router's weight.
    Y: [y_rows][rows of one matrix] bf16 or fp32; rows that nothing is stored
    to keep what they hold (a Y made here: undefined).  All index tensors stay on
    the GPU; nothing waits for them."""
    if isinstance(X, torch.Tensor) and X.is_cuda and _elsewhere(stream, X.device):
        with _inside(stream, X.device):
            return gemm_grouped(w, X, offsets, src, x_scale, dst, row_scale, Y, out_dtype, y_rows, workspace)
    g, Y = _groups(w, X, offsets, src, x_scale, dst, row_scale, Y, out_dtype, y_rows)
    _check_workspace(workspace, Y.device)
    lib = load()
    if workspace is None:
        need = lib.fqm_gemm_grouped_workspace_size(w.ref, ctypes.byref(g))
        workspace = torch.empty(need, dtype=torch.uint8, device=Y.device) if need else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib.fqm_gemm_grouped(w.ref, ctypes.byref(g), workspace.data_ptr() if workspace is not None else None,
                                ws_bytes, _handle(Y.device)), "fqm_gemm_grouped")
    return Y
