"""What completes a block around the quantized products: the product with its
epilogue, the routing to experts and the norms on both sides of a block.

Argument marshalling only, as in ``_layer``: shapes, types, layouts and devices
are checked here, the computation runs in the HIP kernels behind
``fqm_linear``, ``fqm_route`` and ``fqm_block_norm`` (include/fqm.h has their
definitions).  With ``stream`` given, what a call allocates belongs to that
stream.  There are no gradients: outputs are detached from the inputs.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import (FQM_ACT, FQM_GROUP_SCORE, FQM_LUT4, FQM_LUT6, FQM_SCORE, _Block, _check, _check_workspace, _Epilogue,
               _Routing, _WeightsBase, load)
from ._layer import _CODE, _VALUE, NormOut, _elsewhere, _handle, _inside, _need, _row_stride, _vector


def _one_of(table, value, name: str) -> int:
    try:
        return table[value]
    except (KeyError, TypeError):
        raise ValueError(f"{name} must be one of {list(table)}, not {value!r}") from None


# ---------------------------------------------------------------------------
# the product with its epilogue
# ---------------------------------------------------------------------------
def _rows_of_x(x, cols: int) -> int:
    """The row stride of x [M][cols] bf16 whose rows start at multiples of 16 bytes."""
    if x.shape[1] != cols:
        raise ValueError(f"x has shape {tuple(x.shape)}; expected (M, {cols})")
    ld = _row_stride(x, "x", x.shape)
    if x.numel() and (x.data_ptr() % 16 or (ld % 8 and x.shape[0] > 1)):
        raise ValueError(f"x must have rows that start at multiples of 16 bytes (row stride {ld} values)")
    return ld


def _epilogue(w, M: int, act, gated: bool, out_dtype) -> _Epilogue:
    if getattr(w, "fmt", None) not in (FQM_LUT6, FQM_LUT4):
        raise ValueError("linear takes Lut6Weights or Lut4Weights")
    if gated and w.rows % 2:
        raise ValueError(f"{w.rows} rows are not two stacked matrices of equal size")
    if out_dtype not in _VALUE:
        raise ValueError(f"out_dtype must be bfloat16 or float32, not {out_dtype}")
    a = _Epilogue()
    a.M, a.act, a.gated, a.y_dtype = M, _one_of(FQM_ACT, act, "act"), 1 if gated else 0, _CODE[out_dtype]
    return a


def linear_workspace_size(w: _WeightsBase, M: int, gated: bool = False,
                          out_dtype: torch.dtype = torch.bfloat16) -> int:
    """Bytes of workspace that linear needs for M rows on the current device."""
    return int(load().fqm_linear_workspace_size(w.ref, ctypes.byref(_epilogue(w, M, None, gated, out_dtype))))


def linear(w: _WeightsBase, x: torch.Tensor, bias: torch.Tensor | None = None, act: str | None = None,
           gated: bool = False, residual: torch.Tensor | None = None, y: torch.Tensor | None = None,
           out_dtype: torch.dtype = torch.bfloat16, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The product with its epilogue: ``v = W x + bias``, ``y = residual + act(v)``,
    or with ``gated``, where W is two stacked matrices of n rows (the gate's
    first), ``y = residual + act(v[:n]) * v[n:]``; fp32 up to one rounding at the end.

    w: Lut6Weights or Lut4Weights.  x: [M][cols] bf16 (or [cols]), rows of any
    stride that is a multiple of 8 values; any M.  bias: [rows] bf16 or fp32.
    act: None, "relu", "silu", "gelu", "gelu_tanh", "sigmoid" or "tanh".
    residual: [M][n] bf16 or fp32, rows of any stride; ``y`` may be ``residual``
    (the addition in place)."""
    _need(x, "x", (torch.bfloat16,))
    if _elsewhere(stream, x.device):
        with _inside(stream, x.device):
            return linear(w, x, bias, act, gated, residual, y, out_dtype, workspace)
    if x.dim() == 1:
        x = x[None]
    dev = x.device
    _need(x, "x", (torch.bfloat16,), dim=2)
    M = x.shape[0]
    a = _epilogue(w, M, act, gated, out_dtype if y is None else getattr(y, "dtype", None))
    if w.packed.device != dev:
        raise ValueError(f"x is on {dev} but the weights are on {w.packed.device}")
    n = w.rows // 2 if gated else w.rows
    a.X, a.ld_x = x.data_ptr(), _rows_of_x(x, w.cols)
    if bias is not None:
        a.bias = _vector(bias, "bias", w.rows, _VALUE, dev)
        a.bias_dtype = _CODE[bias.dtype]
    if residual is not None:
        _need(residual, "residual", _VALUE, dev)
        a.ld_res = _row_stride(residual, "residual", (M, n))
        a.residual, a.res_dtype = residual.data_ptr(), _CODE[residual.dtype]
    if y is None:
        y = torch.empty((M, n), dtype=out_dtype, device=dev)
        a.ld_y = n
    else:
        _need(y, "y", _VALUE, dev)
        a.ld_y = _row_stride(y, "y", (M, n))
    a.Y = y.data_ptr()
    _check_workspace(workspace, dev)
    lib = load()
    if workspace is None:
        need = lib.fqm_linear_workspace_size(w.ref, ctypes.byref(a))
        workspace = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib.fqm_linear(w.ref, ctypes.byref(a), workspace.data_ptr() if workspace is not None else None, ws_bytes,
                          _handle(dev)), "fqm_linear")
    return y


# ---------------------------------------------------------------------------
# routing to experts
# ---------------------------------------------------------------------------
class Routing(NamedTuple):
    """expert, weight [tokens][k]: a token's experts, best first (-1: none), and
    their weights.  offsets [experts + 1], src, dst, row_scale [tokens * k]: the
    operands of that name of gemm_grouped (None without a plan)."""
    expert: torch.Tensor
    weight: torch.Tensor
    offsets: Optional[torch.Tensor]
    src: Optional[torch.Tensor]
    dst: Optional[torch.Tensor]
    row_scale: Optional[torch.Tensor]


def _routing_sizes(T: int, E: int, k: int, groups: int, top_groups: int | None, plan: bool) -> _Routing:
    a = _Routing()
    a.T, a.E, a.k, a.groups, a.top_groups = T, E, k, groups, groups if top_groups is None else top_groups
    if plan:
        a.offsets = 16  # looked at for being there alone
    return a


def route_workspace_size(tokens: int, experts: int, k: int, plan: bool = True) -> int:
    """Bytes of workspace that route needs."""
    return int(load().fqm_route_workspace_size(ctypes.byref(_routing_sizes(tokens, experts, k, 1, None, plan))))


def route(logits: torch.Tensor, k: int, score: str = "softmax", bias: torch.Tensor | None = None, groups: int = 1,
          top_groups: int | None = None, group_score: str = "max", renormalise: bool = True, scale: float = 1.0,
          plan: bool = True, out: Routing | None = None, workspace: torch.Tensor | None = None, stream=None) -> Routing:
    """Each token's k experts, their weights, and the plan that gemm_grouped takes:
    ``gemm_grouped(up, x, r.offsets, src=r.src)``, then
    ``gemm_grouped(down, h, r.offsets, dst=r.dst, row_scale=r.row_scale)`` leaves
    token t's j-th expert's weighted row in row t * k + j.

    logits: [tokens][experts] bf16 or fp32, rows of any stride.  score: "softmax" or
    "sigmoid".  bias: [experts] fp32, added to the scores for the choice alone.
    groups, top_groups: the experts fall into groups of neighbours, of which a
    token chooses from the best ``top_groups``, by their best expert ("max") or the
    sum of their two best ("top2").  renormalise: a token's weights add up to
    ``scale``; without it they are ``scale`` times the scores.
    An expert whose logit is -infinity or NaN is closed to that token; places
    without an open expert get expert -1 and weight 0, and rows of zeros in the
    products.  ``out``: tensors to write to (dense, as Routing describes them)."""
    _need(logits, "logits", _VALUE, dim=2)
    if _elsewhere(stream, logits.device):
        with _inside(stream, logits.device):
            return route(logits, k, score, bias, groups, top_groups, group_score, renormalise, scale, plan, out, workspace)
    dev = logits.device
    T, E = logits.shape
    if out is not None:
        plan = out.offsets is not None
    if top_groups is None:
        top_groups = groups
    ld = _row_stride(logits, "logits", (T, E))
    by, by_group = _one_of(FQM_SCORE, score, "score"), _one_of(FQM_GROUP_SCORE, group_score, "group_score")
    added = _vector(bias, "bias", E, (torch.float32,), dev)
    if not 1 <= E <= 1024 or not 1 <= groups <= 64 or E % groups or not 1 <= top_groups <= groups:
        raise ValueError(f"{E} experts (1 to 1024) in {groups} equal groups (1 to 64), of which {top_groups} stay")
    if not 1 <= k <= min(32, E // groups * top_groups):
        raise ValueError(f"k = {k}: 1 to 32 experts, as many as {top_groups} of {groups} groups of {E} hold at most")
    n = T * k
    if out is None:
        ints = torch.empty(n * (3 if plan else 1) + (E + 1 if plan else 0), dtype=torch.int32, device=dev)
        floats = torch.empty(n * (2 if plan else 1), dtype=torch.float32, device=dev)
        if plan:
            expert, src, dst, offsets = ints.split_with_sizes((n, n, n, E + 1))
            weight, row_scale = floats.split_with_sizes((n, n))
            out = Routing(expert.view(T, k), weight.view(T, k), offsets, src, dst, row_scale)
        else:
            out = Routing(ints.view(T, k), floats.view(T, k), None, None, None, None)
    else:
        for name, shape, dt in (("expert", (T, k), torch.int32), ("weight", (T, k), torch.float32), ("offsets", (E + 1,), torch.int32),
                                ("src", (n,), torch.int32), ("dst", (n,), torch.int32), ("row_scale", (n,), torch.float32)):
            t = getattr(out, name)
            if t is None and not plan and name not in ("expert", "weight"):
                continue
            _need(t, f"out.{name}", (dt,), dev)
            if tuple(t.shape) != shape or not t.is_contiguous():
                raise ValueError(f"out.{name} has shape {tuple(t.shape)}; expected contiguous {shape}")
    rest = (out.offsets.data_ptr(), out.src.data_ptr(), out.dst.data_ptr(), out.row_scale.data_ptr()) if plan else ()
    a = _Routing(T, E, k, logits.data_ptr(), ld, _CODE[logits.dtype], by, added, groups, top_groups, by_group,
                 1 if renormalise else 0, scale, out.expert.data_ptr(), out.weight.data_ptr(), *rest)
    _check_workspace(workspace, dev)
    lib = load()
    if workspace is None:
        need = lib.fqm_route_workspace_size(ctypes.byref(a))
        workspace = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib.fqm_route(ctypes.byref(a), workspace.data_ptr() if workspace is not None else None, ws_bytes, _handle(dev)),
           "fqm_route")
    return out


# ---------------------------------------------------------------------------
# the norms on both sides of a block
# ---------------------------------------------------------------------------
def block_norm(x: torch.Tensor, residual: torch.Tensor | None = None, post_weight: torch.Tensor | None = None,
               weight: torch.Tensor | None = None, gate: torch.Tensor | None = None, gate_act: str | None = None,
               scale: float = 1.0, residual_scale: float = 1.0, eps: float = 1e-6, weight_offset: float = 0.0,
               post: bool = True, out_dtype: torch.dtype | None = torch.bfloat16, y: torch.Tensor | None = None,
               y_scale: torch.Tensor | None = None, total: torch.Tensor | None = None, keep_total: bool = True,
               stream=None) -> NormOut:
    """The norm behind a block, its gate and scales, the residual's addition and
    the norm in front of the next block, in one pass (fp32 inside):
    ``u`` the sum of x's terms, ``v = u / rms(u) * (post_weight + weight_offset)``
    (``u`` itself without ``post``),
    ``h = residual_scale * residual + scale * gate_act(gate) * v``,
    ``y = h / rms(h) * (weight + weight_offset)``.

    x: [rows][cols], or [rows][terms][cols] whose terms are added up; bf16 or
    fp32, rows of any stride.  residual: [rows][cols] or None.  A weight that is
    None is a factor of 1.  gate: [cols], [rows][1] or [rows][cols].  gate_act: an
    activation of ``linear``.  ``total`` gets h in the residual's dtype (x's without
    one) and may be ``residual`` itself; ``keep_total=False`` leaves it out.
    out_dtype: bfloat16, float32, int8 with one scale a row, or None for no second
    norm (y and scale are None then)."""
    _need(x, "x", _VALUE)
    if _elsewhere(stream, x.device):
        with _inside(stream, x.device):
            return block_norm(x, residual, post_weight, weight, gate, gate_act, scale, residual_scale, eps, weight_offset,
                              post, out_dtype, y, y_scale, total, keep_total)
    if x.dim() not in (2, 3):
        raise ValueError(f"x must be [rows][cols] or [rows][terms][cols]; got shape {tuple(x.shape)}")
    dev, rows, cols = x.device, x.shape[0], x.shape[-1]
    terms = x.shape[1] if x.dim() == 3 else 1
    if not 1 <= terms <= 64:
        raise ValueError(f"x has {terms} terms; 1 to 64 can be added up")
    if cols > 1 and x.stride(-1) != 1:
        raise ValueError("x must have dense rows (stride 1 in the last dimension)")
    ld_x, ld_term = x.stride(0) if rows > 1 else cols, x.stride(1) if terms > 1 else cols
    if ld_x < cols or ld_term < cols:
        raise ValueError("x has overlapping rows")
    ld_res = ld_gate = step_gate = ld_total = ld_y = res_dtype = gate_dtype = 0
    total_dtype = x.dtype
    if residual is not None:
        _need(residual, "residual", _VALUE, dev)
        ld_res = _row_stride(residual, "residual", (rows, cols))
        total_dtype = residual.dtype
        res_dtype = _CODE[total_dtype]
    if post_weight is not None and not post:
        raise ValueError("post_weight belongs to the norm that post=False leaves out")
    w1, w2 = _vector(post_weight, "post_weight", cols, _VALUE, dev), _vector(weight, "weight", cols, _VALUE, dev)
    act = _one_of(FQM_ACT, gate_act, "gate_act")
    if gate is not None:
        _need(gate, "gate", _VALUE, dev)
        gate_dtype = _CODE[gate.dtype]
        if gate.dim() == 1 and gate.shape[0] == cols:
            if cols > 1 and gate.stride(0) != 1:
                raise ValueError("gate must be dense (stride 1 in the last dimension)")
            step_gate = 1
        elif gate.dim() == 2 and gate.shape[0] == rows and gate.shape[1] in (1, cols):
            step_gate = 0 if gate.shape[1] == 1 else 1
            if step_gate and cols > 1 and gate.stride(1) != 1:
                raise ValueError("gate must have dense rows (stride 1 in the last dimension)")
            ld_gate = gate.stride(0) if rows > 1 else 0
            if ld_gate and ld_gate < gate.shape[1]:
                raise ValueError("gate has overlapping rows")
        else:
            raise ValueError(f"gate has shape {tuple(gate.shape)}; expected ({cols},), ({rows}, 1) or ({rows}, {cols})")
    elif gate_act is not None:
        raise ValueError("gate_act without a gate")
    if total is not None:
        _need(total, "total", (total_dtype,), dev)
        ld_total = _row_stride(total, "total", (rows, cols))
    elif keep_total:
        total = torch.empty((rows, cols), dtype=total_dtype, device=dev)
        ld_total = cols
    if y is None and out_dtype is not None:
        if out_dtype not in _CODE:
            raise ValueError(f"out_dtype must be bfloat16, float32, int8 or None, not {out_dtype}")
        y = torch.empty((rows, cols), dtype=out_dtype, device=dev)
        ld_y = cols
    elif y is not None:
        _need(y, "y", tuple(_CODE), dev)
        ld_y = _row_stride(y, "y", (rows, cols))
    if y is None and total is None:
        raise ValueError("nothing to compute: neither y nor total is asked for")
    if y is not None and y.dtype == torch.int8:
        if y_scale is None:
            y_scale = torch.empty(rows, dtype=torch.float32, device=dev)
        _vector(y_scale, "y_scale", rows, (torch.float32,), dev)
    else:
        y_scale = None
    a = _Block(rows, cols, terms, 1 if post else 0, _CODE[x.dtype], res_dtype, 0 if w1 is None else _CODE[post_weight.dtype],
               0 if w2 is None else _CODE[weight.dtype], gate_dtype, 0 if y is None else _CODE[y.dtype], act, eps, weight_offset,
               scale, residual_scale, x.data_ptr(), ld_x, ld_term, w1, None if gate is None else gate.data_ptr(), ld_gate, step_gate,
               None if residual is None else residual.data_ptr(), ld_res, w2, None if total is None else total.data_ptr(), ld_total,
               None if y is None else y.data_ptr(), ld_y, None if y_scale is None else y_scale.data_ptr())
    _check(load().fqm_block_norm(ctypes.byref(a), _handle(dev)), "fqm_block_norm")
    return NormOut(y, y_scale, total)
