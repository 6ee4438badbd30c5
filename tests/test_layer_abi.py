"""Refusals of the operators around the products, on the CPU: the C ABI's
argument checks (fake addresses, never dereferenced) and the binding's."""
import ctypes
import os

import numpy as np
import pytest
import torch

import dequant_matmul_amd as fqm
import oracle

E = dict(OK=0, NULL=1, ALIGN=2, SHAPE=3, FORMAT=4, WORKSPACE=5, UNSUPPORTED=6, HIP=7, SCRATCH=8, BOUNDS=9)
FAKE = 0x7f0000000000


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fqm.LIB_PATH):
        from dequant_matmul_amd import build
        build.build()
    return fqm.load()


@pytest.fixture
def stopped(lib):
    """Arguments that pass the checks stop at the allocation checks: nothing is launched."""
    prev = lib.fqm_set_debug(1)
    yield lib
    lib.fqm_set_debug(prev)


def filled(cls, base, over):
    a = cls()
    for k, v in {**base, **over}.items():
        setattr(a, k, v)
    return a


NORM = dict(rows=4, cols=64, terms=1, eps=1e-6, x=FAKE, ld_x=64, residual=FAKE, ld_res=64, weight=FAKE, total=FAKE,
            ld_total=64, y=FAKE, ld_y=64)


@pytest.mark.parametrize("over,code", [
    (dict(), "BOUNDS"), (dict(rows=0), "OK"), (dict(rows=-1), "SHAPE"), (dict(cols=32769, ld_x=40000), "SHAPE"),
    (dict(terms=0), "SHAPE"), (dict(terms=65, ld_term=64), "SHAPE"), (dict(terms=2, ld_term=63), "SHAPE"),
    (dict(terms=2, ld_term=64), "BOUNDS"), (dict(x_dtype=2), "FORMAT"), (dict(res_dtype=5), "FORMAT"),
    (dict(weight_dtype=2), "FORMAT"), (dict(y_dtype=3), "FORMAT"), (dict(eps=-1.0), "FORMAT"),
    (dict(eps=float("nan")), "FORMAT"), (dict(eps=float("inf")), "FORMAT"), (dict(x=None), "NULL"),
    (dict(y=None), "NULL"), (dict(y_dtype=2), "NULL"), (dict(y_dtype=2, y_scale=FAKE + 2), "ALIGN"),
    (dict(y_dtype=2, y_scale=FAKE, y=FAKE + 1), "BOUNDS"), (dict(ld_x=63), "SHAPE"), (dict(ld_res=0), "SHAPE"),
    (dict(residual=None, ld_res=0), "BOUNDS"), (dict(ld_total=63), "SHAPE"), (dict(ld_y=63), "SHAPE"),
    (dict(ld_x=1 << 62), "SHAPE"), (dict(x=FAKE + 1), "ALIGN"), (dict(x=FAKE + 2), "BOUNDS"),
    (dict(x_dtype=1, x=FAKE + 2), "ALIGN"), (dict(total=FAKE + 1), "ALIGN"), (dict(weight=None), "BOUNDS"),
    (dict(cols=0, ld_x=0, x=None, y=None), "OK"),
])
def test_norm_arguments(stopped, over, code):
    assert stopped.fqm_add_rms_norm(ctypes.byref(filled(fqm._Norm, NORM, over)), None) == E[code]


def test_norm_null(lib):
    assert lib.fqm_add_rms_norm(None, None) == E["NULL"]


ADAPT = dict(count=3, rank=16, rows=40, cols=64, A=FAKE, ld_A=64, B=FAKE, ld_B=16)


@pytest.mark.parametrize("over,call,code", [
    (dict(), {}, "BOUNDS"), (dict(count=0), {}, "FORMAT"), (dict(rank=0), {}, "FORMAT"), (dict(rank=257, ld_B=264), {}, "FORMAT"),
    (dict(rows=-1), {}, "SHAPE"), (dict(cols=60), {}, "SHAPE"), (dict(rows=0), {}, "OK"), (dict(A=None), {}, "NULL"),
    (dict(B=None), {}, "NULL"), (dict(ld_A=56), {}, "SHAPE"), (dict(ld_A=68), {}, "ALIGN"), (dict(ld_B=8), {}, "SHAPE"),
    (dict(ld_B=20), {}, "ALIGN"), (dict(A=FAKE + 2), {}, "ALIGN"), (dict(ld_B=1 << 59), {}, "SHAPE"),
    (dict(scale=FAKE + 2), {}, "ALIGN"), (dict(ranks=FAKE + 1), {}, "ALIGN"),
    (dict(), dict(M=0), "OK"), (dict(), dict(M=-1), "SHAPE"), (dict(), dict(M=(1 << 24) + 1), "SHAPE"),
    (dict(), dict(x=None), "NULL"), (dict(), dict(index=None), "NULL"), (dict(), dict(y=None), "NULL"),
    (dict(), dict(x=FAKE + 8), "ALIGN"), (dict(), dict(y=FAKE + 1), "ALIGN"), (dict(), dict(base=FAKE + 3), "ALIGN"),
    (dict(), dict(ydt=2), "FORMAT"), (dict(), dict(bdt=2), "FORMAT"), (dict(), dict(bdt=2, base=None), "BOUNDS"),
    (dict(), dict(base=FAKE + 64, y=FAKE + 64, ydt=1), "FORMAT"), (dict(), dict(base=FAKE + 64, y=FAKE + 64), "BOUNDS"),
    (dict(), dict(ws=None), "WORKSPACE"), (dict(), dict(wsb=4), "WORKSPACE"), (dict(), dict(ws=FAKE + 4), "ALIGN"),
])
def test_lora_arguments(stopped, over, call, code):
    a = filled(fqm._Adapters, ADAPT, over)
    c = {**dict(x=FAKE, index=FAKE, base=FAKE, bdt=0, y=FAKE + 4096, ydt=0, M=5, ws=FAKE, wsb=1 << 30), **call}
    assert stopped.fqm_lora(ctypes.byref(a), c["x"], c["index"], c["base"], c["bdt"], c["y"], c["ydt"], c["M"], c["ws"],
                            c["wsb"], None) == E[code]


def test_lora_workspace_of_bad_arguments_is_nothing(lib):
    assert lib.fqm_lora(None, FAKE, FAKE, None, 0, FAKE, 0, 1, None, 0, None) == E["NULL"]
    a = filled(fqm._Adapters, ADAPT, {})
    assert lib.fqm_lora_workspace_size(ctypes.byref(a), 4) >= 4 * 16 * 4
    assert lib.fqm_lora_workspace_size(ctypes.byref(a), 0) == 0
    assert lib.fqm_lora_workspace_size(ctypes.byref(filled(fqm._Adapters, ADAPT, dict(rank=0))), 4) == 0


def lut6(rows=60, cols=128, ld=96, fmt=fqm.FQM_LUT6):
    w = fqm._Weights()
    w.format, w.rows, w.cols = fmt, rows, cols
    w.lut6.packed, w.lut6.lut, w.lut6.ld = FAKE, FAKE, ld
    w.lut4.packed, w.lut4.lut, w.lut4.ld = FAKE, FAKE, ld
    return w


GROUPS = dict(count=3, offsets=FAKE, M=7, X=FAKE, x_rows=7, Y=FAKE, y_rows=7)


@pytest.mark.parametrize("wts,over,code", [
    ({}, dict(), "BOUNDS"), (dict(fmt=fqm.FQM_LUT4), dict(), "BOUNDS"), (dict(cols=100), dict(), "SHAPE"),
    (dict(rows=61), dict(), "SHAPE"), (dict(rows=0), dict(), "OK"), ({}, dict(count=0), "FORMAT"),
    ({}, dict(count=4097), "FORMAT"), ({}, dict(M=0), "OK"), ({}, dict(M=-1), "SHAPE"), ({}, dict(M=(1 << 24) + 1), "SHAPE"),
    ({}, dict(x_dtype=1), "FORMAT"), ({}, dict(y_dtype=2), "FORMAT"), ({}, dict(x_dtype=2), "NULL"),
    ({}, dict(x_dtype=2, x_scale=FAKE), "BOUNDS"), ({}, dict(x_dtype=2, x_scale=FAKE + 2), "ALIGN"),
    ({}, dict(x_rows=6), "SHAPE"), ({}, dict(x_rows=6, src=FAKE), "BOUNDS"), ({}, dict(y_rows=6), "SHAPE"),
    ({}, dict(y_rows=6, dst=FAKE), "BOUNDS"), ({}, dict(offsets=None), "NULL"), ({}, dict(X=None), "NULL"),
    ({}, dict(Y=None), "NULL"), ({}, dict(X=FAKE + 8), "ALIGN"), ({}, dict(Y=FAKE + 8), "ALIGN"),
    ({}, dict(offsets=FAKE + 2), "ALIGN"), ({}, dict(src=FAKE + 1), "ALIGN"), ({}, dict(dst=FAKE + 1), "ALIGN"),
    ({}, dict(row_scale=FAKE + 1), "ALIGN"), ({}, dict(x_rows=(1 << 31) // 256, src=FAKE), "SHAPE"),
])
def test_grouped_arguments(stopped, wts, over, code):
    g = filled(fqm._Groups, GROUPS, over)
    assert stopped.fqm_gemm_grouped(ctypes.byref(lut6(**wts)), ctypes.byref(g), FAKE, 1 << 40, None) == E[code]


def test_grouped_formats_and_null(lib):
    g = filled(fqm._Groups, GROUPS, {})
    assert lib.fqm_gemm_grouped(None, ctypes.byref(g), None, 0, None) == E["NULL"]
    assert lib.fqm_gemm_grouped(ctypes.byref(lut6()), None, None, 0, None) == E["NULL"]
    w = fqm._Weights()
    w.format, w.rows, w.cols = fqm.FQM_MDBF, 0, 64
    w.mdbf.r, w.mdbf.l, w.mdbf.P = 4, 1, 1
    assert lib.fqm_gemm_grouped(ctypes.byref(w), ctypes.byref(g), None, 0, None) == E["UNSUPPORTED"]
    assert lib.fqm_gemm_grouped_workspace_size(ctypes.byref(w), ctypes.byref(g)) == 0


# ---- the binding: tensors on the CPU and wrong layouts are refused before any call ----
def test_binding_refuses_cpu_tensors():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU tensors"):
        fqm.add_rms_norm(x)
    with pytest.raises(ValueError, match="GPU tensors"):
        fqm.Adapters(torch.zeros(1, 4, 64, dtype=torch.bfloat16), torch.zeros(1, 8, 4, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="must be a torch.Tensor"):
        fqm.add_rms_norm([1.0])
    with pytest.raises(ValueError, match="dtype"):
        fqm.add_rms_norm(torch.zeros(2, 64, dtype=torch.float16))
    with pytest.raises(ValueError, match="Lut6Weights or Lut4Weights"):
        fqm.gemm_grouped(object(), x, torch.zeros(2, dtype=torch.int32))


# ---- the oracle's definitions, pinned to something other than themselves ----
def test_oracle_norm_has_unit_mean_square():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 3, 40))
    o = oracle.layer.add_rms_norm(x, None, None, 0.0)
    assert np.allclose((o["y"] ** 2).mean(axis=1), 1)
    assert np.allclose(o["total"], x[:, 0] + x[:, 1] + x[:, 2])
    assert np.allclose(o["scale"] * 127, np.abs(o["y"]).max(axis=1))


def test_oracle_lora_and_grouped_are_the_dense_products():
    rng = np.random.default_rng(1)
    A, B, x = rng.standard_normal((2, 3, 8)), rng.standard_normal((2, 5, 3)), rng.standard_normal((4, 8))
    y, _ = oracle.layer.lora(A, B, np.array([2.0, 1.0]), None, x, [0, 1, 0, -1], np.ones((4, 5)))
    assert np.allclose(y[[0, 2]], 1 + 2 * x[[0, 2]] @ (B[0] @ A[0]).T)
    assert np.allclose(y[1], 1 + B[1] @ A[1] @ x[1]) and np.allclose(y[3], 1)
    W = rng.standard_normal((2, 5, 8))
    Y, _ = oracle.layer.grouped(W, [0, 1, 3], x, [3, 0, 9], [2, 0, 1], [1.0, 2.0, 3.0], 4, 7.0)
    assert np.allclose(Y[2], W[0] @ x[3]) and np.allclose(Y[0], 2 * W[1] @ x[0])
    assert (Y[1] == 0).all() and (Y[3] == 7).all()
