"""What a grouped call needs is asked for before its buffers exist: sizes and types decide, on the CPU."""
import ctypes
import os

import pytest

import dequant_matmul_amd as fqm
from test_layer_abi import FAKE, GROUPS, filled, lut6


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fqm.LIB_PATH):
        from dequant_matmul_amd import build
        build.build()
    return fqm.load()


@pytest.mark.parametrize("over", [
    dict(M=7, x_rows=7, y_rows=7), dict(M=900, x_rows=900, y_rows=900), dict(M=900, x_rows=900, y_rows=900, x_dtype=2, x_scale=FAKE),
    dict(M=900, x_rows=20, y_rows=900, src=FAKE), dict(M=900, x_rows=900, y_rows=5, dst=FAKE),
])
def test_grouped_workspace_needs_no_buffers(lib, over):
    w = lut6(rows=3 * 512, cols=1024, ld=768)
    g = filled(fqm._Groups, GROUPS, over)
    need = lib.fqm_gemm_grouped_workspace_size(ctypes.byref(w), ctypes.byref(g))
    assert need > 0
    for name in ("offsets", "X", "x_scale", "Y", "row_scale"):
        setattr(g, name, None)
    assert lib.fqm_gemm_grouped_workspace_size(ctypes.byref(w), ctypes.byref(g)) == need
    # the call itself does need them
    assert lib.fqm_gemm_grouped(ctypes.byref(w), ctypes.byref(g), FAKE, need, None) == 1
    g.x_rows = -1
    assert lib.fqm_gemm_grouped_workspace_size(ctypes.byref(w), ctypes.byref(g)) == 0
