"""The operators around the products, on the CPU: what a grouped call needs is asked for before its buffers exist, and a
stream has to be the operands' device's."""
import ctypes
import os

import pytest
import torch

import dequant_matmul_amd as fqm
from dequant_matmul_amd import _layer
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


class Stream:
    """What the binding looks at of a stream, without a GPU."""

    def __init__(self, index):
        self.device = torch.device("cuda", index)


def test_a_stream_of_another_device_is_refused():
    """Making it current would leave the operands' device, and the call would run on that device's own stream."""
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        _layer._elsewhere(Stream(1), torch.device("cuda", 0))
    assert _layer._elsewhere(Stream(1), torch.device("cuda", 1))
