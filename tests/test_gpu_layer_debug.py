"""The debug checks on the operators around the products: correct calls pass
and match, buffers shorter than their shapes are refused before anything is
enqueued."""
import ctypes

import pytest
import torch

import dequant_matmul_amd as fqm
from gpu_common import DEV, lut6_weights

pytestmark = pytest.mark.gpu

BOUNDS = 9


@pytest.fixture
def debug():
    prev = fqm.set_debug(True)
    yield
    fqm.set_debug(prev)


def calls():
    x = torch.randn(6, 512, device=DEV).to(torch.bfloat16)
    ad = fqm.Adapters(torch.randn(2, 16, 512, device=DEV).to(torch.bfloat16), torch.randn(2, 40, 16, device=DEV).to(torch.bfloat16))
    index = torch.tensor([0, 1, -1, 0, 1, 1], dtype=torch.int32, device=DEV)
    w = lut6_weights(256, 512, 1)
    off = torch.tensor([0, 2, 2, 5, 6], dtype=torch.int32, device=DEV)
    order = torch.tensor([3, 1, 0, 5, 2, 4], dtype=torch.int32, device=DEV)
    q = torch.randint(-127, 128, (6, 512), dtype=torch.int8, device=DEV)
    return [lambda: fqm.add_rms_norm(x, residual=x, out_dtype=torch.int8).y,
            lambda: fqm.lora(ad, x, index),
            lambda: fqm.gemm_grouped(w, x, off),
            lambda: fqm.gemm_grouped(w, q, off, x_scale=torch.ones(6, device=DEV), src=index, dst=order)]


def test_correct_calls_pass_and_match(debug):
    cs = calls()
    checked = [c().clone() for c in cs]
    fqm.set_debug(False)
    for c, v in zip(cs, checked):
        assert torch.equal(c(), v)


def test_short_and_host_buffers_are_refused(debug):
    lib = fqm.load()
    # more rows than any allocation of this process holds
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV)
    a = fqm._Norm(1 << 30, 64, 1, 0, 0, 0, 0, 1e-6, x.data_ptr(), 64, 64)
    a.y, a.ld_y = x.data_ptr(), 64
    assert lib.fqm_add_rms_norm(ctypes.byref(a), None) == BOUNDS
    host = torch.zeros(4, 64, dtype=torch.bfloat16)
    a.rows, a.y = 4, host.data_ptr()
    assert lib.fqm_add_rms_norm(ctypes.byref(a), None) == BOUNDS
    ad = fqm.Adapters(torch.zeros(2, 16, 64, dtype=torch.bfloat16, device=DEV),
                      torch.zeros(2, 40, 16, dtype=torch.bfloat16, device=DEV))
    index = torch.zeros(4, dtype=torch.int32, device=DEV)
    ws = torch.zeros(1 << 16, dtype=torch.uint8, device=DEV)
    y = torch.zeros(4, 40, dtype=torch.bfloat16, device=DEV)
    args = [ad.ref, x.data_ptr(), index.data_ptr(), None, 0, y.data_ptr(), 0, 4, ws.data_ptr(), ws.numel(), None]
    assert lib.fqm_lora(*args) == 0
    args[5] = host.data_ptr()
    assert lib.fqm_lora(*args) == BOUNDS
    w = lut6_weights(256, 512, 1)
    off = torch.zeros(5, dtype=torch.int32, device=DEV)
    X = torch.zeros(4, 512, dtype=torch.bfloat16, device=DEV)
    g = fqm._Groups(4, off.data_ptr(), 4, X.data_ptr(), 0, 4, None, None, y.data_ptr(), 0, 1 << 28, None, None)
    assert lib.fqm_gemm_grouped(w.ref, ctypes.byref(g), None, 0, None) == BOUNDS
