"""The debug checks on the product with its epilogue, the routing and the norms around a block: correct calls pass and
match, buffers shorter than their shapes and host buffers are refused before anything is enqueued."""
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
    w = lut6_weights(256, 512, 1)
    x = torch.randn(70, 512, device=DEV).to(torch.bfloat16)
    res = torch.randn(70, 128, device=DEV)
    gate = torch.randn(70, 512, device=DEV)
    logits = torch.randn(300, 16, device=DEV)
    return [lambda: fqm.linear(w, x[:1], act="gelu"),
            lambda: fqm.linear(w, x[:20], torch.zeros(256, device=DEV), act="silu", gated=True, residual=res[:20]),
            lambda: fqm.linear(w, x, act="silu", gated=True, residual=res),
            lambda: fqm.route(logits[:3], 4).row_scale,
            lambda: fqm.route(logits, 4, bias=torch.zeros(16, device=DEV)).row_scale,
            lambda: fqm.block_norm(x, x, weight=gate[0].contiguous(), gate=gate, out_dtype=torch.int8).y]


def test_correct_calls_pass_and_match(debug):
    cs = calls()
    checked = [c().clone() for c in cs]
    fqm.set_debug(False)
    for c, v in zip(cs, checked):
        assert torch.equal(c(), v)


def test_short_and_host_buffers_are_refused(debug):
    lib = fqm.load()
    host = torch.zeros(1 << 12)
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV)
    # more rows than any allocation of this process holds
    b = fqm._Block(rows=1 << 30, cols=64, terms=1, post=1, eps=1e-6, scale=1.0, x=x.data_ptr(), ld_x=64, ld_term=64, y=x.data_ptr(), ld_y=64)
    assert lib.fqm_block_norm(ctypes.byref(b), None) == BOUNDS
    b.rows, b.y = 4, host.data_ptr()
    assert lib.fqm_block_norm(ctypes.byref(b), None) == BOUNDS
    w = lut6_weights(64, 64, 1)
    a = fqm._Epilogue(M=1, X=x.data_ptr(), ld_x=64, Y=host.data_ptr(), ld_y=64, y_dtype=1)
    assert lib.fqm_linear(w.ref, ctypes.byref(a), None, 0, None) == BOUNDS
    out = torch.zeros(64, device=DEV)
    a.Y, a.bias, a.bias_dtype = out.data_ptr(), host.data_ptr(), 1
    assert lib.fqm_linear(w.ref, ctypes.byref(a), None, 0, None) == BOUNDS
    logits = torch.zeros(4, 16, device=DEV)
    ints, floats = torch.zeros(64, dtype=torch.int32, device=DEV), torch.zeros(64, device=DEV)
    r = fqm._Routing(T=4, E=16, k=2, logits=logits.data_ptr(), ld_x=16, x_dtype=1, groups=1, top_groups=1, scale=1.0,
                     expert=ints.data_ptr(), weight=host.data_ptr())
    assert lib.fqm_route(ctypes.byref(r), None, 0, None) == BOUNDS
    r.weight, r.T, r.logits = floats.data_ptr(), 4, host.data_ptr()
    assert lib.fqm_route(ctypes.byref(r), None, 0, None) == BOUNDS
    torch.cuda.synchronize()
