"""Refusals of the product with its epilogue, the routing and the block's norms, on the CPU: the C ABI's argument
checks (fake addresses, never dereferenced) and the binding's; the oracle's definitions against others."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

import dequant_matmul_amd as fqm
import oracle
from test_layer_abi import E, FAKE, filled, lut6


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


LINEAR = dict(M=5, X=FAKE, ld_x=128, act=2, bias=FAKE, residual=FAKE, ld_res=60, Y=FAKE + 4096, ld_y=60)


@pytest.mark.parametrize("wts,over,code", [
    ({}, dict(), "BOUNDS"), (dict(fmt=fqm.FQM_LUT4), dict(), "BOUNDS"), ({}, dict(gated=1, ld_y=30, ld_res=30), "BOUNDS"),
    ({}, dict(gated=1, ld_y=29), "SHAPE"), (dict(rows=61), dict(gated=1), "SHAPE"), ({}, dict(gated=2), "FORMAT"),
    ({}, dict(M=0), "OK"), ({}, dict(M=-1), "SHAPE"), ({}, dict(M=(1 << 24) + 1), "SHAPE"), (dict(rows=0), dict(), "OK"),
    (dict(cols=100), dict(), "SHAPE"), (dict(cols=1 << 22, ld=1 << 22), dict(ld_x=1 << 22), "SHAPE"),
    (dict(rows=(1 << 24) + 2), dict(), "SHAPE"), ({}, dict(act=7), "FORMAT"), ({}, dict(act=-1), "FORMAT"),
    ({}, dict(y_dtype=2), "FORMAT"), ({}, dict(bias_dtype=2), "FORMAT"), ({}, dict(res_dtype=2), "FORMAT"),
    ({}, dict(bias_dtype=2, bias=None), "BOUNDS"), ({}, dict(X=None), "NULL"), ({}, dict(Y=None), "NULL"),
    ({}, dict(ld_x=127), "SHAPE"), ({}, dict(ld_x=132), "ALIGN"), ({}, dict(ld_x=(1 << 21) + 8), "SHAPE"),
    ({}, dict(X=FAKE + 8), "ALIGN"), ({}, dict(Y=FAKE + 1), "ALIGN"), ({}, dict(Y=FAKE + 2), "BOUNDS"),
    ({}, dict(bias=FAKE + 1), "ALIGN"), ({}, dict(residual=FAKE + 1), "ALIGN"), ({}, dict(ld_y=59), "SHAPE"),
    ({}, dict(ld_res=59), "SHAPE"), ({}, dict(ld_y=1 << 62), "SHAPE"),
    ({}, dict(residual=FAKE + 4096, y_dtype=1), "FORMAT"), ({}, dict(residual=FAKE + 4096, ld_res=61), "FORMAT"),
    ({}, dict(residual=FAKE + 4096), "BOUNDS"),
])
def test_linear_arguments(stopped, wts, over, code):
    a = filled(fqm._Epilogue, LINEAR, over)
    assert stopped.fqm_linear(ctypes.byref(lut6(**wts)), ctypes.byref(a), FAKE, 1 << 40, None) == E[code]


def test_linear_formats_null_and_workspace(lib):
    a = filled(fqm._Epilogue, LINEAR, {})
    assert lib.fqm_linear(None, ctypes.byref(a), None, 0, None) == E["NULL"]
    assert lib.fqm_linear(ctypes.byref(lut6()), None, None, 0, None) == E["NULL"]
    w = fqm._Weights()
    w.format, w.rows, w.cols = fqm.FQM_MDBF, 0, 64
    w.mdbf.r, w.mdbf.l, w.mdbf.P = 4, 1, 1
    assert lib.fqm_linear(ctypes.byref(w), ctypes.byref(a), None, 0, None) == E["UNSUPPORTED"]
    assert lib.fqm_linear_workspace_size(ctypes.byref(w), ctypes.byref(a)) == 0
    big = lut6(rows=1024, cols=8192, ld=8192)
    sizes = filled(fqm._Epilogue, dict(M=40), {})  # sizes alone: no buffers yet
    need = lib.fqm_linear_workspace_size(ctypes.byref(big), ctypes.byref(sizes))
    assert need > 0
    a = filled(fqm._Epilogue, dict(LINEAR, M=40, ld_x=8192, ld_y=1024, ld_res=1024), {})
    call = lambda ws, n: lib.fqm_linear(ctypes.byref(big), ctypes.byref(a), ws, n, None)  # noqa: E731
    assert call(None, need) == call(FAKE, need - 1) == E["WORKSPACE"]
    assert call(FAKE + 4, need) == E["ALIGN"]


@pytest.mark.parametrize("gated", [0, 1])
def test_linear_workspace_goes_by_the_row_stride_as_well(stopped, gated):
    """Rows of codes so far apart that 32-bit offsets do not reach both matrices take another kernel: the size asked for
    the same descriptor is enough, one byte less is refused."""
    sizes = []
    for ld in (768, 1 << 18, 1 << 19):
        w = lut6(rows=16384, cols=1024, ld=ld)
        a = filled(fqm._Epilogue, dict(LINEAR, M=16, ld_x=1024, ld_y=16384, ld_res=16384, gated=gated), {})
        need = stopped.fqm_linear_workspace_size(ctypes.byref(w), ctypes.byref(a))
        sizes.append(need)
        call = lambda n: stopped.fqm_linear(ctypes.byref(w), ctypes.byref(a), FAKE, n, None)  # noqa: E731
        assert call(need) == E["BOUNDS"]
        assert need == 0 or call(need - 1) == E["WORKSPACE"]
    assert gated == 0 or sizes[0] != sizes[2]


ROUTE = dict(T=9, E=24, k=3, logits=FAKE, ld_x=24, x_dtype=1, groups=4, top_groups=2, scale=1.0, expert=FAKE, weight=FAKE,
             offsets=FAKE, src=FAKE, dst=FAKE, row_scale=FAKE)


@pytest.mark.parametrize("over,code", [
    (dict(), "BOUNDS"), (dict(T=-1), "SHAPE"), (dict(T=1 << 24), "SHAPE"), (dict(E=0), "FORMAT"), (dict(E=1025), "FORMAT"),
    (dict(k=0), "FORMAT"), (dict(k=33), "FORMAT"), (dict(k=13), "SHAPE"), (dict(k=12), "BOUNDS"), (dict(groups=0), "FORMAT"),
    (dict(groups=65), "FORMAT"), (dict(groups=5), "SHAPE"), (dict(top_groups=0), "FORMAT"), (dict(top_groups=5), "FORMAT"),
    (dict(x_dtype=2), "FORMAT"), (dict(score=2), "FORMAT"), (dict(group_score=-1), "FORMAT"), (dict(renormalise=2), "FORMAT"),
    (dict(scale=math.inf), "FORMAT"), (dict(scale=math.nan), "FORMAT"), (dict(logits=None), "NULL"), (dict(expert=None), "NULL"),
    (dict(weight=None), "NULL"), (dict(src=None), "NULL"), (dict(dst=None), "NULL"), (dict(row_scale=None), "NULL"),
    (dict(offsets=None, src=None, dst=None, row_scale=None), "BOUNDS"), (dict(ld_x=23), "SHAPE"), (dict(ld_x=1 << 61), "SHAPE"),
    (dict(logits=FAKE + 2), "ALIGN"), (dict(logits=FAKE + 2, x_dtype=0), "BOUNDS"), (dict(bias=FAKE + 2), "ALIGN"),
    (dict(offsets=FAKE + 2), "ALIGN"), (dict(src=FAKE + 1), "ALIGN"), (dict(T=0, offsets=None), "OK"),
])
def test_route_arguments(stopped, over, code):
    a = filled(fqm._Routing, ROUTE, over)
    assert stopped.fqm_route(ctypes.byref(a), FAKE, 1 << 30, None) == E[code]


def test_route_null_and_workspace(lib):
    assert lib.fqm_route(None, None, 0, None) == E["NULL"]
    a = filled(fqm._Routing, ROUTE, dict(T=40000))
    need = lib.fqm_route_workspace_size(ctypes.byref(a))
    assert need > 0
    assert lib.fqm_route(ctypes.byref(a), None, need, None) == lib.fqm_route(ctypes.byref(a), FAKE, need - 1, None) == E["WORKSPACE"]
    assert lib.fqm_route(ctypes.byref(a), FAKE + 4, need, None) == E["ALIGN"]
    a.offsets = None
    assert lib.fqm_route_workspace_size(ctypes.byref(a)) == 0


BLOCK = dict(rows=4, cols=64, terms=1, post=1, eps=1e-6, scale=1.0, residual_scale=1.0, x=FAKE, ld_x=64, residual=FAKE, ld_res=64,
             post_weight=FAKE, weight=FAKE, gate=FAKE, ld_gate=64, step_gate=1, total=FAKE, ld_total=64, y=FAKE, ld_y=64)


@pytest.mark.parametrize("over,code", [
    (dict(), "BOUNDS"), (dict(rows=0), "OK"), (dict(rows=-1), "SHAPE"), (dict(cols=32769, ld_x=40000), "SHAPE"),
    (dict(terms=0), "SHAPE"), (dict(terms=65, ld_term=64), "SHAPE"), (dict(terms=2, ld_term=63), "SHAPE"),
    (dict(x_dtype=2), "FORMAT"), (dict(res_dtype=5), "FORMAT"), (dict(post_dtype=2), "FORMAT"), (dict(weight_dtype=2), "FORMAT"),
    (dict(gate_dtype=2), "FORMAT"), (dict(y_dtype=3), "FORMAT"), (dict(gate_act=7), "FORMAT"), (dict(post=2), "FORMAT"),
    (dict(eps=-1.0), "FORMAT"), (dict(eps=math.nan), "FORMAT"), (dict(scale=math.inf), "FORMAT"),
    (dict(residual_scale=math.nan), "FORMAT"), (dict(weight_offset=-math.inf), "FORMAT"), (dict(step_gate=2), "FORMAT"),
    (dict(x=None), "NULL"), (dict(y=None), "BOUNDS"), (dict(y=None, total=None), "NULL"), (dict(y_dtype=2), "NULL"),
    (dict(y_dtype=2, y=None), "BOUNDS"), (dict(y_dtype=2, y_scale=FAKE + 2), "ALIGN"), (dict(y_dtype=2, y_scale=FAKE, y=FAKE + 1), "BOUNDS"),
    (dict(ld_x=63), "SHAPE"), (dict(ld_res=0), "SHAPE"), (dict(residual=None, ld_res=0), "BOUNDS"), (dict(ld_total=63), "SHAPE"),
    (dict(ld_y=63), "SHAPE"), (dict(ld_gate=63), "SHAPE"), (dict(ld_gate=0), "BOUNDS"), (dict(ld_gate=1, step_gate=0), "BOUNDS"),
    (dict(ld_gate=-1, step_gate=0), "SHAPE"), (dict(x=FAKE + 1), "ALIGN"), (dict(x=FAKE + 2), "BOUNDS"), (dict(gate=FAKE + 1), "ALIGN"),
    (dict(gate_dtype=1, gate=FAKE + 2), "ALIGN"), (dict(total=FAKE + 1), "ALIGN"), (dict(total=FAKE, ld_total=65), "SHAPE"),
    (dict(cols=0, ld_x=0, x=None, y=None), "OK"), (dict(cols=0, y_dtype=2), "NULL"),
])
def test_block_arguments(stopped, over, code):
    assert stopped.fqm_block_norm(ctypes.byref(filled(fqm._Block, BLOCK, over)), None) == E[code]


def test_block_null(lib):
    assert lib.fqm_block_norm(None, None) == E["NULL"]


def test_structs_are_the_headers_size(lib):
    """Fields in the header's order, naturally aligned."""
    assert ctypes.sizeof(fqm._Epilogue) == 88
    assert ctypes.sizeof(fqm._Routing) == 120
    assert ctypes.sizeof(fqm._Block) == 192


def test_binding_refuses_on_the_host():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU tensors"):
        fqm.linear(object(), x)
    with pytest.raises(ValueError, match="GPU tensors"):
        fqm.route(x, 2)
    with pytest.raises(ValueError, match="GPU tensors"):
        fqm.block_norm(x)
    for call in (lambda t: fqm.linear(None, t), lambda t: fqm.route(t, 1), fqm.block_norm):
        with pytest.raises(ValueError, match="must be a torch.Tensor"):
            call([1.0])
    with pytest.raises(ValueError, match="dtype"):
        fqm.linear(object(), torch.zeros(2, 64))
    with pytest.raises(ValueError, match="dtype"):
        fqm.route(torch.zeros(2, 64, dtype=torch.float16), 2)


# ---- the oracle's definitions, pinned to something other than themselves ----
@pytest.mark.parametrize("name,torch_name", [("relu", "relu"), ("silu", "silu"), ("gelu", "gelu"), ("sigmoid", "sigmoid"), ("tanh", "tanh")])
def test_oracle_activations_are_torchs(name, torch_name):
    v = np.linspace(-12, 12, 301)
    f = getattr(torch.nn.functional, torch_name)
    y, b, slope = oracle.block.act(v, name)
    assert np.allclose(y, f(torch.from_numpy(v)).numpy(), rtol=1e-9, atol=1e-12)
    assert (np.abs(np.diff(y)) <= slope * np.diff(v) + 1e-12).all()
    assert (np.abs(f(torch.from_numpy(v).float()).numpy()[b > 0] - y[b > 0]) < 1e-5).all()


def test_oracle_gelu_tanh_is_torchs():
    v = np.linspace(-12, 12, 301)
    want = torch.nn.functional.gelu(torch.from_numpy(v), approximate="tanh").numpy()
    assert np.allclose(oracle.block.act(v, "gelu_tanh")[0], want, rtol=1e-9, atol=1e-12)


def test_oracle_linear_is_the_dense_layer():
    rng = np.random.default_rng(2)
    W, x, b, r = rng.standard_normal((6, 8)), rng.standard_normal((4, 8)), rng.standard_normal(6), rng.standard_normal((4, 3))
    y, bound = oracle.block.linear(W, x, b, "silu", True, r)
    t = torch.nn.functional.linear(*(torch.from_numpy(v) for v in (x, W, b)))
    want = torch.from_numpy(r) + torch.nn.functional.silu(t[:, :3]) * t[:, 3:]
    assert np.allclose(y, want.numpy())
    # the same in fp32: its roundings stay within the bound on them
    t = torch.nn.functional.linear(*(torch.from_numpy(v).float() for v in (x, W, b)))
    single = torch.from_numpy(r).float() + torch.nn.functional.silu(t[:, :3]) * t[:, 3:]
    rounded_inputs, _ = oracle.block.linear(*(v.astype(np.float32).astype(np.float64) for v in (W, x, b)), "silu", True,
                                            r.astype(np.float32).astype(np.float64))
    assert (np.abs(single.double().numpy() - rounded_inputs) <= bound).all()


def test_oracle_route_is_topk_of_softmax():
    rng = np.random.default_rng(3)
    l = rng.standard_normal((20, 12))
    o = oracle.block.route(l, 4, "softmax", None, 1, 1, "max", False, 2.0)
    w, e = torch.topk(torch.softmax(torch.from_numpy(l), 1), 4)
    assert np.array_equal(o["expert"], e.numpy()) and np.allclose(o["weight"], 2 * w.numpy())
    assert o["offsets"][-1] == 80 and np.array_equal(np.bincount(e.numpy().ravel(), minlength=12), np.diff(o["offsets"]))
    assert np.array_equal(o["dst"], np.argsort(e.numpy().ravel(), kind="stable")) and np.array_equal(o["src"], o["dst"] // 4)
    # two groups of six, one kept: all of a token's experts from the group of the larger sum of two
    o = oracle.block.route(l, 4, "sigmoid", np.zeros(12), 2, 1, "top2", True, 1.0)
    s = np.sort(1 / (1 + np.exp(-l)).reshape(20, 2, 6), axis=2)[:, :, -2:].sum(2)
    assert (o["expert"] // 6 == s.argmax(1)[:, None]).all() and np.allclose(o["weight"].sum(1), 1)


def test_oracle_block_norm_is_two_norms():
    rng = np.random.default_rng(4)
    x, r, w1, w2 = rng.standard_normal((5, 2, 16)), rng.standard_normal((5, 16)), rng.standard_normal(16), rng.standard_normal(16)
    o = oracle.block.block_norm(x, r, w1, w2, None, None, 0.5, 2.0, 1e-5, 1.0, True)
    inner = oracle.layer.add_rms_norm(x, None, w1 + 1, 1e-5)["y"]
    outer = oracle.layer.add_rms_norm((0.5 * inner)[:, None], 2 * r, w2 + 1, 1e-5)
    assert np.allclose(o["total"], outer["total"]) and np.allclose(o["y"], outer["y"]) and np.allclose(o["scale"], outer["scale"])
