"""The product with its epilogue, the routing and the norms together, as a layer of experts uses them."""
import os
import subprocess
import sys

import pytest
import torch

import dequant_matmul_amd as fqm
from conftest import ROOT
from gpu_common import DEV

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(ROOT, "examples"))


def norm(h, w):
    return h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6) * (1 + w.double())


def layer_and_inputs(tokens):
    from experts_layer import ExpertsLayer
    layer = ExpertsLayer(hidden=512, inner=256, experts=8, k=3, groups=4, top_groups=2, seed=tokens)
    g = torch.Generator(device=DEV)
    g.manual_seed(tokens)
    return layer, *(torch.randn(tokens, 512, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))


@pytest.mark.parametrize("tokens", [1, 5, 40, 300])
def test_layer_matches_fp64(tokens):
    layer, attention, residual = layer_and_inputs(tokens)
    x, h, r = layer(attention, residual)
    torch.cuda.synchronize()

    # the same in fp64, with the experts that the layer took (a near tie may go either way): every one of ten or so
    # roundings to bf16 in a row leaves at most 2^-9 of a value's root mean square, 2 % is all of them in step
    h64 = residual.double() + norm(attention.double(), layer.norms[0])
    x64 = norm(h64, layer.norms[1])
    w = fqm.dequant(layer.shared_in).double()
    h64 = h64 + torch.nn.functional.silu(x64 @ w[:256].t()) * (x64 @ w[256:].t()) @ fqm.dequant(layer.shared_out).double().t()
    up, down = fqm.dequant(layer.up).double().view(8, 256, 512), fqm.dequant(layer.down).double().view(8, 512, 256)
    scores = torch.sigmoid(x64 @ layer.router.double())
    taken = torch.gather(scores, 1, r.expert.long())
    weight = 2.5 * taken / taken.sum(1, keepdim=True)
    total = torch.zeros_like(h64)
    for t in range(tokens):
        for j in range(3):
            e = int(r.expert[t, j])
            total[t] += weight[t, j] * (down[e] @ torch.nn.functional.silu(up[e] @ x64[t]))
    h64 = h64 + norm(total, layer.norms[2]) * layer.gate.double()
    x64 = norm(h64, layer.norms[3])
    assert (r.weight.double() - weight).abs().max().item() < 0.02 * 2.5
    assert torch.isfinite(x).all()
    assert ((h.double() - h64).norm() / h64.norm()).item() < 0.02
    assert ((x.double() - x64).norm() / x64.norm()).item() < 0.02


@pytest.mark.parametrize("tokens", [1, 40, 300])
def test_layer_in_a_graph(tokens):
    """Replays after other work and other inputs give the eager call's bits."""
    layer, attention, residual = layer_and_inputs(tokens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(attention, residual)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x, h, r = layer(attention, residual)
    for i in range(4):
        attention.copy_(torch.randn(tokens, 512, device=DEV).to(torch.bfloat16))
        want = layer(attention, residual)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(x, want[0]) and torch.equal(h, want[1])
        for name in ("expert", "weight", "offsets", "src", "dst", "row_scale"):
            assert torch.equal(getattr(r, name), getattr(want[2], name)), (i, name)


def test_two_graphs_with_one_workspace():
    """Graphs replayed one after the other may share a workspace: no call reads what another one left there."""
    layer, attention, residual = layer_and_inputs(300)
    logits = torch.randn(300, 8, device=DEV)
    need = max(fqm.linear_workspace_size(layer.shared_in, 300, True), fqm.route_workspace_size(300, 8, 3), 16)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    calls = (lambda: fqm.linear(layer.shared_in, attention, act="silu", gated=True, workspace=ws),
             lambda: fqm.route(logits, 3, workspace=ws).row_scale)
    want = [c().clone() for c in calls]
    graphs, got = [], []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(c())
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 1, 0)):
        ws.fill_(0xff)
        for o in got:
            o.zero_()
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_example_runs():
    out = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "experts_layer.py"), "5"], capture_output=True, text=True,
                         timeout=100)
    assert out.returncode == 0 and "us a layer" in out.stdout, out.stderr
