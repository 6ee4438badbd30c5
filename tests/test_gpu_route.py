"""The routing to experts against its definition, token by token: scores, biases, groups, ties, closed experts,
scores that fp32 cannot tell apart, the plan, strides, streams and graphs."""
import math

import numpy as np
import pytest
import torch

import dequant_matmul_amd as fqm
import oracle
from gpu_common import DEV, canaries_intact, guarded, to_f64

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f32": torch.float32}


def check(logits, k, got, score="softmax", bias=None, groups=1, top_groups=None, group_score="max", renormalise=True, scale=1.0):
    o = oracle.block.route(to_f64(logits), k, score, None if bias is None else to_f64(bias), groups, top_groups or groups,
                           group_score, renormalise, float(np.float32(scale)))
    for name in ("expert", "offsets", "src", "dst"):
        assert np.array_equal(getattr(got, name).cpu().numpy(), o[name]), name
    assert (np.abs(to_f64(got.weight) - o["weight"]) <= o["bound"]).all()
    rs = to_f64(got.weight).ravel()[o["dst"]]
    assert np.array_equal(to_f64(got.row_scale), rs)
    return o


def run(logits, k, **kw):
    return check(logits, k, fqm.route(logits, k, **kw), **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens,E,k,x,bias,groups,top,gs,renorm,scale,pad", [
    (1, 1, 1, "f32", False, 1, 1, "max", True, 1.0, 0),
    (1, 64, 8, "bf16", False, 1, 1, "max", True, 1.0, 0),
    (3, 2, 2, "f32", True, 1, 1, "max", False, 2.5, 3),
    (5, 7, 3, "f32", False, 1, 1, "max", False, 1.0, 1),
    (48, 256, 8, "f32", True, 8, 4, "top2", True, 2.5, 0),
    (33, 60, 6, "f32", True, 1, 1, "max", False, 1.0, 5),
    (17, 65, 32, "f32", False, 5, 3, "max", True, 1.0, 0),
    (40, 128, 4, "bf16", False, 4, 2, "top2", True, 1.0, 8),
    (29, 128, 12, "bf16", True, 64, 30, "top2", False, 0.5, 0),
    (21, 129, 9, "f32", True, 3, 2, "max", True, -1.5, 0),
    (11, 513, 20, "f32", True, 1, 1, "max", True, 1.0, 2),
    (9, 1024, 32, "f32", True, 16, 5, "top2", True, 1.0, 0),
    (300, 96, 6, "f32", False, 8, 3, "top2", True, 1.0, 0),
    (1300, 40, 2, "f32", True, 4, 1, "top2", False, 1.0, 0),
    (64, 63, 1, "f32", False, 7, 7, "max", True, 1.0, 0),
])
def test_against_definition(tokens, E, k, x, bias, groups, top, gs, renorm, scale, pad, score):
    print(f"route {tokens}x{E} k {k} {score} {x} bias {bias} groups {groups}/{top} {gs} renorm {renorm}", flush=True)
    rng = np.random.default_rng([tokens, E, k])
    wide = torch.from_numpy(2 * rng.standard_normal((tokens, E + pad))).to(DEV, T[x])
    b = torch.from_numpy(0.1 * rng.standard_normal(E)).to(DEV, torch.float32) if bias else None
    run(wide[:, :E], k, score=score, bias=b, groups=groups, top_groups=top, group_score=gs, renormalise=renorm, scale=scale)


@pytest.mark.parametrize("tokens", [2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513, 1023, 1025, 2049, 5000])
def test_plans_around_the_tiles(tokens):
    print(f"route plan {tokens}", flush=True)
    rng = np.random.default_rng(tokens)
    liked = np.where(np.arange(24) % 5 == 0, 3.0, 0.0)
    logits = torch.from_numpy(rng.standard_normal((tokens, 24)) + liked).to(DEV, torch.float32)
    run(logits, 4)


def test_a_long_prompt():
    """65536 tokens, the plan against a stable sort; the choice against torch on a sample."""
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    logits = torch.randn(65536, 128, generator=g, device=DEV)
    r = fqm.route(logits, 8)
    order = torch.argsort(r.expert.flatten(), stable=True)
    assert torch.equal(r.dst, order.int()) and torch.equal(r.src, (order // 8).int())
    assert torch.equal(r.offsets.diff(), torch.bincount(r.expert.flatten(), minlength=128).int()) and r.offsets[0] == 0
    assert torch.equal(r.row_scale, r.weight.flatten()[order])
    pick = torch.arange(0, 65536, 1000, device=DEV)
    o = oracle.block.route(to_f64(logits[pick]), 8, "softmax", None, 1, 1, "max", True, 1.0)
    assert np.array_equal(r.expert[pick].cpu().numpy(), o["expert"])


@pytest.mark.parametrize("E", [24, 100, 256, 500, 1000])
@pytest.mark.parametrize("tokens", [1500, 4100, 9000])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_many_tokens_by_the_number_of_experts(tokens, E, score):
    """Every 16th token's scores are within 1e-6 of each other, biased: what fp32 leaves open is taken up after the
    others.  The plan against a stable sort, the choice against the definition and against a call of few tokens."""
    print(f"route {tokens}x{E} {score}", flush=True)
    rng = np.random.default_rng([tokens, E])
    l = rng.standard_normal(E).astype(np.float32)
    s = 1 / (1 + np.exp(-l.astype(np.float64))) if score == "sigmoid" else np.exp(l.astype(np.float64)) / np.exp(l.astype(np.float64)).sum()
    bias = torch.from_numpy((0.9 - s).astype(np.float32)).to(DEV)
    rows = rng.standard_normal((tokens, E)).astype(np.float32)
    rows[::16] = l
    rows[32] = -np.inf
    logits = torch.from_numpy(rows).to(DEV)
    kw = dict(score=score, bias=bias, groups=4, top_groups=3, group_score="top2")
    r = fqm.route(logits, 6, **kw)
    key = torch.where(r.expert < 0, E, r.expert).flatten()
    order = torch.argsort(key, stable=True)
    assert torch.equal(r.dst, order.int())
    assert torch.equal(r.src, torch.where(key[order] < E, order // 6, -1).int())
    counts = torch.bincount(key, minlength=E + 1)
    counts[E - 1] += counts[E]
    assert torch.equal(r.offsets.diff(), counts[:E].int()) and r.offsets[0] == 0
    assert torch.equal(r.row_scale, r.weight.flatten()[order])
    pick = torch.tensor([0, 1, 16, 31, 32, tokens // 16 * 16 - 16, tokens - 2, tokens - 1], device=DEV)
    few = run(logits[pick].contiguous(), 6, **kw)
    got = fqm.route(logits[pick].contiguous(), 6, **kw)
    assert np.array_equal(r.expert[pick].cpu().numpy(), few["expert"])
    assert torch.equal(r.expert[pick], got.expert) and torch.equal(r.weight[pick], got.weight)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("gs", ["max", "top2"])
def test_ties_go_to_the_lowest_index(score, gs):
    rng = np.random.default_rng(7)
    logits = torch.from_numpy(rng.integers(-2, 3, (60, 96)).astype(np.float32)).to(DEV)
    logits[0] = 1.5
    logits[1] = 0
    run(logits, 10, score=score, group_score=gs)
    run(logits, 10, score=score, groups=8, top_groups=3, group_score=gs)
    run(logits, 10, score=score, groups=8, top_groups=3, group_score=gs, bias=torch.zeros(96, device=DEV))
    run(logits.to(torch.bfloat16), 5, score=score, bias=torch.full((96,), 0.25, device=DEV))


def test_scores_that_fp32_cannot_tell_apart():
    """Biases that bring all experts to scores within 1e-7 of each other: only fp64 knows their order."""
    rng = np.random.default_rng(8)
    E = 64
    l = rng.standard_normal(E).astype(np.float32)
    s = 1 / (1 + np.exp(-l.astype(np.float64)))
    bias = (0.9 - s).astype(np.float32)
    c = s + bias
    assert len(np.unique(c)) == E and c.max() - c.min() < 2e-7
    logits = torch.from_numpy(np.tile(l, (5, 1))).to(DEV)
    logits[1, 10:20] += 1e-6
    logits[2] = torch.from_numpy(rng.standard_normal(E).astype(np.float32))
    b = torch.from_numpy(bias).to(DEV)
    run(logits, 12, score="sigmoid", bias=b)
    run(logits, 12, score="sigmoid", bias=b, groups=8, top_groups=2, group_score="top2")
    run(logits, 4, score="sigmoid", bias=b, groups=16, top_groups=3, group_score="max")
    p = np.exp(l.astype(np.float64) - l.max())
    p /= p.sum()
    b = torch.from_numpy((0.5 - p).astype(np.float32)).to(DEV)
    run(logits, 12, score="softmax", bias=b, renormalise=False)
    run(logits, 3, score="softmax", bias=b, groups=8, top_groups=2, group_score="top2")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_closed_experts_empty_rows_and_what_is_not_finite(score, renorm):
    rng = np.random.default_rng(9)
    l = rng.standard_normal((40, 24)).astype(np.float32)
    l[rng.random(l.shape) < 0.5] = -np.inf
    l[3] = -np.inf              # a padded row
    l[4] = np.nan
    l[5, 1:] = -np.inf          # one open expert
    l[6, ::2] = np.nan
    l[7, 2] = l[7, 9] = np.inf  # counts as the largest number
    l[8] = -np.inf
    l[8, 20] = np.inf
    l[9, :12] = -np.inf         # whole groups closed
    l[10] = np.finfo(np.float32).min
    l[11] = -200.0 - np.arange(24)
    l[12] = 300.0 + np.arange(24)
    l[13, 0] = -0.0
    l[30:] = -np.inf
    logits = torch.from_numpy(l).to(DEV)
    kw = dict(score=score, renormalise=renorm)
    o = run(logits, 6, **kw)
    assert (o["expert"][3] == -1).all() and (o["expert"][5, 1:] == -1).all() and (o["expert"][30:] == -1).all()
    run(logits, 6, groups=4, top_groups=2, group_score="top2", **kw)
    run(logits, 6, groups=24, top_groups=6, group_score="top2", **kw)
    run(logits, 6, groups=4, top_groups=2, group_score="max", **kw)
    bias = torch.from_numpy(0.1 * rng.standard_normal(24)).to(DEV, torch.float32)
    bias[2], bias[5], bias[6] = -math.inf, math.nan, math.inf
    run(logits, 6, bias=bias, **kw)
    run(logits, 6, bias=bias, groups=4, top_groups=2, group_score="top2", **kw)


def test_the_plan_runs_the_products():
    """Rows grouped by the plan, through gemm_grouped and back to their slots: each slot has its expert's product,
    slots without an expert zeros."""
    E, K, N, k, tokens = 6, 256, 40, 3, 50
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    codes = torch.randint(0, 64, (E * N, K), generator=g, device=DEV, dtype=torch.uint8)
    lut = torch.randn(E * N, 64, generator=g, device=DEV).to(torch.bfloat16)
    w = fqm.Lut6Weights.from_codes(codes, lut.view(torch.int16), device=DEV)
    x = torch.randn(tokens, K, generator=g, device=DEV).to(torch.bfloat16)
    logits = torch.randn(tokens, E, generator=g, device=DEV)
    logits[::7] = -math.inf
    logits[3, 1:] = -math.inf
    r = fqm.route(logits, k)
    y = fqm.gemm_grouped(w, x, r.offsets, src=r.src, dst=r.dst, row_scale=r.row_scale, out_dtype=torch.float32)
    W = fqm.dequant(w).double().view(E, N, K)
    want = torch.zeros(tokens, k, N, dtype=torch.float64, device=DEV)
    for t in range(tokens):
        for j in range(k):
            e = int(r.expert[t, j])
            if e >= 0:
                want[t, j] = r.weight[t, j].double() * (W[e] @ x[t].double())
    assert ((y.double().view_as(want) - want).norm() / want.norm()).item() < 1e-5
    assert (y.view(tokens, k, N)[::7] == 0).all() and (y.view(tokens, k, N)[3, 1:] == 0).all()


def test_without_a_plan_into_given_tensors_and_empty():
    logits = torch.randn(70, 30, device=DEV)
    full = fqm.route(logits, 4)
    r = fqm.route(logits, 4, plan=False)
    assert r.offsets is None and r.src is None and torch.equal(r.expert, full.expert) and torch.equal(r.weight, full.weight)
    bufs = [guarded(s, dt, fill=-77) for s, dt in (((70, 4), torch.int32), ((70, 4), torch.float32), ((31,), torch.int32),
                                                   ((280,), torch.int32), ((280,), torch.int32), ((280,), torch.float32))]
    out = fqm.Routing(*(v for _, v in bufs))
    assert fqm.route(logits, 4, out=out) is out
    torch.cuda.synchronize()
    assert all(canaries_intact(b, fill=-77) for b, _ in bufs)
    assert all(torch.equal(a, b) for a, b in zip(out, full))
    r = fqm.route(torch.zeros(0, 30, device=DEV), 4)
    assert r.expert.shape == (0, 4) and (r.offsets == 0).all() and r.offsets.shape == (31,) and r.src.shape == (0,)


@pytest.mark.parametrize("tokens", [1, 100, 3000])
def test_streams_workspaces_and_graph_replays(tokens):
    print(f"route graph {tokens}", flush=True)
    logits = torch.randn(tokens, 64, device=DEV)
    bias = 0.1 * torch.randn(64, device=DEV)
    kw = dict(score="sigmoid", bias=bias, groups=4, top_groups=2, group_score="top2")
    want = fqm.route(logits, 6, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side = fqm.route(logits, 6, stream=side, **kw)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(on_side, want))
    out = fqm.Routing(*(torch.empty_like(t) for t in want))
    ws = torch.full((max(fqm.route_workspace_size(tokens, 64, 6), 1),), 255, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fqm.route(logits, 6, out=out, workspace=ws, **kw)
    for _ in range(3):
        logits.copy_(torch.roll(logits, 1, 1))
        want = fqm.route(logits, 6, **kw)
        ws.fill_(255)
        for t in out:
            t.fill_(-5)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_refusals_of_the_binding():
    l = torch.zeros(4, 24, device=DEV)
    for kw, match in ((dict(k=0), "k = 0"), (dict(k=25), "k = 25"), (dict(k=33), "k = 33"), (dict(k=2, groups=5), "groups"),
                      (dict(k=7, groups=4, top_groups=1), "k = 7"), (dict(k=2, groups=4, top_groups=5), "groups"),
                      (dict(k=2, score="max"), "score must be"), (dict(k=2, group_score="sum"), "group_score must be"),
                      (dict(k=2, bias=torch.zeros(23, device=DEV)), "bias"), (dict(k=2, bias=torch.zeros(24, dtype=torch.bfloat16, device=DEV)), "bias"),
                      (dict(k=2, workspace=torch.zeros(8)), "workspace")):
        with pytest.raises(ValueError, match=match):
            fqm.route(l, **kw)
    with pytest.raises(ValueError, match="dense rows"):
        fqm.route(torch.zeros(24, 4, device=DEV).t(), 2)
    with pytest.raises(ValueError, match="overlapping"):
        fqm.route(torch.zeros(1, 24, device=DEV).expand(4, 24), 2)
    r = fqm.route(l, 2)
    for name, t in (("expert", r.expert.long()), ("src", r.src[:-1]), ("row_scale", r.row_scale.double()), ("weight", r.weight.t())):
        with pytest.raises(ValueError, match=f"out.{name}"):
            fqm.route(l, 2, out=r._replace(**{name: t}))
    with pytest.raises(ValueError, match="out.dst"):
        fqm.route(l, 2, out=r._replace(dst=None))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("tokens,E", [(1, 4), (1, 24), (5, 24), (70, 100), (60, 256), (40, 600), (7000, 24)])
def test_zeros_of_both_signs_are_equal(tokens, E, x, score):
    """-0 and +0 tie as any two equal logits do: the lowest index first, whichever of them has the sign."""
    print(f"route zeros {tokens}x{E} {x} {score}", flush=True)
    rng = np.random.default_rng([tokens, E])
    l = rng.choice([-1.0, -0.0, 0.0], (tokens, E))
    l[0] = np.where(np.arange(E) % 2 == 0, -0.0, 0.0)
    logits = torch.from_numpy(l).to(DEV, T[x])
    assert torch.signbit(logits[0, 0]) and not torch.signbit(logits[0, 1])
    for kw in (dict(), dict(renormalise=False), dict(bias=torch.zeros(E, device=DEV)), dict(bias=-torch.zeros(E, device=DEV)),
               dict(groups=4, top_groups=2, group_score="max"), dict(groups=2, group_score="top2")):
        run(logits, min(3, E // 2), score=score, **kw)
