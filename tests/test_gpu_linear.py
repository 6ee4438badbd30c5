"""The product with its epilogue against its fp64 definition: formats, row counts, widths, activations, the gated
form, bias, residual, strides, in place, streams and graphs."""
import numpy as np
import pytest
import torch

import dequant_matmul_amd as fqm
import oracle
import synth
from gpu_common import DEV, bf16_dev, canaries_intact, guarded, to_f64

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f32": torch.float32}


def weights(bits, rows, cols, seed=0):
    """Weights and their decoded values [rows][cols]."""
    make, cls, dec = ((synth.lut6_input, fqm.Lut6Weights, oracle.lut6.decode) if bits == 6 else
                      (synth.lut4_input, fqm.Lut4Weights, oracle.lut4.decode))
    inp = make(rows, cols, 57 + seed, level_jitter=0.3)
    return cls.from_codes(inp.codes, inp.lut, device=DEV), dec(inp.codes, inp.lut)


def rows_at(v, dtype, pad, start=0):
    """The rows of v inside rows that are `pad + start` values wider, `start` values in."""
    wide = torch.full((v.shape[0], v.shape[1] + pad + start), 9.0, dtype=T[dtype], device=DEV)
    view = wide[:, start:start + v.shape[1]]
    view.copy_(torch.from_numpy(np.ascontiguousarray(v)))
    return view


def run_case(bits, M, K, n, gated, act, bias, res, out, padx=0, pad=0, seed=0):
    print(f"linear {bits} bits M {M} {K}->{n} gated {gated} {act} bias {bias} residual {res} {out} pad {padx} {pad}", flush=True)
    rng = np.random.default_rng([M, K, n, seed])
    rows = n * (1 + gated)
    w, W = weights(bits, rows, K)
    size = max(np.sqrt((W * W).sum(1)).mean(), 1e-30)  # so that v is of the order of one
    x = rows_at(rng.standard_normal((M, K)) / size, "bf16", padx)
    b = torch.from_numpy(rng.standard_normal(rows)).to(DEV, T[bias]) if bias else None
    r = rows_at(rng.standard_normal((M, n)), res, pad, pad and 1) if res else None
    buf, Y = guarded((M, n), T[out])
    y = fqm.linear(w, x, bias=b, act=act, gated=gated, residual=r, y=Y)
    torch.cuda.synchronize()
    assert y is Y and canaries_intact(buf)
    yo, lim = oracle.block.linear(W, to_f64(x), None if b is None else to_f64(b), act, gated, None if r is None else to_f64(r))
    off = np.abs(to_f64(Y) - yo) - oracle.layer.rounded(lim, yo, out)
    assert (off <= 0).all(), (off.max(), np.unravel_index(off.argmax(), off.shape))


@pytest.mark.parametrize("bits", [6, 4])
@pytest.mark.parametrize("M,K,n,gated,act,bias,res,out,padx,pad", [
    (1, 64, 1, False, None, None, None, "f32", 0, 0),
    (1, 1024, 77, False, None, None, "bf16", "bf16", 0, 0),
    (1, 1024, 65, True, "silu", "f32", None, "f32", 0, 0),
    (1, 5120, 200, True, "silu", None, None, "bf16", 0, 0),
    (1, 17408, 130, False, None, "bf16", "f32", "f32", 0, 0),
    (1, 9216, 41, True, "gelu", "bf16", "bf16", "bf16", 0, 3),
    (1, 32768, 35, True, "relu", None, None, "f32", 0, 0),
    (1, 704, 50, True, "gelu_tanh", "f32", "f32", "f32", 8, 5),
    (2, 2048, 100, True, "silu", None, "bf16", "bf16", 0, 0),
    (2, 19456, 21, False, "gelu", "f32", None, "f32", 8, 0),
    (2, 1088, 33, False, "tanh", "f32", "f32", "f32", 64, 1),
    (3, 4096, 99, False, "silu", None, "f32", "bf16", 8, 7),
    (3, 12288, 17, True, "sigmoid", "bf16", None, "f32", 0, 0),
    (3, 13312, 40, True, None, None, None, "f32", 0, 0),
    (4, 512, 130, True, "silu", "f32", "bf16", "f32", 0, 0),
    (5, 1536, 70, False, "gelu", "bf16", None, "bf16", 8, 0),
    (7, 576, 129, False, "relu", "f32", "f32", "f32", 16, 2),
    (8, 5120, 48, True, "gelu", None, None, "bf16", 0, 0),
    (13, 2560, 300, True, "silu", "bf16", "f32", "f32", 8, 3),
    (16, 4096, 1000, False, None, "f32", "bf16", "bf16", 0, 0),
    (16, 192, 515, True, "gelu_tanh", None, "f32", "f32", 0, 0),
    (17, 1024, 64, False, "silu", "f32", "f32", "f32", 0, 0),
    (33, 320, 257, True, "gelu", "bf16", "bf16", "bf16", 24, 9),
    (64, 2048, 300, True, "silu", None, None, "f32", 0, 0),
    (77, 4160, 100, False, "gelu", "f32", "f32", "f32", 8, 3),
    (129, 640, 1000, True, "silu", "f32", "bf16", "bf16", 0, 0),
    (257, 128, 70, False, "tanh", "bf16", "f32", "f32", 0, 1),
    (300, 1088, 130, True, "relu", None, "f32", "f32", 8, 0),
    (1031, 512, 260, True, "silu", "bf16", None, "bf16", 0, 0),
    (2050, 320, 515, False, None, "f32", "bf16", "f32", 0, 5),
])
def test_against_definition(bits, M, K, n, gated, act, bias, res, out, padx, pad):
    run_case(bits, M, K, n, gated, act, bias, res, out, padx, pad)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M", [1, 2, 3, 4, 8, 9, 15, 16, 17, 31, 32, 33, 47, 63, 64, 65, 95, 127, 128, 129, 255, 256, 257])
def test_row_counts_around_the_tiles(M, gated):
    run_case(6 if M % 2 else 4, M, 1024, 70, gated, "silu", "f32", "f32", "f32", seed=M)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("n", [1, 2, 8, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257])
@pytest.mark.parametrize("M,K", [(1, 1024), (6, 512), (40, 256), (260, 192)])
def test_output_counts_around_the_tiles(M, K, n, gated):
    run_case(6 if n % 2 else 4, M, K, n, gated, "silu", "bf16", "bf16", "f32", pad=1, seed=n)


@pytest.mark.parametrize("M,K,n", [(1, 5120, 17408), (16, 5120, 9000), (3, 1024, 17000), (3, 5120, 14000), (5, 1024, 33000),
                                   (64, 512, 17408)])
def test_large_outputs(M, K, n):
    """Enough rows of W that K is not split, a sample of the outputs checked (the oracle takes their rows of W alone)."""
    rng = np.random.default_rng([M, K, n])
    for bits, gated in ((6, False), (4, True)):
        n_out = n // 2 if gated else n
        print(f"linear {bits} bits M {M} {K}->{n_out} gated {gated}", flush=True)
        w, W = weights(bits, n_out * (1 + gated), K)
        x = torch.from_numpy(rng.standard_normal((M, K)) / np.sqrt((W[:64] ** 2).sum(1)).mean()).to(DEV, torch.bfloat16)
        y = to_f64(fqm.linear(w, x, act="silu", gated=gated, out_dtype=torch.float32))
        pick = np.unique(np.r_[0:40, rng.integers(0, n_out, 200), n_out - 40:n_out])
        rows = np.r_[pick, pick + n_out] if gated else pick
        yo, lim = oracle.block.linear(W[rows], to_f64(x), None, "silu", gated, None)
        assert (np.abs(y[:, pick] - yo) <= oracle.layer.rounded(lim, yo, "f32")).all()


@pytest.mark.parametrize("M", [1, 3, 9, 40, 300])
def test_the_plain_product_is_gemms_and_gemvs(M):
    """No epilogue: the same sums as the product calls give, up to the order of the additions."""
    w, W = weights(6, 200, 1024)
    x = bf16_dev(synth.activations(M, 1024, 5))
    y = to_f64(fqm.linear(w, x, out_dtype=torch.float32))
    yo, lim = oracle.block.linear(W, to_f64(x), None, None, False, None)
    assert (np.abs(y - yo) <= lim).all()
    other = fqm.gemv(w, x, out_dtype=torch.float32) if M <= 16 else fqm.gemm(w, x)
    assert (np.abs(to_f64(other) - yo) <= oracle.layer.rounded(lim, yo, "f32" if M <= 16 else "bf16")).all()


@pytest.mark.parametrize("M", [1, 2, 8, 50, 300])
@pytest.mark.parametrize("gated", [False, True])
def test_in_place_of_the_residual_and_strided(M, gated):
    w, _ = weights(6, 140, 1024)
    n = 70 if gated else 140
    x = bf16_dev(synth.activations(M, 1024, 5))
    for dt in (torch.bfloat16, torch.float32):
        wide = torch.randn(M, n + 11, device=DEV).to(dt)
        r = wide[:, 5:5 + n]
        before = wide.clone()
        want = fqm.linear(w, x, act="gelu", gated=gated, residual=r, out_dtype=dt)
        got = fqm.linear(w, x, act="gelu", gated=gated, residual=r, y=r)
        assert got.data_ptr() == r.data_ptr() and torch.equal(got, want)
        assert torch.equal(wide[:, :5], before[:, :5]) and torch.equal(wide[:, 5 + n:], before[:, 5 + n:])


@pytest.mark.parametrize("M", [1, 2, 3, 6, 40, 300])
def test_a_row_does_not_depend_on_the_others(M):
    w, _ = weights(4, 140, 1024)
    x = bf16_dev(synth.activations(M, 1024, 5))
    want = fqm.linear(w, x, act="silu", gated=True, out_dtype=torch.float32)
    bad = x.clone()
    bad[M // 2] = float("nan")
    bad[M // 2, 3] = float("inf")
    got = fqm.linear(w, bad, act="silu", gated=True, out_dtype=torch.float32)
    keep = [m for m in range(M) if m != M // 2]
    assert torch.equal(got[keep], want[keep]) and torch.isnan(got[M // 2]).all()


def test_what_is_not_finite_goes_through():
    w, _ = weights(6, 64, 1024)
    x = torch.zeros(3, 1024, dtype=torch.bfloat16, device=DEV)
    bias = torch.zeros(64, device=DEV)
    bias[0], bias[1], bias[2] = float("nan"), float("inf"), -100.0
    y = fqm.linear(w, x, bias=bias, act="silu", out_dtype=torch.float32)
    assert torch.isnan(y[:, 0]).all() and (y[:, 1] == float("inf")).all() and (y[:, 2].abs() < 1e-40).all() and (y[:, 3:] == 0).all()
    y = fqm.linear(w, x, bias=bias, act="relu", out_dtype=torch.float32)
    assert torch.isnan(y[:, 0]).all() and (y[:, 2] == 0).all()


@pytest.mark.parametrize("gated", [False, True])
def test_empty(gated):
    n = 10
    codes = np.zeros((20 if gated else 10, 0), dtype=np.uint8)
    w = fqm.Lut6Weights(torch.zeros(codes.shape[0], 16, dtype=torch.uint8, device=DEV),
                        torch.zeros(codes.shape[0], 64, dtype=torch.bfloat16, device=DEV), codes.shape[0], 0)
    bias = torch.arange(codes.shape[0], device=DEV).float()
    res = torch.ones(4, n, device=DEV)
    y = fqm.linear(w, torch.zeros(4, 0, dtype=torch.bfloat16, device=DEV), bias=bias, act="relu", gated=gated, residual=res,
                   out_dtype=torch.float32)
    want = 1 + (bias[:n] * bias[n:] if gated else bias)
    assert torch.equal(y, want.expand(4, n))
    w, _ = weights(6, 20, 128)
    assert fqm.linear(w, torch.zeros(0, 128, dtype=torch.bfloat16, device=DEV), gated=gated).shape == (0, 10 if gated else 20)


@pytest.mark.parametrize("M,K,n", [(1, 5120, 300), (3, 1024, 200), (8, 2048, 200), (40, 2048, 300), (300, 1024, 200)])
def test_streams_workspaces_and_graph_replays(M, K, n):
    print(f"linear graph M {M} {K}->{n}", flush=True)
    w, _ = weights(6, 2 * n, K)
    x = bf16_dev(synth.activations(M, K, 5))
    res = torch.randn(M, n, device=DEV)
    call = lambda **kw: fqm.linear(w, x, act="silu", gated=True, residual=res, **kw)  # noqa: E731
    want = call(out_dtype=torch.float32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side = call(out_dtype=torch.float32, stream=side)
    side.synchronize()
    assert torch.equal(on_side, want)
    need = fqm.linear_workspace_size(w, M, gated=True, out_dtype=torch.float32)
    ws = torch.full((max(need, 1),), 255, dtype=torch.uint8, device=DEV)  # NaN in fp32
    y = torch.empty(M, n, device=DEV)
    assert torch.equal(call(y=y, workspace=ws), want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(y=y, workspace=ws)
    for _ in range(3):
        x.copy_(torch.roll(x, 1, 1))
        want = call(out_dtype=torch.float32)
        y.zero_()
        ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_refusals_of_the_binding():
    w, _ = weights(6, 21, 128)
    x = torch.zeros(3, 128, dtype=torch.bfloat16, device=DEV)
    for kw, match in ((dict(gated=True), "two stacked"), (dict(act="swish"), "act must be"), (dict(out_dtype=torch.float16), "out_dtype"),
                      (dict(bias=torch.zeros(20, device=DEV)), "bias"), (dict(residual=torch.zeros(3, 20, device=DEV)), "residual"),
                      (dict(residual=torch.zeros(1, 21, device=DEV).expand(3, 21)), "overlapping"),
                      (dict(residual=torch.zeros(21, 3, device=DEV).t()), "dense rows"),
                      (dict(y=torch.zeros(3, 21, dtype=torch.float64, device=DEV)), "out_dtype"), (dict(y=torch.zeros(3, 22, device=DEV)), "y has"),
                      (dict(workspace=torch.zeros(8)), "workspace"), (dict(bias=torch.zeros(21)), "GPU tensors")):
        with pytest.raises(ValueError, match=match):
            fqm.linear(w, x, **kw)
    with pytest.raises(ValueError, match="multiples of 16 bytes"):
        fqm.linear(w, torch.zeros(3, 132, dtype=torch.bfloat16, device=DEV)[:, :128])
    with pytest.raises(ValueError, match="multiples of 16 bytes"):
        fqm.linear(w, torch.zeros(3, 136, dtype=torch.bfloat16, device=DEV)[:, 1:129])
    with pytest.raises(ValueError, match="expected"):
        fqm.linear(w, torch.zeros(3, 64, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(fqm.FqmError, match="workspace"):
        big, _ = weights(6, 200, 8192)
        fqm.linear(big, torch.zeros(40, 8192, dtype=torch.bfloat16, device=DEV), workspace=torch.zeros(8, dtype=torch.uint8, device=DEV))


# Nine to 32 rows, and fewer where no other kernel takes the width: tiles that up to 16 workgroups share through the
# workspace, tiles of a workgroup's own between them (K 192 and 320), K of an odd number of steps.
SHARED = [(12, 5120, 300), (16, 1024, 130), (24, 1088, 300), (32, 5120, 1000), (5, 4160, 200), (1, 704, 515), (17, 8192, 64),
          (16, 192, 515), (31, 320, 2000)]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,K,n", SHARED)
def test_shared_tiles_on_streams_with_any_workspace_and_in_graphs(M, K, n, gated):
    """No call reads what its workspace held before, nor does a replay."""
    print(f"linear shared tiles M {M} {K}->{n} gated {gated}", flush=True)
    w, _ = weights(6 if n % 8 else 4, n * (1 + gated), K)
    x = bf16_dev(synth.activations(M, K, 5))
    res = torch.randn(M, n, device=DEV)
    call = lambda **kw: fqm.linear(w, x, act="silu", gated=gated, residual=res, **kw)  # noqa: E731
    want = call(out_dtype=torch.float32)
    need = fqm.linear_workspace_size(w, M, gated=gated, out_dtype=torch.float32)
    assert need > 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side = call(out_dtype=torch.float32, stream=side)
    side.synchronize()
    assert torch.equal(on_side, want)
    buf, y = guarded((M, n), torch.float32)
    for fill in (255, 127, 0):  # NaN, about 3e38, 0
        guard = torch.full((need + 4096,), fill, dtype=torch.uint8, device=DEV)
        y.zero_()
        assert torch.equal(call(y=y, workspace=guard[:need]), want)
        assert canaries_intact(buf) and (guard[need:] == fill).all()
    ws = guard[:need]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(y=y, workspace=ws)
    for _ in range(3):
        x.copy_(torch.roll(x, 1, 1))
        want = call(out_dtype=torch.float32)
        y.zero_()
        ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,K,n", SHARED)
def test_shared_tiles_in_place_of_the_residual(M, K, n, gated):
    w, _ = weights(6 if n % 8 else 4, n * (1 + gated), K)
    x = bf16_dev(synth.activations(M, K, 5))
    for dt in (torch.bfloat16, torch.float32):
        wide = torch.randn(M, n + 11, device=DEV).to(dt)
        r = wide[:, 5:5 + n]
        before = wide.clone()
        want = fqm.linear(w, x, act="gelu", gated=gated, residual=r, out_dtype=dt)
        got = fqm.linear(w, x, act="gelu", gated=gated, residual=r, y=r)
        assert got.data_ptr() == r.data_ptr() and torch.equal(got, want)
        assert torch.equal(wide[:, :5], before[:, :5]) and torch.equal(wide[:, 5 + n:], before[:, 5 + n:])


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,K,n", [c for c in SHARED if c[0] > 1])
def test_shared_tiles_keep_a_row_from_the_others(M, K, n, gated):
    """All rows but one NaN and infinite: that one keeps its bits, first, last and in between."""
    w, _ = weights(6 if n % 8 else 4, n * (1 + gated), K)
    x = bf16_dev(synth.activations(M, K, 5))
    want = fqm.linear(w, x, act="silu", gated=gated, out_dtype=torch.float32)
    for m in sorted({0, 1, M // 2, M - 1}):
        bad = torch.full_like(x, float("nan"))
        bad[:, ::3] = float("inf")
        bad[m] = x[m]
        got = fqm.linear(w, bad, act="silu", gated=gated, out_dtype=torch.float32)
        assert torch.equal(got[m], want[m])
        assert torch.isnan(got[[i for i in range(M) if i != m]]).all()


@pytest.mark.parametrize("M", [9, 16, 31])
def test_two_calls_at_once_with_workspaces_of_their_own(M):
    w, _ = weights(6, 2000, 5120)
    x = bf16_dev(synth.activations(M, 5120, 5))
    want = fqm.linear(w, x, act="silu", gated=True, out_dtype=torch.float32)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(8):
        for s in streams:
            outs.append(fqm.linear(w, x, act="silu", gated=True, out_dtype=torch.float32, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
