"""Products grouped by expert against their fp64 definition: both formats,
ragged and empty groups, gathers and scatters, 8-bit rows, odd widths."""
import numpy as np
import pytest
import torch

import dequant_matmul_amd as fqm
import oracle
import synth
from gpu_common import DEV, bf16_dev, canaries_intact, guarded, to_f64

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f32": torch.float32}


def experts(bits, E, N, K, seed=0):
    """Stacked weights of E matrices and their decoded values [E][N][K]."""
    make, cls, dec = ((synth.lut6_input, fqm.Lut6Weights, oracle.lut6.decode) if bits == 6 else
                      (synth.lut4_input, fqm.Lut4Weights, oracle.lut4.decode))
    inp = make(E * N, K, 31 + seed, level_jitter=0.3)
    return cls.from_codes(inp.codes, inp.lut, device=DEV), dec(inp.codes, inp.lut).reshape(E, N, K)


def sizes(kind, E, M, rng):
    """Offsets of M rows over E groups."""
    if kind == "even":
        cut = np.linspace(0, M, E + 1).astype(int)
    elif kind == "last":
        cut = np.r_[np.zeros(E, int), M]
    elif kind == "first":
        cut = np.r_[0, np.full(E, M)]
    else:  # ragged, some empty
        cut = np.r_[0, np.sort(rng.integers(0, M + 1, size=E - 1)), M]
    return cut


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def run_case(bits, E, N, K, M, kind, way, xt, out, seed=0):
    rng = np.random.default_rng([E, N, K, M, seed])
    w, W = experts(bits, E, N, K)
    off = sizes(kind, E, M, rng)
    src = dst = rs = xs = None
    x_rows = M
    if way == "gather":
        x_rows = max(1, M // 3)
        src = rng.integers(0, x_rows, size=M)
    if way == "scatter":
        dst = rng.permutation(M)
        rs = rng.uniform(0.1, 1.5, size=M).astype(np.float32)
    x = bf16_dev(synth.activations(x_rows, K, 3))
    xv = to_f64(x)
    if xt == "i8":
        xs = torch.from_numpy((np.abs(xv).max(axis=1, initial=1e-3) / 127).astype(np.float32)).to(DEV)
        x = torch.round(x.float() / xs[:, None]).to(torch.int8)
        xv = to_f64(x) * to_f64(xs)[:, None]
    buf, Y = guarded((M, N), T[out])
    fqm.gemm_grouped(w, x, i32(off), src=None if src is None else i32(src), x_scale=xs,
                     dst=None if dst is None else i32(dst),
                     row_scale=None if rs is None else torch.from_numpy(rs).to(DEV), Y=Y)
    torch.cuda.synchronize()
    assert canaries_intact(buf)
    Yo, lim = oracle.layer.grouped(W, off, xv, src, dst, rs, M, -12345.0)
    assert (np.abs(to_f64(Y) - Yo) <= oracle.layer.rounded(lim, Yo, out)).all()


@pytest.mark.parametrize("bits", [6, 4])
@pytest.mark.parametrize("E,N,K,M,kind,way,xt,out", [
    (1, 1, 64, 1, "even", "plain", "bf16", "f32"),
    (3, 77, 64, 2, "ragged", "gather", "bf16", "bf16"),
    (8, 256, 512, 8, "even", "gather", "bf16", "bf16"),
    (8, 130, 1088, 5, "ragged", "scatter", "bf16", "f32"),
    (4, 33, 704, 11, "ragged", "gather", "i8", "f32"),
    (5, 257, 1024, 40, "ragged", "scatter", "bf16", "bf16"),
    (6, 100, 2048, 90, "ragged", "gather", "i8", "bf16"),
    (2, 300, 320, 64, "last", "plain", "bf16", "f32"),
    (3, 512, 640, 200, "first", "gather", "bf16", "bf16"),
    (4, 129, 576, 333, "ragged", "scatter", "bf16", "f32"),
    (7, 260, 192, 600, "ragged", "gather", "i8", "bf16"),
    (2, 515, 128, 700, "ragged", "plain", "bf16", "bf16"),
    (40, 20, 256, 300, "ragged", "gather", "bf16", "f32"),
    (70, 16, 128, 69, "ragged", "scatter", "bf16", "bf16"),
    (3, 24, 5120, 48, "even", "plain", "bf16", "f32"),
])
def test_against_definition(bits, E, N, K, M, kind, way, xt, out):
    print(f"grouped {bits} bits E {E} {K}->{N} M {M} {kind} {way} {xt} {out}", flush=True)
    run_case(bits, E, N, K, M, kind, way, xt, out)


@pytest.mark.parametrize("m", [1, 2, 3, 4, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257])
def test_group_sizes_around_the_tiles(m):
    print(f"grouped group size {m}", flush=True)
    run_case(6, 3, 70, 320, 3 * m, "even", "gather", "bf16", "f32", seed=m)


@pytest.mark.parametrize("M", [6, 500])
def test_rows_outside_any_group_keep_what_they_hold(M):
    w, W = experts(6, 3, 90, 256)
    x = bf16_dev(synth.activations(M, 256, 1))
    off = np.array([2, 3, 3, M - 2])
    buf, Y = guarded((M, 90), torch.float32)
    fqm.gemm_grouped(w, x, i32(off), Y=Y)
    torch.cuda.synchronize()
    assert canaries_intact(buf)
    Yo, lim = oracle.layer.grouped(W, off, to_f64(x), None, None, None, M, -12345.0)
    assert (np.abs(to_f64(Y) - Yo) <= oracle.layer.rounded(lim, Yo, "f32")).all()


@pytest.mark.parametrize("M", [9, 400])
def test_indices_outside_read_zeros_and_store_nothing(M):
    w, W = experts(4, 2, 140, 192)
    rng = np.random.default_rng(M)
    src, dst = rng.integers(0, 7, size=M), rng.permutation(M)
    src[::4], src[1::4] = -1, 7
    dst[2::5], dst[3::5] = -2147483648, M
    x = bf16_dev(synth.activations(7, 192, 1))
    off = np.array([0, M // 3, M])
    buf, Y = guarded((M, 140), torch.bfloat16, fill=-64.0)
    fqm.gemm_grouped(w, x, i32(off), src=i32(src), dst=i32(dst), Y=Y)
    torch.cuda.synchronize()
    assert canaries_intact(buf, fill=-64.0)
    Yo, lim = oracle.layer.grouped(W, off, to_f64(x), src, dst, None, M, -64.0)
    assert (np.abs(to_f64(Y) - Yo) <= oracle.layer.rounded(lim, Yo, "bf16")).all()


@pytest.mark.parametrize("M", [5, 300])
def test_offsets_that_lead_outside_stay_inside(M):
    """Values outside the rows are taken as the rows' ends."""
    w, W = experts(6, 4, 64, 128)
    x = bf16_dev(synth.activations(M, 128, 1))
    buf, Y = guarded((M, 64), torch.float32)
    fqm.gemm_grouped(w, x, i32([-50, 2, 2, 3, 2 ** 31 - 1]), Y=Y)
    torch.cuda.synchronize()
    assert canaries_intact(buf)
    Yo, lim = oracle.layer.grouped(W, [0, 2, 2, 3, M], to_f64(x), None, None, None, M, 0.0)
    assert (np.abs(to_f64(Y) - Yo) <= oracle.layer.rounded(lim, Yo, "f32")).all()
    # a group that ends before it starts is empty
    Y.fill_(5.0)
    fqm.gemm_grouped(w, x, i32([1, 2, 0, 0, 0]), Y=Y)
    torch.cuda.synchronize()
    assert canaries_intact(buf)
    assert (np.abs(to_f64(Y[1]) - W[0] @ to_f64(x)[1]) <= oracle.layer.rounded(
        oracle.layer.grouped(W, [1, 2, 2, 2, 2], to_f64(x), None, None, None, M, 0.0)[1][1], W[0] @ to_f64(x)[1], "f32")).all()
    assert (Y[0] == 5).all() and (Y[2:] == 5).all()


@pytest.mark.parametrize("M", [4, 80])
def test_no_rows_and_no_columns(M):
    w, _ = experts(6, 3, 50, 128)
    Y = torch.full((M, 50), 3.0, device=DEV)
    x = bf16_dev(synth.activations(M, 128, 1))
    fqm.gemm_grouped(w, x, i32([0, 0, 0, 0]), Y=Y)
    assert (Y == 3).all()
    assert fqm.gemm_grouped(w, x[:0], i32([0, 0, 0, 0])).shape == (0, 50)
    none = fqm.Lut6Weights(w.packed, w.lut, 150, 0)
    fqm.gemm_grouped(none, x[:, :0].contiguous(), i32([0, 1, 1, M - 1]), Y=Y)
    assert (Y[:M - 1] == 0).all() and (Y[M - 1:] == 3).all()


@pytest.mark.parametrize("M", [6, 150])
def test_what_is_not_finite_stays_in_its_row(M):
    w, _ = experts(6, 2, 80, 256)
    x = bf16_dev(synth.activations(M, 256, 1))
    off = i32([0, M // 2, M])
    clean = fqm.gemm_grouped(w, x, off)
    x[1, 5], x[M - 1, 200] = float("nan"), float("inf")
    got = fqm.gemm_grouped(w, x, off)
    assert torch.isnan(got[1]).all() and not torch.isfinite(got[M - 1]).any()
    keep = torch.ones(M, dtype=torch.bool, device=DEV)
    keep[[1, M - 1]] = False
    assert torch.equal(got[keep], clean[keep])


@pytest.mark.parametrize("M", [4, 160])
def test_a_row_without_x_is_zeros_whatever_is_not_finite(M):
    w, _ = experts(6, 2, 80, 256)
    w.lut[:80, 3] = 0x7F80  # infinity in the first expert's tables
    x = bf16_dev(synth.activations(M, 256, 1))
    src = np.arange(M)
    src[::2] = -1
    scale = torch.full((M,), float("nan"), device=DEV)
    Y = torch.full((M, 80), 7.0, device=DEV)
    fqm.gemm_grouped(w, x, i32([0, M // 2, M]), src=i32(src), row_scale=scale, Y=Y)
    assert (Y[::2] == 0).all() and torch.isnan(Y[1::2]).all()
    # no columns: zeros too
    none = fqm.Lut6Weights(w.packed, w.lut, 160, 0)
    Y.fill_(7.0)
    fqm.gemm_grouped(none, x[:, :0].contiguous(), i32([0, M // 2, M]), row_scale=scale, Y=Y)
    assert (Y == 0).all()


def test_one_group_agrees_with_the_plain_product():
    w, W = experts(6, 1, 300, 512)
    x = bf16_dev(synth.activations(70, 512, 2))
    Y = fqm.gemm_grouped(w, x, i32([0, 70]))
    yo = to_f64(x) @ W[0].T
    ok, m = oracle.compare.check(to_f64(Y), yo, "bf16")
    assert ok, m


@pytest.mark.parametrize("M,xt", [(6, "bf16"), (6, "i8"), (400, "bf16"), (400, "i8")])
def test_another_stream_and_graph_replays(M, xt):
    w, _ = experts(6, 4, 200, 512)
    x = bf16_dev(synth.activations(M, 512, 1))
    xs = None
    if xt == "i8":
        x, xs = torch.randint(-127, 128, (M, 512), dtype=torch.int8, device=DEV), torch.rand(M, device=DEV)
    off = i32([0, M // 4, M // 2, M // 2, M])
    need = fqm.gemm_grouped_workspace_size(w, x, off, x_scale=xs)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV) if need else None
    Y = torch.empty(M, 200, dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    fqm.gemm_grouped(w, x, off, x_scale=xs, Y=Y, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(Y, fqm.gemm_grouped(w, x, off, x_scale=xs))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fqm.gemm_grouped(w, x, off, x_scale=xs, Y=Y, workspace=ws)
    for k in range(3):
        off.copy_(i32([0, k, max(k, M // 2 - k), M - 1, M]))
        ref = fqm.gemm_grouped(w, x, off, x_scale=xs)
        Y.zero_()
        if ws is not None:
            ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, ref)
