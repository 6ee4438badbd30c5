"""Products grouped by expert with few rows a group: the kernel whose waves own
rows of W, at 1, 2 and 4 rows of W a wave, passes of 1 to 4 rows of X, widths
of part of a chunk to thirty chunks, against the fp64 definition."""
import numpy as np
import pytest
import torch

import dequant_matmul_amd as fqm
import oracle
from gpu_common import DEV, canaries_intact, guarded, to_f64
from test_gpu_grouped import T, i32

pytestmark = pytest.mark.gpu


def few(E, K, M):
    """The sizes that this kernel is chosen for."""
    return M * 4096 <= E * K


def rows_of_w(E, N, M):
    r = min(E, M) * N // 4096
    return 4 if r >= 4 else 2 if r >= 2 else 1


def uneven(E, M):
    """Offsets: groups of 0 to 9 rows, the empty ones between them and at the end."""
    sizes, left = [], M
    for e in range(E):
        m = min(left, (0, 9, 0, 1, 0, 0, 4, 2, 0, 3, 5, 0)[e % 12])
        sizes.append(m if e < E - 1 else left)
        left -= sizes[-1]
    return np.r_[0, np.cumsum(sizes)]


class Experts:
    """Random codes and tables of E matrices; the decoded values of those asked for."""

    def __init__(self, bits, E, N, K, seed=0):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        n = 1 << bits
        self.E, self.N, self.K = E, N, K
        self.codes = torch.randint(0, n, (E * N, K), generator=g, device=DEV, dtype=torch.uint8)
        level = torch.arange(n, device=DEV) - (n - 1) / 2 + torch.rand(E * N, n, generator=g, device=DEV) - 0.5
        self.lut = (level * (0.01 + torch.rand(E * N, 1, generator=g, device=DEV))).to(torch.bfloat16)
        cls = fqm.Lut6Weights if bits == 6 else fqm.Lut4Weights
        self.weights = cls.from_codes(self.codes, self.lut.view(torch.int16), device=DEV)

    def decoded(self, e):
        r = slice(e * self.N, (e + 1) * self.N)
        return to_f64(torch.gather(self.lut[r].float(), 1, self.codes[r].long()))

    def definition(self, off, x, src, dst, row_scale, y_rows, fill):
        """oracle.layer.grouped over the groups that have rows."""
        off = np.clip(off, 0, None)
        met = [e for e in range(self.E) if off[e + 1] > off[e]]
        W = np.stack([self.decoded(e) for e in met]) if met else np.zeros((0, self.N, self.K))
        return oracle.layer.grouped(W, [off[e] for e in met] + [off[met[-1] + 1] if met else 0], x, src, dst, row_scale, y_rows,
                                    fill)


def rows(rng, M, K, xt):
    """Rows of X (bf16 or 8 bits with scales) and their values."""
    v = rng.standard_normal((M, K))
    if xt == "bf16":
        x = torch.from_numpy(v).to(DEV).to(torch.bfloat16)
        return x, None, to_f64(x)
    xs = (np.abs(v).max(axis=1, initial=1e-3) / 127).astype(np.float32)
    q = np.rint(v / xs[:, None]).astype(np.int8)
    q[0, : min(K, 2)] = -128  # all of int8
    return torch.from_numpy(q).to(DEV), torch.from_numpy(xs).to(DEV), q.astype(np.float64) * xs.astype(np.float64)[:, None]


@pytest.mark.parametrize("bits", [6, 4])
@pytest.mark.parametrize("E,N,K,M,way,xt,out", [
    (1, 1, 4096, 1, "plain", "bf16", "f32"),
    (128, 33, 64, 2, "gather", "bf16", "bf16"),     # K of a part of a piece row
    (64, 77, 1088, 16, "scatter", "bf16", "f32"),   # a last chunk of four pieces
    (64, 515, 1088, 16, "gather", "i8", "bf16"),    # two rows of W a wave
    (64, 1025, 1088, 16, "scatter", "i8", "f32"),   # four
    (24, 1031, 1024, 6, "plain", "bf16", "bf16"),   # one chunk: a row of W is one step
    (16, 700, 5120, 13, "gather", "bf16", "f32"),
    (20, 1500, 2112, 10, "scatter", "bf16", "bf16"),
    (8, 130, 8192, 16, "gather", "i8", "f32"),      # three rows of X a pass
    (5, 100, 12288, 15, "scatter", "bf16", "f32"),  # two
    (4, 40, 16384, 16, "gather", "bf16", "bf16"),   # one
    (2, 20, 30720, 15, "plain", "i8", "f32"),       # the widest
    (3, 2900, 5120, 3, "plain", "bf16", "f32"),
])
def test_against_definition(bits, E, N, K, M, way, xt, out):
    print(f"grouped rows {bits} bits E {E} {K}->{N} M {M} {way} {xt} {out}, {rows_of_w(E, N, M)} rows of W a wave", flush=True)
    assert few(E, K, M)
    rng = np.random.default_rng([E, N, K, M])
    ex = Experts(bits, E, N, K, seed=M)
    off = uneven(E, M)
    src = dst = rs = None
    x_rows = M
    if way == "gather":
        x_rows = max(1, M // 3)
        src = rng.integers(0, x_rows, size=M)
    if way == "scatter":
        dst = rng.permutation(M)
        rs = rng.uniform(0.1, 1.5, size=M).astype(np.float32)
    x, xs, xv = rows(rng, x_rows, K, xt)
    buf, Y = guarded((M, N), T[out])
    assert fqm.gemm_grouped_workspace_size(ex.weights, x, i32(off), src=None if src is None else i32(src), x_scale=xs) == 0
    fqm.gemm_grouped(ex.weights, x, i32(off), src=None if src is None else i32(src), x_scale=xs,
                     dst=None if dst is None else i32(dst), row_scale=None if rs is None else torch.from_numpy(rs).to(DEV), Y=Y)
    torch.cuda.synchronize()
    assert canaries_intact(buf)
    Yo, lim = ex.definition(off, xv, src, dst, rs, M, -12345.0)
    assert (np.abs(to_f64(Y) - Yo) <= oracle.layer.rounded(lim, Yo, out)).all()


def test_all_rows_a_wave_are_met():
    assert {rows_of_w(E, N, M) for E, N, M in ((64, 77, 16), (64, 515, 16), (64, 1025, 16))} == {1, 2, 4}


@pytest.mark.parametrize("E,N,K,M", [(32, 90, 1088, 8), (32, 1030, 1088, 8)])
def test_rows_outside_any_group_keep_what_they_hold(E, N, K, M):
    assert few(E, K, M)
    ex = Experts(6, E, N, K)
    x, _, xv = rows(np.random.default_rng(1), M, K, "bf16")
    off = np.r_[2, 3, np.full(E - 2, 3), M - 2]
    buf, Y = guarded((M, N), torch.float32)
    fqm.gemm_grouped(ex.weights, x, i32(off), Y=Y)
    torch.cuda.synchronize()
    assert canaries_intact(buf)
    Yo, lim = ex.definition(off, xv, None, None, None, M, -12345.0)
    assert (np.abs(to_f64(Y) - Yo) <= oracle.layer.rounded(lim, Yo, "f32")).all()
    # ends outside the rows are taken as the rows' ends, a group that ends before it starts is empty
    Y.fill_(5.0)
    fqm.gemm_grouped(ex.weights, x, i32(np.r_[-50, 2, np.full(E - 2, 2), 2 ** 31 - 1]), Y=Y)
    torch.cuda.synchronize()
    assert canaries_intact(buf)
    Yo, lim = ex.definition(np.r_[0, 2, np.full(E - 2, 2), M], xv, None, None, None, M, 5.0)
    assert (np.abs(to_f64(Y) - Yo) <= oracle.layer.rounded(lim, Yo, "f32")).all()
    Y.fill_(5.0)
    fqm.gemm_grouped(ex.weights, x, i32(np.r_[1, 2, np.zeros(E - 1)]), Y=Y)
    torch.cuda.synchronize()
    Yo, lim = ex.definition(np.r_[1, 2, np.full(E - 1, 2)], xv, None, None, None, M, 5.0)
    assert (np.abs(to_f64(Y) - Yo) <= oracle.layer.rounded(lim, Yo, "f32")).all()


@pytest.mark.parametrize("xt", ["bf16", "i8"])
def test_indices_outside_read_zeros_and_store_nothing(xt):
    E, N, K, M = 32, 140, 1088, 8
    assert few(E, K, M)
    ex = Experts(4, E, N, K)
    src = np.array([3, -1, 0, 7, 1, 2 ** 31 - 1, 6, 5])
    dst = np.array([1, 0, M, 3, -2147483648, 4, 7, 2])
    x, xs, xv = rows(np.random.default_rng(2), 7, K, xt)
    off = uneven(E, M)
    buf, Y = guarded((M, N), torch.bfloat16, fill=-64.0)
    fqm.gemm_grouped(ex.weights, x, i32(off), src=i32(src), x_scale=xs, dst=i32(dst), Y=Y)
    torch.cuda.synchronize()
    assert canaries_intact(buf, fill=-64.0)
    Yo, lim = ex.definition(off, xv, src, dst, None, M, -64.0)
    assert (np.abs(to_f64(Y) - Yo) <= oracle.layer.rounded(lim, Yo, "bf16")).all()


@pytest.mark.parametrize("N", [80, 1030])
def test_what_is_not_finite_stays_in_its_row(N):
    E, K, M = 32, 1088, 8
    assert few(E, K, M)
    ex = Experts(6, E, N, K)
    x, _, _ = rows(np.random.default_rng(3), M, K, "bf16")
    off = i32(np.r_[0, 5, np.full(E - 1, M)])
    clean = fqm.gemm_grouped(ex.weights, x, off)
    x[1, 5], x[M - 1, 1087] = float("nan"), float("inf")
    got = fqm.gemm_grouped(ex.weights, x, off)
    assert torch.isnan(got[1]).all() and not torch.isfinite(got[M - 1]).any()
    keep = torch.ones(M, dtype=torch.bool, device=DEV)
    keep[[1, M - 1]] = False
    assert torch.equal(got[keep], clean[keep])
    # a row without a row of X is zeros whatever tables and factors hold
    ex.weights.lut[:N] = float("inf")
    src = np.arange(M)
    src[::2] = -1
    Y = torch.full((M, N), 7.0, device=DEV)
    fqm.gemm_grouped(ex.weights, x, off, src=i32(src), row_scale=torch.full((M,), float("nan"), device=DEV), Y=Y)
    assert (Y[::2] == 0).all() and torch.isnan(Y[1::2]).all()


@pytest.mark.parametrize("N,xt", [(200, "bf16"), (600, "i8"), (2100, "bf16")])
def test_another_stream_and_graph_replays(N, xt):
    E, K, M = 32, 1088, 8
    assert few(E, K, M)
    ex = Experts(6, E, N, K)
    x, xs, _ = rows(np.random.default_rng(4), M, K, xt)
    off = i32(uneven(E, M))
    Y = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    fqm.gemm_grouped(ex.weights, x, off, x_scale=xs, Y=Y, stream=side)
    side.synchronize()
    assert torch.equal(Y, fqm.gemm_grouped(ex.weights, x, off, x_scale=xs))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fqm.gemm_grouped(ex.weights, x, off, x_scale=xs, Y=Y)
    for k in range(3):
        off.copy_(i32(np.r_[0, k, np.full(E - 2, k + 1), M]))
        ref = fqm.gemm_grouped(ex.weights, x, off, x_scale=xs)
        Y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, ref)
