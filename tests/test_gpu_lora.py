"""The low-rank adapters against their fp64 definition: ranks, rows per
adapter, rows without one, types, odd widths, index orders."""
import numpy as np
import pytest
import torch

import dequant_matmul_amd as fqm
import oracle
import synth
from gpu_common import DEV, bf16_dev, canaries_intact, guarded, lut6_weights, to_f64

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f32": torch.float32}


def pool(count, rank, K, N, seed=0, mixed=False, scale=True):
    g = torch.Generator().manual_seed(seed)
    A = (torch.randn(count, rank, K, generator=g) * K ** -0.5).to(torch.bfloat16).to(DEV)
    B = (torch.randn(count, N, rank, generator=g) * 0.3).to(torch.bfloat16).to(DEV)
    sc = (0.5 + torch.rand(count, generator=g)).to(DEV) if scale else None
    ranks = torch.randint(0, rank + 1, (count,), generator=g, dtype=torch.int32).to(DEV) if mixed else None
    return fqm.Adapters(A, B, sc, ranks), (A, B, sc, ranks)


def order(kind, M, count, rng):
    if kind == "one":
        return np.full(M, count - 1)
    if kind == "none":
        return np.where(np.arange(M) % 2, -1, count + 3)
    if kind == "runs":
        cut = np.sort(rng.integers(0, M + 1, size=count - 1))
        return np.repeat(np.arange(count), np.diff(np.concatenate([[0], cut, [M]])))
    return rng.integers(-1, count, size=M)  # any order, some without


def want(parts, x, index, base):
    A, B, sc, ranks = parts
    return oracle.layer.lora(to_f64(A), to_f64(B), None if sc is None else to_f64(sc),
                             None if ranks is None else ranks.cpu().numpy(), to_f64(x), index,
                             None if base is None else to_f64(base))


@pytest.mark.parametrize("M,count,rank,K,N,kind,base,out,mixed", [
    (1, 1, 16, 512, 256, "one", "bf16", "bf16", False),
    (1, 3, 1, 8, 1, "one", None, "f32", False),
    (2, 2, 5, 264, 77, "any", "f32", "bf16", True),
    (8, 8, 16, 5120, 1000, "any", "bf16", "bf16", False),
    (16, 4, 64, 1088, 129, "any", "f32", "f32", True),
    (17, 30, 8, 2048, 640, "any", "bf16", "f32", True),
    (33, 2, 128, 520, 300, "runs", "bf16", "bf16", False),
    (64, 5, 256, 1024, 65, "runs", None, "f32", True),
    (65, 3, 32, 4096, 512, "none", "bf16", "bf16", False),
    (70, 70, 12, 768, 200, "any", "f32", "f32", True),
    (100, 7, 100, 1096, 130, "runs", None, "bf16", False),
    (257, 6, 16, 640, 1001, "runs", "bf16", "bf16", True),
    (300, 40, 4, 328, 90, "any", "bf16", "f32", False),
    (5, 3, 33, 16, 0, "any", None, "f32", False),
])
def test_against_definition(M, count, rank, K, N, kind, base, out, mixed):
    print(f"lora M {M} count {count} rank {rank} {K}->{N} {kind} {base} {out}", flush=True)
    rng = np.random.default_rng([M, rank, K])
    ad, parts = pool(count, rank, K, N, seed=M, mixed=mixed, scale=M % 3 != 0)
    x = bf16_dev(synth.activations(M, K, 5))
    index = order(kind, M, count, rng)
    b = torch.from_numpy(rng.standard_normal((M, N))).to(DEV).to(T[base]) if base else None
    buf, y = guarded((M, N), T[out])
    fqm.lora(ad, x, torch.from_numpy(index.astype(np.int32)).to(DEV), base=b, y=y)
    torch.cuda.synchronize()
    assert canaries_intact(buf)
    yo, lim = want(parts, x, index, b)
    assert (np.abs(to_f64(y) - yo) <= oracle.layer.rounded(lim, yo, out)).all()


def test_rows_without_an_adapter_are_the_base_bit_for_bit():
    ad, _ = pool(3, 16, 512, 300)
    x = torch.randn(40, 512, device=DEV).to(torch.bfloat16)
    index = torch.tensor([-1, 0, 3, 2, -2147483648, 2147483647, 1, 3] * 5, dtype=torch.int32, device=DEV)
    base = torch.randn(40, 300, device=DEV).to(torch.bfloat16)
    y = fqm.lora(ad, x, index, base=base)
    bare = (index < 0) | (index > 2)
    assert torch.equal(y[bare], base[bare])
    assert not torch.equal(y[~bare], base[~bare])


def test_in_place_and_padded_layouts_give_the_same():
    g = torch.Generator().manual_seed(4)
    A = torch.randn(4, 12, 640, generator=g).to(torch.bfloat16).to(DEV)
    wide = torch.full((4, 200, 24), float("nan"), dtype=torch.bfloat16, device=DEV)
    B = torch.randn(4, 200, 12, generator=g).to(torch.bfloat16).to(DEV)
    wide[:, :, :12] = B
    x = torch.randn(9, 640, device=DEV).to(torch.bfloat16)
    index = torch.arange(9, dtype=torch.int32, device=DEV) % 4
    base = torch.randn(9, 200, device=DEV)
    want_ = fqm.lora(fqm.Adapters(A, B), x, index, base=base, out_dtype=torch.float32)
    got = fqm.lora(fqm.Adapters(A, wide[:, :, :12]), x, index, base=base, y=base)
    assert got.data_ptr() == base.data_ptr() and torch.equal(got, want_)
    Aw = torch.full((4, 12, 704), float("nan"), dtype=torch.bfloat16, device=DEV)
    Aw[:, :, :640] = A
    assert torch.equal(fqm.lora(fqm.Adapters(Aw[:, :, :640], B), x, index), fqm.lora(fqm.Adapters(A, B), x, index))


def test_what_lies_past_an_adapters_rank_is_not_used():
    A = torch.randn(3, 20, 256, device=DEV).to(torch.bfloat16)
    B = torch.randn(3, 130, 20, device=DEV).to(torch.bfloat16)
    ranks = torch.tensor([7, 0, 55], dtype=torch.int32, device=DEV)  # 55: the layout's 20
    for fill in (0.0, float("nan"), float("inf")):
        A[0, 7:], B[0, :, 7:], A[1], B[1] = fill, fill, fill, fill
        for M in (6, 80):
            index = torch.arange(M, dtype=torch.int32, device=DEV) % 3
            torch.manual_seed(M)
            x = torch.randn(M, 256, device=DEV).to(torch.bfloat16)
            y = fqm.lora(fqm.Adapters(A, B, ranks=ranks), x, index, out_dtype=torch.float32)
            if fill == 0.0:
                clean = {**locals().get("clean", {}), M: y}
            assert torch.equal(y, clean[M])
            assert (y[1::3] == 0).all()


def test_a_row_that_is_not_finite_stays_alone():
    ad, _ = pool(2, 16, 512, 140)
    for M in (5, 90):
        x = torch.randn(M, 512, device=DEV).to(torch.bfloat16)
        index = torch.arange(M, dtype=torch.int32, device=DEV) % 3 - 1
        clean = fqm.lora(ad, x, index)
        x[4, 7] = float("nan")
        x[2, 9] = float("inf")
        y = fqm.lora(ad, x, index)
        rest = torch.ones(M, dtype=torch.bool, device=DEV)
        rest[[2, 4]] = False
        assert torch.equal(y[rest], clean[rest])
        assert torch.isnan(y[4]).any() if index[4] >= 0 else torch.equal(y[4], clean[4])


def test_results_do_not_depend_on_the_order_of_rows():
    ad, _ = pool(9, 24, 1024, 333, mixed=True)
    x = torch.randn(200, 1024, device=DEV).to(torch.bfloat16)
    index = torch.randint(-1, 9, (200,), dtype=torch.int32, device=DEV)
    y = fqm.lora(ad, x, index, out_dtype=torch.float32)
    p = torch.randperm(200, device=DEV)
    assert torch.equal(fqm.lora(ad, x[p].contiguous(), index[p].contiguous(), out_dtype=torch.float32), y[p])


def test_beside_the_shared_projection():
    """gemv in fp32, the adapters on top, one rounding to bf16."""
    w = lut6_weights(256, 512, 1)
    ad, parts = pool(3, 16, 512, 256)
    x = bf16_dev(synth.activations(4, 512, 9))
    index = np.array([2, -1, 0, 2])
    base = fqm.gemv(w, x, out_dtype=torch.float32)
    y = fqm.lora(ad, x, torch.from_numpy(index.astype(np.int32)).to(DEV), base=base)
    yo, lim = want(parts, x, index, base)
    assert (np.abs(to_f64(y) - yo) <= oracle.layer.rounded(lim, yo, "bf16")).all()


def test_another_stream_and_graph_replays():
    ad, _ = pool(5, 16, 1024, 500)
    for M in (3, 80):
        x = torch.randn(M, 1024, device=DEV).to(torch.bfloat16)
        index = torch.randint(0, 5, (M,), dtype=torch.int32, device=DEV)
        base = torch.randn(M, 500, device=DEV).to(torch.bfloat16)
        ws = torch.empty(fqm.lora_workspace_size(ad, M), dtype=torch.uint8, device=DEV)
        y = torch.empty_like(base)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        fqm.lora(ad, x, index, base=base, y=y, workspace=ws, stream=side)
        side.synchronize()
        assert torch.equal(y, fqm.lora(ad, x, index, base=base))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fqm.lora(ad, x, index, base=base, y=y, workspace=ws)
        for k in range(3):
            index.copy_(torch.roll(index, 1))
            ref = fqm.lora(ad, x, index, base=base)
            y.zero_()
            ws.fill_(255)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, ref)


@pytest.mark.parametrize("M,count,rank,K,N,kind,base,out", [
    (100, 3, 256, 264, 300, "runs", "bf16", "bf16"),
    (65, 64, 256, 72, 1030, "any", "f32", "f32"),
    (130, 2, 17, 5128, 64, "runs", None, "bf16"),
    (1000, 3, 16, 40, 63, "any", "bf16", "f32"),
])
def test_wide_ranks_and_narrow_layers_in_blocks_of_rows(M, count, rank, K, N, kind, base, out):
    print(f"lora blocks M {M} count {count} rank {rank} {K}->{N}", flush=True)
    rng = np.random.default_rng([M, rank, K])
    ad, parts = pool(count, rank, K, N, seed=M)
    x = bf16_dev(synth.activations(M, K, 5))
    index = order(kind, M, count, rng)
    b = torch.from_numpy(rng.standard_normal((M, N))).to(DEV).to(T[base]) if base else None
    buf, y = guarded((M, N), T[out])
    fqm.lora(ad, x, torch.from_numpy(index.astype(np.int32)).to(DEV), base=b, y=y)
    torch.cuda.synchronize()
    assert canaries_intact(buf)
    yo, lim = want(parts, x, index, b)
    assert (np.abs(to_f64(y) - yo) <= oracle.layer.rounded(lim, yo, out)).all()


@pytest.mark.parametrize("M,count,rank,K,N,kind,base,out,mixed", [
    (321, 3, 256, 264, 200, "runs", "bf16", "f32", False),
    (260, 2, 100, 1096, 131, "runs", "f32", "bf16", True),
    (400, 5, 64, 648, 1025, "any", None, "bf16", True),
    (290, 4, 40, 56, 130, "runs", "bf16", "bf16", False),
    (700, 2, 33, 2056, 77, "one", "f32", "f32", False),
    (257, 3, 16, 320, 512, "none", "bf16", "bf16", False),
])
def test_many_rows_of_all_ranks_and_types(M, count, rank, K, N, kind, base, out, mixed):
    print(f"lora many rows M {M} count {count} rank {rank} {K}->{N} {kind} {base} {out}", flush=True)
    rng = np.random.default_rng([M, rank, K])
    ad, parts = pool(count, rank, K, N, seed=M, mixed=mixed, scale=M % 2 == 0)
    x = bf16_dev(synth.activations(M, K, 5))
    index = order(kind, M, count, rng)
    b = torch.from_numpy(rng.standard_normal((M, N))).to(DEV).to(T[base]) if base else None
    buf, y = guarded((M, N), T[out])
    fqm.lora(ad, x, torch.from_numpy(index.astype(np.int32)).to(DEV), base=b, y=y)
    torch.cuda.synchronize()
    assert canaries_intact(buf)
    yo, lim = want(parts, x, index, b)
    assert (np.abs(to_f64(y) - yo) <= oracle.layer.rounded(lim, yo, out)).all()


def test_many_rows_keep_to_themselves_and_to_their_ranks():
    """What is not finite in a row of x, past an adapter's rank, or in another adapter, touches nothing else."""
    M, K, N = 300, 328, 140
    A = torch.randn(4, 20, K, device=DEV).to(torch.bfloat16)
    B = torch.randn(4, N, 20, device=DEV).to(torch.bfloat16)
    ranks = torch.tensor([7, 0, 55, 20], dtype=torch.int32, device=DEV)
    index = (torch.arange(M, dtype=torch.int32, device=DEV) % 5) - 1
    x = torch.randn(M, K, device=DEV).to(torch.bfloat16)
    base = torch.randn(M, N, device=DEV).to(torch.bfloat16)
    clean = fqm.lora(fqm.Adapters(A, B, ranks=ranks), x, index, base=base)
    A[0, 7:], B[0, :, 7:], A[1], B[1], A[3, 2, 5] = (float("nan"),) * 5
    x[11, 3] = float("inf")
    y = fqm.lora(fqm.Adapters(A, B, ranks=ranks), x, index, base=base)
    keep = index != 3
    keep[11] = False
    assert torch.equal(y[keep], clean[keep])
    assert torch.equal(y[index == 1], base[index == 1]) and torch.equal(y[index == -1], base[index == -1])
    assert torch.isnan(y[index == 3]).all()


@pytest.mark.parametrize("M", [3, 300])
def test_a_stream_of_its_own_gets_its_own_memory(M):
    """Outputs and workspace of a call on another stream are that stream's: work that the current
    stream does meanwhile does not get their memory."""
    ad, _ = pool(4, 16, 1024, 300)
    x = torch.randn(M, 1024, device=DEV).to(torch.bfloat16)
    index = torch.arange(M, dtype=torch.int32, device=DEV) % 4
    ref = fqm.lora(ad, x, index)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ys = []
    for _ in range(8):
        ys.append(fqm.lora(ad, x, index, stream=side))
        for n in (1 << 12, 1 << 16, 1 << 20):
            torch.full((n,), float("nan"), device=DEV)
    side.synchronize()
    assert all(torch.equal(y, ref) for y in ys)
