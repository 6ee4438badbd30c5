"""The adapters on more than 256 rows, taken in blocks of 64 as they lie: wide
ranks, narrow layers, one to four passes of outputs a workgroup, y in place of
base, graph replays."""
import numpy as np
import pytest
import torch

import dequant_matmul_amd as fqm
import oracle
import synth
from gpu_common import DEV, bf16_dev, canaries_intact, guarded, to_f64
from test_gpu_lora import T, order, pool, want

pytestmark = pytest.mark.gpu


def passes_of_a_workgroup(M, N):
    return max(1, min(4, (M + 63) // 64 * ((N + 127) // 128) // 1024))


def run(M, count, rank, K, N, kind, base, out, mixed, pick):
    assert M > 256
    rng = np.random.default_rng([M, rank, K])
    ad, parts = pool(count, rank, K, N, seed=M, mixed=mixed)
    x = bf16_dev(synth.activations(M, K, 5))
    index = order(kind, M, count, rng)
    b = torch.from_numpy(rng.standard_normal((M, N))).to(DEV).to(T[base]) if base else None
    buf, y = guarded((M, N), T[out])
    fqm.lora(ad, x, torch.from_numpy(index.astype(np.int32)).to(DEV), base=b, y=y)
    torch.cuda.synchronize()
    assert canaries_intact(buf)
    yo, lim = want(parts, x[pick], index[pick], None if b is None else b[pick])
    assert (np.abs(to_f64(y[pick]) - yo) <= oracle.layer.rounded(lim, yo, out)).all()


@pytest.mark.parametrize("M,count,rank,K,N,kind,base,out", [
    (300, 3, 256, 264, 300, "runs", "bf16", "bf16"),
    (321, 64, 256, 72, 1030, "any", "f32", "f32"),
    (258, 2, 17, 5128, 64, "runs", None, "bf16"),
    (1000, 3, 200, 40, 63, "any", "bf16", "f32"),
])
def test_wide_ranks_and_narrow_layers(M, count, rank, K, N, kind, base, out):
    print(f"lora blocks M {M} count {count} rank {rank} {K}->{N}", flush=True)
    run(M, count, rank, K, N, kind, base, out, False, np.arange(M))


@pytest.mark.parametrize("M,count,rank,K,N,kind,base,out,passes", [
    (2100, 5, 16, 72, 8201, "runs", "bf16", "bf16", 2),
    (2100, 3, 40, 64, 8200, "any", "f32", "f32", 2),
    (2111, 4, 72, 72, 12001, "runs", None, "bf16", 3),
    (2111, 4, 12, 72, 12001, "any", "bf16", "f32", 3),
    (2110, 6, 64, 72, 16001, "runs", "bf16", "bf16", 4),
    (2110, 3, 20, 128, 16100, "runs", "f32", "bf16", 4),
])
def test_several_passes_of_outputs(M, count, rank, K, N, kind, base, out, passes):
    print(f"lora blocks M {M} count {count} rank {rank} {K}->{N} {passes} passes", flush=True)
    assert passes_of_a_workgroup(M, N) == passes
    pick = np.unique(np.r_[0, 1, 63, 64, 65, M // 2, M - 65, M - 1, np.arange(7, M, 97)])
    run(M, count, rank, K, N, kind, base, out, True, pick)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,rank,N", [(300, 16, 333), (2111, 40, 12001)])
def test_y_in_place_of_base(M, rank, N, dtype):
    ad, _ = pool(4, rank, 264, N, mixed=True)
    x = bf16_dev(synth.activations(M, 264, 5))
    index = torch.randint(-1, 4, (M,), dtype=torch.int32, device=DEV)
    base = torch.randn(M, N, device=DEV).to(T[dtype])
    ref = fqm.lora(ad, x, index, base=base, out_dtype=T[dtype])
    got = fqm.lora(ad, x, index, base=base, y=base)
    assert got.data_ptr() == base.data_ptr() and torch.equal(got, ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K,N", [(300, 1024, 500), (2111, 72, 12001)])
def test_graph_replays(M, K, N, dtype):
    ad, _ = pool(5, 24, K, N, mixed=True)
    x = bf16_dev(synth.activations(M, K, 5))
    index = torch.randint(-1, 5, (M,), dtype=torch.int32, device=DEV)
    base = torch.randn(M, N, device=DEV).to(T[dtype])
    ws = torch.empty(fqm.lora_workspace_size(ad, M), dtype=torch.uint8, device=DEV)
    y = torch.empty_like(base)
    fqm.lora(ad, x, index, base=base, y=y, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fqm.lora(ad, x, index, base=base, y=y, workspace=ws)
    for k in range(3):
        index.copy_(torch.roll(index, 1))
        ref = fqm.lora(ad, x, index, base=base, out_dtype=T[dtype])
        y.zero_()
        ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ref)
