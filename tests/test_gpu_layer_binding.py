"""The binding of the operators around the products: what its calls allocate, take and refuse."""
import numpy as np
import pytest
import torch

import dequant_matmul_amd as fqm
from gpu_common import DEV

pytestmark = pytest.mark.gpu


def experts(E, N, K):
    codes = torch.randint(0, 64, (E * N, K), dtype=torch.uint8, device=DEV)
    return fqm.Lut6Weights.from_codes(codes, np.zeros((E * N, 64), dtype=np.int16), device=DEV)


@pytest.mark.parametrize("xt", ["bf16", "i8"])
def test_asking_for_the_workspace_allocates_nothing(xt):
    w = experts(4, 512, 256)
    X = torch.zeros(2000, 256, dtype=torch.int8 if xt == "i8" else torch.bfloat16, device=DEV)
    xs = torch.ones(2000, device=DEV) if xt == "i8" else None
    off = torch.tensor([0, 500, 900, 900, 2000], dtype=torch.int32, device=DEV)
    src = torch.zeros(3000, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    sizes = [fqm.gemm_grouped_workspace_size(w, X, off, x_scale=xs),
             fqm.gemm_grouped_workspace_size(w, X, off, src=src, x_scale=xs, out_dtype=torch.float32)]
    assert torch.cuda.max_memory_allocated() == before
    # and they are enough for the calls they were asked for
    for need, s, dt in zip(sizes, (None, src), (torch.bfloat16, torch.float32)):
        ws = torch.empty(need, dtype=torch.uint8, device=DEV) if need else None
        assert fqm.gemm_grouped(w, X, off, src=s, x_scale=xs, out_dtype=dt, workspace=ws).dtype == dt


@pytest.mark.parametrize("M", [3, 300])
def test_adapters_without_inputs_add_nothing(M):
    A = torch.zeros(2, 4, 0, dtype=torch.bfloat16, device=DEV)
    B = torch.randn(2, 70, 4, device=DEV).to(torch.bfloat16)
    x = torch.zeros(M, 0, dtype=torch.bfloat16, device=DEV)
    index = torch.arange(M, dtype=torch.int32, device=DEV) % 3 - 1
    base = torch.randn(M, 70, device=DEV)
    ad = fqm.Adapters(A, B)
    assert torch.equal(fqm.lora(ad, x, index, base=base, out_dtype=torch.float32), base)
    assert (fqm.lora(ad, x, index) == 0).all()


def test_adapters_at_any_address():
    flat = torch.randn(3 * 8 * 256 + 8, device=DEV).to(torch.bfloat16)
    A = flat[3:3 + 3 * 8 * 256].view(3, 8, 256)
    B = torch.randn(3 * 70 * 8 + 8, device=DEV).to(torch.bfloat16)[5:5 + 3 * 70 * 8].view(3, 70, 8)
    assert A.data_ptr() % 16 and B.data_ptr() % 16
    x = torch.randn(4, 256, device=DEV).to(torch.bfloat16)
    index = torch.tensor([2, 0, -1, 1], dtype=torch.int32, device=DEV)
    assert torch.equal(fqm.lora(fqm.Adapters(A, B), x, index), fqm.lora(fqm.Adapters(A.clone(), B.clone()), x, index))


def test_an_output_that_is_no_matrix_is_refused_like_the_other_operands():
    w = experts(2, 64, 128)
    X = torch.zeros(4, 128, dtype=torch.bfloat16, device=DEV)
    off = torch.tensor([0, 1, 4], dtype=torch.int32, device=DEV)
    for Y in ([1.0], torch.tensor(1.0, device=DEV), torch.zeros(4 * 64, device=DEV)):
        with pytest.raises(ValueError, match="Y "):
            fqm.gemm_grouped(w, X, off, Y=Y)
