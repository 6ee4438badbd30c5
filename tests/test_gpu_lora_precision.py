"""What the adapters' second product keeps of t = scale * (A x): every bit of
the fp32 value, whatever type y has, in both forms of the call (rows collected
from a small batch, blocks of 64 rows of a large one)."""
import numpy as np
import pytest
import torch

import dequant_matmul_amd as fqm
import oracle
import synth
from gpu_common import DEV, bf16_dev, to_f64
from test_gpu_lora import T, order, pool, want

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("base", [None, "bf16", "f32"])
@pytest.mark.parametrize("M,count,rank,K,N,kind,mixed", [
    (1, 4, 16, 1024, 4096, "one", False),
    (48, 9, 32, 2048, 1000, "any", True),
    (200, 5, 100, 520, 257, "runs", True),
    (300, 6, 64, 1024, 640, "runs", False),
    (513, 3, 24, 328, 1025, "any", True),
])
def test_a_bf16_output_is_the_fp32_one_rounded(M, count, rank, K, N, kind, mixed, base):
    """The type of y decides its last rounding and nothing else."""
    print(f"lora bf16 and f32 M {M} count {count} rank {rank} {K}->{N} {kind} {base}", flush=True)
    rng = np.random.default_rng([M, rank, K])
    ad, _ = pool(count, rank, K, N, seed=M, mixed=mixed)
    x = bf16_dev(synth.activations(M, K, 5))
    index = torch.from_numpy(order(kind, M, count, rng).astype(np.int32)).to(DEV)
    b = torch.from_numpy(rng.standard_normal((M, N))).to(DEV).to(T[base]) if base else None
    fine = fqm.lora(ad, x, index, base=b, out_dtype=torch.float32)
    y = fqm.lora(ad, x, index, base=b, out_dtype=torch.bfloat16)
    assert torch.equal(y, fine.to(torch.bfloat16))


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M", [4, 300])
def test_all_24_bits_of_t_reach_y(M, out):
    """t = 1 + 2^-12 + 2^-23 (or its negative): three products of eight bits and less, exact in fp32, and so are its
    products with powers of two.  Two bf16 terms of it would lose the last one."""
    K, N = 64, 140
    A = torch.zeros(1, 2, K, dtype=torch.bfloat16, device=DEV)
    A[0, 0, 0], A[0, 0, 1], A[0, 0, 2] = 1.0, 2.0 ** -12, 2.0 ** -23
    A[0, 1] = -A[0, 0]
    B = torch.zeros(1, N, 2, dtype=torch.bfloat16, device=DEV)
    B[0, ::2, 0], B[0, 1::2, 1] = 4.0, 0.5
    x = torch.zeros(M, K, dtype=torch.bfloat16, device=DEV)
    x[:, :3] = 1.0
    index = torch.zeros(M, dtype=torch.int32, device=DEV)
    # the base takes all but t's last bit away
    base = torch.zeros(M, N, device=DEV)
    base[:, ::2], base[:, 1::2] = -4 * (1 + 2.0 ** -12), 0.5 * (1 + 2.0 ** -12)
    y = fqm.lora(fqm.Adapters(A, B), x, index, base=base, out_dtype=T[out])
    assert (y[:, ::2] == 2.0 ** -21).all() and (y[:, 1::2] == -(2.0 ** -24)).all()


@pytest.mark.parametrize("M", [5, 300])
def test_a_t_near_the_largest_fp32_stays_finite(M):
    """t between bf16's largest value and fp32's: its leading bf16 term must not round up to infinity."""
    K, N = 64, 70
    A = torch.zeros(1, 2, K, dtype=torch.bfloat16, device=DEV)
    A[0, 0, 0], A[0, 1, 0] = 2.0 ** 127, -(2.0 ** 127)
    B = torch.full((1, N, 2), 0.0, dtype=torch.bfloat16, device=DEV)
    B[0, ::2, 0], B[0, 1::2, 1] = 2.0 ** -100, 2.0 ** -100
    scale = torch.tensor([1.99951171875], device=DEV)  # 2 - 2^-11: t = +-2^127 (2 - 2^-11), exact in fp32
    x = torch.zeros(M, K, dtype=torch.bfloat16, device=DEV)
    x[:, 0] = 1.0
    index = torch.zeros(M, dtype=torch.int32, device=DEV)
    y = fqm.lora(fqm.Adapters(A, B, scale), x, index, out_dtype=torch.float32)
    t = 2.0 ** 27 * 1.99951171875  # one product, exact
    assert (y[:, ::2] == t).all() and (y[:, 1::2] == -t).all()


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M", [1, 40, 300])
@pytest.mark.parametrize("rank", [3, 40, 72])
def test_infinities_and_nan_of_b_give_what_the_sum_gives(rank, M, out):
    """Small whole numbers: t and y are exact, and t's lower bf16 terms are zeros, which must not meet an infinity."""
    K, N, count = 64, 150, 2
    g = torch.Generator().manual_seed(rank)
    A = torch.randint(-1, 2, (count, rank, K), generator=g).double()
    B = torch.randint(-4, 5, (count, N, rank), generator=g).double()
    inf = float("inf")
    B[0, 5, 0], B[0, 9, rank - 1], B[0, 64, 1], B[1, 149, 2] = inf, -inf, float("nan"), inf
    B[0, 17, 0], B[0, 17, 1] = inf, -inf
    x = torch.randint(-2, 3, (M, K), generator=g).double()
    index = torch.arange(M, dtype=torch.int32) % 3 - 1 if M > 1 else torch.zeros(1, dtype=torch.int32)
    base = torch.randint(-8, 9, (M, N), generator=g).double()
    ad = fqm.Adapters(A.to(torch.bfloat16).to(DEV), B.to(torch.bfloat16).to(DEV))
    y = fqm.lora(ad, x.to(torch.bfloat16).to(DEV), index.to(DEV), base=base.to(torch.bfloat16).to(DEV), out_dtype=T[out])
    want_ = base.clone()
    for m in range(M):
        i = int(index[m])
        if i >= 0:
            want_[m] += (B[i] * (A[i] @ x[m])).sum(1)
    assert torch.isinf(want_).any() and torch.isnan(want_).any()
    assert torch.equal(torch.nan_to_num(y.cpu().float(), nan=1e30, posinf=2e30, neginf=-2e30),
                       torch.nan_to_num(want_.to(T[out]).float(), nan=1e30, posinf=2e30, neginf=-2e30))
