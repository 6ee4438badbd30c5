"""The operators together, as a decoder block uses them, against the same block in fp64."""
import os
import sys

import pytest
import torch

import dequant_matmul_amd as fqm
from conftest import ROOT
from gpu_common import DEV

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(ROOT, "examples"))


def norm(h, w):
    return h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6) * w.double()


@pytest.mark.parametrize("tokens", [1, 5, 40, 300])
def test_block_matches_fp64(tokens):
    from decoder_block import DecoderBlock
    block = DecoderBlock(hidden=512, inner=256, experts=6, top_k=2, adapters=3, rank=8, seed=tokens)
    g = torch.Generator(device=DEV)
    g.manual_seed(tokens)
    attention, residual = (torch.randn(tokens, 512, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    request = torch.randint(-1, 3, (tokens,), generator=g, device=DEV, dtype=torch.int32)
    x, h = block(attention, residual, request)
    torch.cuda.synchronize()

    # the same in fp64; roundings to bf16 (2^-8) and 8 bits (1/254 of a row's largest) leave about 1 % in all
    h64 = attention.double() + residual.double()
    x64 = norm(h64, block.norms[0])
    ad = block.adapters
    out = x64 @ fqm.dequant(block.shared).double().t()
    for a in range(ad.count):
        m = request == a
        out[m] += x64[m] @ ad.A[a].double().t() @ ad.B[a].double().t()
    h64 = h64 + out
    x64 = norm(h64, block.norms[1])
    up, down = fqm.dequant(block.up).double().view(6, 256, 512), fqm.dequant(block.down).double().view(6, 512, 256)
    # the experts as the block itself took them (a near tie may go either way)
    first = fqm.add_rms_norm(attention, block.norms[0], residual=residual)
    shared = fqm.lora(ad, first.y, request, base=block.project(first.y))
    q, scale, _ = fqm.add_rms_norm(shared, block.norms[1], residual=first.total, out_dtype=torch.int8)
    offsets, order, weight = block.route(q, scale)
    off, total = offsets.tolist(), torch.zeros_like(h64)
    for e in range(6):
        rows = order[off[e]:off[e + 1]].long()
        tok = rows // 2
        mid = torch.nn.functional.silu(x64[tok] @ up[e].t())
        total.index_add_(0, tok, weight[off[e]:off[e + 1], None].double() * (mid @ down[e].t()))
    h64 = h64 + total
    x64 = norm(h64, block.norms[2])
    assert torch.isfinite(x).all()
    assert ((h.double() - h64).norm() / h64.norm()).item() < 0.02
    assert ((x.double() - x64).norm() / x64.norm()).item() < 0.02
