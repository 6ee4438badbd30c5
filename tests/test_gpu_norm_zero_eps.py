"""The residual norm with eps = 0: a row of zeros in 8 bits has scale 0 and codes 0."""
import pytest
import torch

import dequant_matmul_amd as fqm
from gpu_common import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols,dtype", [(6, 200, "f32"), (6, 5120, "bf16"), (2100, 5120, "bf16"), (6, 7, "f32")])
def test_rows_of_zeros_in_8_bits(rows, cols, dtype):
    print(f"add_rms_norm eps 0 {rows}x{cols} {dtype}", flush=True)
    x = torch.randn(rows, cols, device=DEV).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    x[1], x[rows - 1] = 0, -0.0
    x[3] = 0
    x[3, cols - 1] = float("nan")
    w = 1 + 0.1 * torch.randn(cols, device=DEV)
    q = fqm.add_rms_norm(x, w, eps=0.0, out_dtype=torch.int8)
    for r in (1, rows - 1):
        assert q.scale[r] == 0 and (q.y[r] == 0).all()
    assert torch.isnan(q.scale[3]) and (q.y[3] == 0).all()
    rest = torch.ones(rows, dtype=torch.bool, device=DEV)
    rest[[1, 3, rows - 1]] = False
    assert torch.isfinite(q.scale[rest]).all() and (q.y[rest].abs().amax(1) == 127).all()
    # zeros met by a weight that is not finite: not a row of zeros
    w[0] = float("inf")
    q = fqm.add_rms_norm(x[1:2], w, eps=0.0, out_dtype=torch.int8)
    assert torch.isnan(q.scale).all() and (q.y == 0).all()


def test_a_residual_that_cancels_the_row():
    x = torch.randn(3, 640, device=DEV)
    q = fqm.add_rms_norm(x, eps=0.0, residual=-x, out_dtype=torch.int8)
    assert (q.scale == 0).all() and (q.y == 0).all() and (q.total == 0).all()
