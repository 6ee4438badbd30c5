"""The activations over their whole range, in the product's epilogue and at the block's gate, against their fp64
definition: the tails where an exponential leaves fp32's range and the product with it does not, and far beyond."""
import numpy as np
import pytest
import torch

import dequant_matmul_amd as fqm
import oracle
from gpu_common import DEV, lut6_weights, to_f64

pytestmark = pytest.mark.gpu

ACTS = [None, "relu", "silu", "gelu", "gelu_tanh", "sigmoid", "tanh"]


def arguments():
    """-110 to 110, dense where exp(-v) passes fp32's largest number, Phi(v) and gelu_tanh's factor their smallest; the
    smallest and largest magnitudes."""
    tails = [np.linspace(-93, -80, 521), np.linspace(-14.5, -9, 441), np.linspace(-64.01, -63.99, 41)]
    sizes = np.concatenate([10.0 ** np.arange(-37, 39, 1.0), [2.0 ** -126, 2.0 ** -140, np.finfo(np.float32).max]])
    return np.concatenate([np.linspace(-110, 110, 881), *tails, sizes, -sizes, [0.0]]).astype(np.float32)


def limit(name, v, factor):
    """(value, bound) of act(v) * factor in fp32.

    act's own bound is relative; on top, a result below 2^-126 is stored in steps of 2^-149, and so is erfc(z) before
    gelu multiplies it by v / 2.  With two roundings on the way: at most 2 |v| / 2 + 2 such steps, times the factor."""
    v = v.astype(np.float64)
    y, e, _ = oracle.block.act(v, name)
    steps = np.where(np.abs(y) < 1e-30, np.minimum(np.abs(v), 200) + 2, 2) * 2.0 ** -149
    y, e = y * factor, (e + steps) * abs(factor)
    return y, oracle.layer.rounded(e, y, "f32")


def check(name, v, got, factor=1.0):
    y, lim = limit(name, v, factor)
    off = np.abs(to_f64(got) - y) - lim
    worst = off.argmax()
    assert (off <= 0).all(), (name, v[worst], to_f64(got)[worst], y[worst], int((off > 0).sum()))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [1, 5, 12, 40])
def test_in_the_products_epilogue(M, act):
    """x is zeros, so v is the bias; a number of rows for each of the product's kernels."""
    print(f"activation {act} M {M}", flush=True)
    b = arguments()
    n = len(b)
    x = torch.zeros(M, 1024, dtype=torch.bfloat16, device=DEV)
    bias = torch.from_numpy(b).to(DEV)
    y = fqm.linear(lut6_weights(n, 1024, 3), x, bias=bias, act=act, out_dtype=torch.float32)
    assert torch.equal(y, y[:1].expand(M, n))
    check(act, b, y[M - 1])
    both = torch.cat([bias, torch.full((n,), 0.75, device=DEV)])
    y = fqm.linear(lut6_weights(2 * n, 1024, 3), x, bias=both, act=act, gated=True, out_dtype=torch.float32)
    assert torch.equal(y, y[:1].expand(M, n))
    check(act, b, y[M - 1], 0.75)


@pytest.mark.parametrize("act", ACTS)
def test_at_the_blocks_gate(act):
    g = arguments()
    gate = torch.from_numpy(g).to(DEV)
    x = torch.ones(2, len(g), device=DEV)
    out = fqm.block_norm(x, gate=gate, gate_act=act, post=False, out_dtype=None).total  # a value for each column
    check(act, g, out[1])
    out = fqm.block_norm(torch.ones(len(g), 1, device=DEV), gate=gate[:, None], gate_act=act, post=False, out_dtype=None).total
    check(act, g, out[:, 0])  # one for each row


@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "sigmoid"])
@pytest.mark.parametrize("M", [1, 5, 12, 40, 300])
def test_a_value_does_not_depend_on_its_neighbours(M, act):
    """One far tail among a wave's values: the others keep their bits, with a residual behind the activation."""
    n = 520
    g = torch.Generator(device=DEV)
    g.manual_seed(M)
    bias = 3 * torch.randn(2 * n, generator=g, device=DEV)
    x = torch.zeros(M, 1024, dtype=torch.bfloat16, device=DEV)
    res = torch.randn(M, 2 * n, generator=g, device=DEV)
    far = bias.clone()
    far[::40] = -90.0
    keep = torch.ones(2 * n, dtype=torch.bool, device=DEV)
    keep[::40] = False
    w = lut6_weights(2 * n, 1024, 3)
    for gated in (False, True):
        cols = n if gated else 2 * n
        a, b = (fqm.linear(w, x, bias=v, act=act, gated=gated, residual=res[:, :cols], out_dtype=torch.float32) for v in (bias, far))
        kept = keep[:n] & keep[n:] if gated else keep
        assert torch.equal(a[:, kept], b[:, kept]) and not torch.equal(a, b)
    gates = [fqm.block_norm(res, res.flip(1), gate=v, gate_act=act, post=False, out_dtype=None).total for v in (bias, far)]
    assert torch.equal(gates[0][:, keep], gates[1][:, keep]) and not torch.equal(*gates)
