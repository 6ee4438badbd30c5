"""A layer of experts between its two norms, on quantized weights, decode or prefill:

    x, h    = block_norm(attention output, residual h)          the norm behind it, the sum, the norm in front
    h      += W2 (silu(W0 x) * W1 x)                            the shared expert: two calls of linear, the first gated
    route   : each token's k of E experts, and the plan of the products
    up, down: the experts' products, grouped by expert          (LUT6 up, LUT4 down)
    x, h    = block_norm(the token's k rows, residual h)        their sum, its norm and gate, the sum, the next norm

Weights are random codes and tables, activations random; the point is how the
calls fit together.  Run:  python examples/experts_layer.py [tokens]
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import dequant_matmul_amd as fqm  # noqa: E402


def table_weights(rows, cols, bits, g, device):
    """Random LUT6 / LUT4 weights: equal-width levels, codes uniform."""
    n = 1 << bits
    lut = (torch.arange(n, device=device) - (n - 1) / 2) * (2 * cols ** -0.5 / n) * torch.ones(rows, 1, device=device)
    codes = torch.randint(0, n, (rows, cols), generator=g, device=device, dtype=torch.uint8)
    cls = fqm.Lut6Weights if bits == 6 else fqm.Lut4Weights
    return cls.from_codes(codes, lut.to(torch.bfloat16).view(torch.int16), device=device)


class ExpertsLayer:
    def __init__(self, hidden=2048, inner=1024, experts=32, k=4, groups=4, top_groups=2, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def randn(*shape):
            return torch.randn(*shape, generator=g, device=device)

        self.hidden, self.k = hidden, k
        self.norms = [(0.1 * randn(hidden)).to(torch.bfloat16) for _ in range(4)]  # stored less one
        self.gate = (0.5 + 0.1 * randn(hidden)).to(torch.bfloat16)                 # of the experts' output, a factor a column
        self.router = (randn(hidden, experts) * hidden ** -0.5).to(torch.bfloat16)
        self.routing = dict(k=k, score="sigmoid", bias=0.05 * randn(experts), groups=groups, top_groups=top_groups, group_score="top2",
                            scale=2.5)
        self.shared_in = table_weights(2 * inner, hidden, 6, g, device)    # the gate's rows, then the other factor's
        self.shared_out = table_weights(hidden, inner, 6, g, device)
        self.up = table_weights(experts * inner, hidden, 6, g, device)     # the experts' matrices, one below the other
        self.down = table_weights(experts * hidden, inner, 4, g, device)

    def __call__(self, attention, residual):
        """attention, residual [tokens][hidden] bf16 -> (the next layer's normed input, the residual stream, the routing)."""
        x, _, h = fqm.block_norm(attention, residual, post_weight=self.norms[0], weight=self.norms[1], weight_offset=1.0)
        mid = fqm.linear(self.shared_in, x, act="silu", gated=True)
        fqm.linear(self.shared_out, mid, residual=h, y=h)
        r = fqm.route(x @ self.router, **self.routing)
        up = torch.nn.functional.silu(fqm.gemm_grouped(self.up, x, r.offsets, src=r.src))
        down = fqm.gemm_grouped(self.down, up, r.offsets, dst=r.dst, row_scale=r.row_scale)  # back to the tokens' slots
        x, _, h = fqm.block_norm(down.view(-1, self.k, self.hidden), h, post_weight=self.norms[2], weight=self.norms[3], gate=self.gate,
                                 weight_offset=1.0)
        return x, h, r


def main():
    tokens = int(sys.argv[1]) if len(sys.argv) > 1 else 8
    layer = ExpertsLayer()
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    attention, residual = (torch.randn(tokens, layer.hidden, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    for _ in range(3):
        x, h, r = layer(attention, residual)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(20):
        x, h, r = layer(attention, residual)
    b.record()
    torch.cuda.synchronize()
    print(f"{tokens} tokens: {a.elapsed_time(b) / 20 * 1e3:.0f} us a layer, the fullest expert has "
          f"{int((r.offsets[1:] - r.offsets[:-1]).max())} rows, normed rows' root mean square {x.float().square().mean().sqrt().item():.3f}")


if __name__ == "__main__":
    main()
