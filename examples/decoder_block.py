"""A decoder layer's feed-forward block on quantized weights, decode or prefill:

    h, x      = add_rms_norm(attention output, residual)           bf16
    shared    = W x  + the requests' low-rank adapters              (LUT6, fp32 between the two)
    h, q      = add_rms_norm(shared, residual h)                    8 bits, one scale a row
    router    : each token takes k of E experts (plain torch)
    up, down  = the experts' products, grouped by expert            (LUT6 up, LUT4 down)
    h, x      = add_rms_norm(the token's k rows, residual h)        their sum, the residual, the next norm

Weights are random codes and tables, activations random; the point is how the
calls fit together.  Run:  python examples/decoder_block.py [tokens]
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
    sigma = cols ** -0.5
    lut = (torch.arange(n, device=device) - (n - 1) / 2) * (2 * sigma / n) * torch.ones(rows, 1, device=device)
    codes = torch.randint(0, n, (rows, cols), generator=g, device=device, dtype=torch.uint8)
    cls = fqm.Lut6Weights if bits == 6 else fqm.Lut4Weights
    return cls.from_codes(codes, lut.to(torch.bfloat16).view(torch.int16), device=device)


class DecoderBlock:
    def __init__(self, hidden=2048, inner=1024, experts=16, top_k=4, adapters=8, rank=16, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def randn(*shape):
            return torch.randn(*shape, generator=g, device=device)

        self.hidden, self.experts, self.top_k = hidden, experts, top_k
        self.norms = [(1 + 0.1 * randn(hidden)).to(torch.bfloat16) for _ in range(3)]
        self.shared = table_weights(hidden, hidden, 6, g, device)
        self.adapters = fqm.Adapters((randn(adapters, rank, hidden) * hidden ** -0.5).to(torch.bfloat16),
                                     (randn(adapters, hidden, rank) * 0.05).to(torch.bfloat16))
        self.router = randn(hidden, experts) * hidden ** -0.5
        self.up = table_weights(experts * inner, hidden, 6, g, device)      # the experts' matrices, one below the other
        self.down = table_weights(experts * hidden, inner, 4, g, device)

    def project(self, x):
        """The shared projection in fp32: GEMV up to 16 rows, GEMM (bf16) above."""
        return fqm.gemv(self.shared, x, out_dtype=torch.float32) if x.shape[0] <= 16 else fqm.gemm(self.shared, x)

    def route(self, q, scale):
        """Each token's experts: rows sorted by expert, where each came from, its weight."""
        logits = (q.float() * scale[:, None]) @ self.router
        weight, expert = torch.topk(torch.softmax(logits, 1), self.top_k, dim=1)
        order = torch.argsort(expert.flatten(), stable=True)
        offsets = torch.zeros(self.experts + 1, dtype=torch.int32, device=q.device)
        offsets[1:] = torch.cumsum((expert.flatten()[:, None] == torch.arange(self.experts, device=q.device)).sum(0), 0)
        weight = (weight / weight.sum(1, keepdim=True)).flatten()[order].contiguous()
        return offsets, order.to(torch.int32), weight

    def __call__(self, attention, residual, request):
        """attention, residual [tokens][hidden] bf16, request [tokens] int32 (-1: no adapter)
        -> (the next layer's normed input, the residual stream)."""
        x, _, h = fqm.add_rms_norm(attention, self.norms[0], residual=residual)
        base = self.project(x)
        out = fqm.lora(self.adapters, x, request, base=base)
        q, scale, h = fqm.add_rms_norm(out, self.norms[1], residual=h, out_dtype=torch.int8)
        offsets, order, weight = self.route(q, scale)
        token = torch.div(order, self.top_k, rounding_mode="floor").to(torch.int32)
        up = fqm.gemm_grouped(self.up, q, offsets, src=token, x_scale=scale)
        up = torch.nn.functional.silu(up)
        down = fqm.gemm_grouped(self.down, up, offsets, dst=order, row_scale=weight)  # back to the tokens' slots
        x, _, h = fqm.add_rms_norm(down.view(-1, self.top_k, self.hidden), self.norms[2], residual=h)
        return x, h


def main():
    tokens = int(sys.argv[1]) if len(sys.argv) > 1 else 8
    block = DecoderBlock()
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    attention, residual = (torch.randn(tokens, block.hidden, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    request = torch.randint(-1, block.adapters.count, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    for _ in range(3):
        x, h = block(attention, residual, request)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(20):
        x, h = block(attention, residual, request)
    b.record()
    torch.cuda.synchronize()
    print(f"{tokens} tokens: {a.elapsed_time(b) / 20 * 1e3:.0f} us a block, "
          f"normed rows' root mean square {x.float().square().mean().sqrt().item():.3f}")


if __name__ == "__main__":
    main()
