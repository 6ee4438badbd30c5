"""Cases of the operators around the quantized products, their plain forms and their 64-bit values.

Three operators that stand beside ``y = W x`` in a decoder layer:

``norm``     fqm.add_rms_norm: the residual's addition (over one or several terms, as the rows that a
             token's experts return), the root-mean-square norm, and the normed row in bf16 or in 8 bits
             with one scale a row.
``lora``     fqm.lora: the low-rank adapters of many requests, added to the shared projection's output.
``grouped``  fqm.gemm_grouped: products grouped by expert, ragged sizes, weights in the per-row table
             formats (6- and 4-bit codes), rows gathered on the way in or scattered and weighted on the
             way out.

``run`` computes them with elementary torch operations in 32 bits, or, where ``own`` is true, through the
package.  Widths are those of the package's configurations (5120, 17408, 4096, 1088, 1000) or generic.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ---------------------------------------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------------------------------------
def listed():
    return [
        # one token between two projections of a decode step: only latency counts
        dict(name="norm_token", op="norm", rows=1, cols=5120, terms=1, x="bf16", res="bf16", out="bf16", pad=0),
        # a decode batch whose normed rows go to the experts in 8 bits
        dict(name="norm_decode_i8", op="norm", rows=16, cols=5120, terms=1, x="bf16", res="bf16", out="i8", pad=0),
        # a ragged prompt on a narrow odd layer that keeps its residual stream in fp32, rows inside wider ones
        dict(name="norm_prompt_f32", op="norm", rows=1031, cols=1087, terms=1, x="f32", res="f32", out="bf16", pad=9),
        # a prompt's rows after eight experts each: their sum, the residual, the next layer's norm in 8 bits
        dict(name="norm_experts_i8", op="norm", rows=4096, cols=5120, terms=8, x="bf16", res="bf16", out="i8", pad=0),
        # one token of one request beside the up projection
        dict(name="lora_token", op="lora", M=1, count=8, rank=16, mixed=False, K=5120, N=17408, base="bf16", out="bf16",
             runs=False, none=0),
        # a decode batch of many requests beside the down projection, ranks of their own, some without an adapter
        dict(name="lora_decode", op="lora", M=48, count=32, rank=32, mixed=True, K=17408, N=5120, base="f32",
             out="bf16", runs=False, none=5),
        # mixed short prompts on an odd layer, the correction alone in fp32
        dict(name="lora_ragged", op="lora", M=777, count=12, rank=12, mixed=True, K=4096, N=1000, base="no", out="f32",
             runs=True, none=100),
        # prompts of sixteen requests together beside the up projection
        dict(name="lora_prompts", op="lora", M=4096, count=16, rank=64, mixed=False, K=5120, N=17408, base="bf16",
             out="bf16", runs=True, none=0),
        # one token through its eight experts' up projection
        dict(name="experts_token", op="grouped", bits=6, T=1, k=8, E=64, K=5120, N=1024, way="up", x="bf16",
             out="bf16", skew=0.0),
        # a decode batch through its experts' down projection, weighted, each row back to its token's slot
        dict(name="experts_decode", op="grouped", bits=4, T=24, k=4, E=32, K=1024, N=5120, way="down", x="bf16",
             out="f32", skew=0.5),
        # a mid-sized batch, rows in 8 bits, an odd width, experts of very different load
        dict(name="experts_batch_i8", op="grouped", bits=6, T=200, k=6, E=40, K=2048, N=1000, way="up", x="i8",
             out="bf16", skew=1.0),
        # a prompt through its experts' up projection
        dict(name="experts_prompt", op="grouped", bits=6, T=2048, k=8, E=64, K=5120, N=1024, way="up", x="bf16",
             out="bf16", skew=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "lora", "grouped"])
    if op == "norm":
        cols, terms = _log(rng, 64, 17408), rng.choice([1, 1, 2, 4, 8])
        rows = _log(rng, 1, min(16384, max(2, 160_000_000 // (cols * terms))))
        x = rng.choice(["bf16", "bf16", "f32"])
        return dict(op=op, rows=rows, cols=cols, terms=terms, x=x, res=rng.choice([x, x, "no"]),
                    out=rng.choice(["bf16", "bf16", "f32", "i8"]), pad=rng.choice([0, 0, 8, 3]))
    if op == "lora":
        K, N = 16 * _log(rng, 8, 1088), _log(rng, 100, 17408)
        rank = rng.choice([1, 4, 8, 12, 16, 32, 64, 100, 128])
        M = _log(rng, 1, min(4096, max(2, 370_000_000_000 // (rank * (K + N) * 16))))
        return dict(op=op, M=M, count=_log(rng, 1, 64 if rank <= 32 else 16), rank=rank, mixed=rng.random() < 0.5, K=K, N=N,
                    base=rng.choice(["bf16", "bf16", "f32", "no"]), out=rng.choice(["bf16", "f32"]),
                    runs=M > 64 or rng.random() < 0.3, none=rng.randrange(0, M // 4 + 1))
    K, N = 64 * _log(rng, 4, 80), _log(rng, 64, 5120)
    E = _log(rng, 2, min(128, max(3, 330_000_000 // (K * N))))
    k = min(E, rng.choice([1, 2, 4, 6, 8]))
    T = _log(rng, 1, min(2048, max(2, 85_000_000_000 // (k * K * N))))
    way = rng.choice(["up", "down"])
    return dict(op=op, bits=rng.choice([6, 6, 4]), T=T, k=k, E=E, K=K, N=N, way=way,
                x="bf16" if way == "down" else rng.choice(["bf16", "i8"]), out=rng.choice(["bf16", "f32"]),
                skew=rng.choice([0.0, 0.5, 1.0]))


_SIZE = {"bf16": 2, "f32": 4, "i8": 1, "no": 0}


def _ranks(c):
    """The adapters' ranks: all of them the largest, or eighths of it in turn."""
    return [max(1, c["rank"] * ((7 * a) % 8 + 1) // 8) if c["mixed"] else c["rank"] for a in range(c["count"])]


def work(c):
    if c["op"] == "norm":
        n = c["rows"] * c["cols"]
        total = c["res"] != "no" or c["terms"] > 1
        b = n * (c["terms"] * _SIZE[c["x"]] + _SIZE[c["res"]] + _SIZE[c["out"]]) + 2 * c["cols"]
        b += n * (_SIZE[c["x"] if c["res"] == "no" else c["res"]] if total else 0)
        b += 4 * c["rows"] if c["out"] == "i8" else 0
        return {"bytes": b, "flops": n * (c["terms"] + 5)}
    if c["op"] == "lora":
        M, K, N, ranks = c["M"], c["K"], c["N"], _ranks(c)
        used = min(c["count"], M - c["none"])
        b = M * (2 * K + N * (_SIZE[c["base"]] + _SIZE[c["out"]]) + 4) + sum(ranks[:used]) * (K + N) * 2
        return {"bytes": b, "flops": 2 * (M - c["none"]) * sum(ranks) // c["count"] * (K + N)}
    E, K, N, M = c["E"], c["K"], c["N"], c["T"] * c["k"]
    met = E * (1.0 - (1.0 - c["k"] / E) ** c["T"])  # experts that some token takes, were they drawn evenly
    b = met * N * (K * c["bits"] / 8 + 2 * 2 ** c["bits"])
    b += (c["T"] if c["way"] == "up" else M) * (K * _SIZE[c["x"]]) + M * N * _SIZE[c["out"]] + 4 * M
    return {"bytes": int(b), "flops": 2 * M * N * K}


# ---------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) % (2 ** 62))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _rows_in(v, pad):
    """The rows of v inside rows that are `pad` values wider."""
    if not pad:
        return v.contiguous()
    wide = torch.zeros(*v.shape[:-1], v.shape[-1] + pad, dtype=v.dtype, device=v.device)
    wide[..., :v.shape[-1]] = v
    return wide[..., :v.shape[-1]]


def _prepare_norm(c, g):
    rows, cols, terms = c["rows"], c["cols"], c["terms"]
    # a residual stream: rows of different size, a few columns far above the rest
    size = torch.exp(0.5 * _randn(g, rows, 1))
    column = torch.where(torch.rand(cols, generator=g, device=DEV) < 0.002, 20.0, 1.0)
    x = _randn(g, rows, terms, cols) * (size * column)[:, None] if terms > 1 else _randn(g, rows, cols) * size * column
    s = dict(x=_rows_in(x.to(_DT[c["x"]]), c["pad"]), weight=(1 + 0.2 * _randn(g, cols)).to(torch.bfloat16), res=None)
    if c["res"] != "no":
        s["res"] = _rows_in((3 * _randn(g, rows, cols) * size * column).to(_DT[c["res"]]), c["pad"])
    return s


def _prepare_lora(c, g, seed):
    M, K, N, R, count = c["M"], c["K"], c["N"], c["rank"], c["count"]
    ldb = (R + 7) // 8 * 8
    rng = np.random.default_rng([int(seed) % (2 ** 62), 3])
    live = M - c["none"]
    if c["runs"]:  # prompts: every adapter's rows together, of ragged lengths
        cut = np.sort(rng.integers(0, live + 1, size=count - 1))
        idx = np.repeat(np.arange(count), np.diff(np.concatenate([[0], cut, [live]])))
        idx = np.concatenate([idx, np.full(c["none"], -1)])
    else:  # single tokens: any order; every adapter is met while there are rows for it
        idx = np.concatenate([np.arange(min(live, count)), rng.integers(0, count, size=max(0, live - count)),
                              np.full(c["none"], -1)])
        rng.shuffle(idx)
    ranks = _ranks(c)
    kept = torch.tensor(ranks, device=DEV)
    A = _randn(g, count, R, K).mul_(K ** -0.5)
    B = _randn(g, count, N, ldb).mul_(0.1)
    A *= (torch.arange(R, device=DEV)[None, :, None] < kept[:, None, None])
    B *= (torch.arange(ldb, device=DEV)[None, None, :] < kept[:, None, None])
    s = dict(A=A.to(torch.bfloat16), B=B.to(torch.bfloat16), rank=R,
             scale=0.5 + 1.5 * torch.rand(count, generator=g, device=DEV), ranks=kept.to(torch.int32),
             x=_randn(g, M, K).to(torch.bfloat16), index=torch.from_numpy(idx.astype(np.int32)).to(DEV),
             base=_randn(g, M, N).to(_DT[c["base"]]) if c["base"] != "no" else None, out=_DT[c["out"]])
    if own:
        import dequant_matmul_amd as fqm
        s["adapters"] = fqm.Adapters(s["A"], s["B"][:, :, :R], s["scale"], s["ranks"])
    return s


def _pack(codes, bits):
    """Little-endian fields of 6 or 4 bits, rows padded to 16 bytes."""
    rows, cols = codes.shape
    if bits == 6:
        q = codes.view(rows, cols // 4, 4).to(torch.int32)
        v = q[..., 0] | (q[..., 1] << 6) | (q[..., 2] << 12) | (q[..., 3] << 18)
        b = torch.stack([v & 255, (v >> 8) & 255, v >> 16], -1).to(torch.uint8).view(rows, -1)
    else:
        q = codes.view(rows, cols // 2, 2)
        b = q[..., 0] | (q[..., 1] << 4)
    ld = (b.shape[1] + 15) // 16 * 16
    out = torch.zeros(rows, ld, dtype=torch.uint8, device=DEV)
    out[:, :b.shape[1]] = b
    return out


def _codes(g, rows, cols, bits):
    """Codes of Gaussian weights under equal-width shells, the outermost at 4.5 standard deviations."""
    tiers = 2 ** (bits - 1)
    out = torch.empty(rows, cols, dtype=torch.uint8, device=DEV)
    step = max(1, 50_000_000 // cols)
    for r in range(0, rows, step):
        w = _randn(g, min(step, rows - r), cols)
        t = (w.abs() * (tiers / 4.5)).clamp_(max=tiers - 1).to(torch.uint8)
        out[r:r + step] = torch.where(w >= 0, t + tiers, tiers - 1 - t)
    return out


def _prepare_grouped(c, g):
    E, K, N, T, k, bits = c["E"], c["K"], c["N"], c["T"], c["k"], c["bits"]
    tiers = 2 ** (bits - 1)
    sigma = torch.exp(torch.rand(E * N, 1, generator=g, device=DEV) * math.log(10.0) + math.log(0.005))
    level = torch.arange(2 * tiers, device=DEV) - tiers + 0.5
    level = level + 0.3 * (2 * torch.rand(E * N, 2 * tiers, generator=g, device=DEV) - 1)
    lut = (level * (sigma * 4.5 / tiers)).to(torch.bfloat16)
    packed = _pack(_codes(g, E * N, K, bits), bits)
    # routing: each token takes k experts, some experts far more often than others
    liked = c["skew"] * _randn(g, E)
    score, expert = torch.topk(_randn(g, T, E) + liked, k, dim=1)
    order = torch.argsort(expert.reshape(-1), stable=True)
    counts = torch.bincount(expert.reshape(-1), minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.cumsum(counts, 0)
    s = dict(packed=packed, lut=lut, offsets=offsets, E=E, N=N, K=K, bits=bits, way=c["way"], out=_DT[c["out"]],
             x_scale=None, src=None, dst=None, row_scale=None, M=T * k)
    if c["way"] == "up":  # rows of the tokens, one for each expert that a token takes
        x = _randn(g, T, K)
        s["src"] = torch.div(order, k, rounding_mode="floor").to(torch.int32)
        if c["x"] == "i8":
            s["x_scale"] = x.abs().amax(1) / 127
            x = torch.round(x / s["x_scale"][:, None]).to(torch.int8)
        s["X"] = x if c["x"] == "i8" else x.to(torch.bfloat16)
    else:  # rows in the experts' order; each goes back to its token's slot, weighted
        s["X"] = _randn(g, T * k, K).to(torch.bfloat16)
        s["dst"] = order.to(torch.int32)
        s["row_scale"] = torch.softmax(score, 1).reshape(-1)[order].contiguous()
    if own:
        import dequant_matmul_amd as fqm
        s["weights"] = (fqm.Lut6Weights if bits == 6 else fqm.Lut4Weights)(packed, lut, E * N, K)
    return s


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "norm":
        s = _prepare_norm(case, g)
        s["out"] = case["out"]
    elif case["op"] == "lora":
        s = _prepare_lora(case, g, seed)
    else:
        s = _prepare_grouped(case, g)
    s["op"] = case["op"]
    return s


# ---------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------
def _run_norm(s):
    x, res = s["x"], s["res"]
    total = None
    if own:
        import dequant_matmul_amd as fqm
        dt = torch.int8 if s["out"] == "i8" else _DT[s["out"]]
        y, scale, total = fqm.add_rms_norm(x, s["weight"], eps=EPS, residual=res, out_dtype=dt)
        if s["out"] != "i8":
            return dict(y=y, total=total)
    else:
        h = x.float()
        if x.dim() == 3:
            h = h.sum(1)
        if res is not None:
            h = h + res.float()
        if res is not None or x.dim() == 3:
            total = h.to(x.dtype if res is None else res.dtype)
        y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * s["weight"].float()
        if s["out"] != "i8":
            return dict(y=y.to(_DT[s["out"]]), total=total)
        scale = y.abs().amax(1) / 127
        y = torch.round(y / torch.where(scale > 0, scale, 1.0)[:, None])
    # what the 8 bits stand for, to be compared as such
    value = torch.empty(y.shape, dtype=torch.bfloat16, device=y.device)
    torch.mul(y, scale[:, None], out=value)
    return dict(y=value, scale=scale, total=total)


def _run_lora(s):
    if own:
        import dequant_matmul_amd as fqm
        return fqm.lora(s["adapters"], s["x"], s["index"], base=s["base"], out_dtype=s["out"])
    count, R, K = s["A"].shape
    N = s["B"].shape[1]
    # every row against every adapter, then only its own kept
    t = (s["x"].float() @ s["A"].float().reshape(count * R, K).t()).view(-1, count, R)
    mine = s["index"][:, None] == torch.arange(count, dtype=torch.int32, device=DEV)
    t = t * (mine * s["scale"])[:, :, None]
    y = t.view(-1, count * R) @ s["B"][:, :, :R].float().permute(0, 2, 1).reshape(count * R, N)
    if s["base"] is not None:
        y = y + s["base"].float()
    return y.to(s["out"])


def _unpack(packed, cols, bits):
    b = packed[..., :cols * bits // 8]
    if bits == 4:
        return torch.stack([b & 15, b >> 4], -1).view(*b.shape[:-1], cols)
    b = b.reshape(*b.shape[:-1], cols // 4, 3).to(torch.int32)
    v = b[..., 0] | (b[..., 1] << 8) | (b[..., 2] << 16)
    return torch.stack([v & 63, (v >> 6) & 63, (v >> 12) & 63, v >> 18], -1).view(*v.shape[:-1], cols)


def _run_grouped(s):
    if own:
        import dequant_matmul_amd as fqm
        return fqm.gemm_grouped(s["weights"], s["X"], s["offsets"], src=s["src"], x_scale=s["x_scale"], dst=s["dst"],
                                row_scale=s["row_scale"], out_dtype=s["out"])
    E, N, K, M = s["E"], s["N"], s["K"], s["M"]
    counts = s["offsets"].diff()
    met = torch.nonzero(counts).flatten()  # the experts that have rows
    codes = _unpack(s["packed"].view(E, N, -1)[met], K, s["bits"])
    W = torch.gather(s["lut"].float().view(E, N, -1)[met], 2, codes.long())
    x = s["X"].float()
    if s["x_scale"] is not None:
        x = x * s["x_scale"][:, None]
    if s["src"] is not None:
        x = x[s["src"].long()]
    # the rows of each expert, padded to the longest
    at = s["offsets"][:-1][met].long()[:, None] + torch.arange(int(counts.max()), device=DEV)
    live = torch.arange(at.shape[1], device=DEV) < counts[met][:, None]
    y = torch.bmm(x[at.clamp(max=M - 1)], W.transpose(1, 2).contiguous())[live]
    if s["row_scale"] is not None:
        y = y * s["row_scale"][:, None]
    if s["dst"] is not None:
        out = torch.empty_like(y)
        out[s["dst"].long()] = y
        y = out
    return y.to(s["out"])


def run(state):
    return {"norm": _run_norm, "lora": _run_lora, "grouped": _run_grouped}[state["op"]](state)


# ---------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        parts = [s["x"]] if s["x"].dim() == 2 else list(s["x"].unbind(1))
        if s["res"] is not None:
            parts.append(s["res"])
        h = torch.zeros(parts[0].shape, dtype=torch.float64, device=DEV)
        for p in parts:
            h += p.double()
        norm = torch.sqrt((h * h).sum(1) / h.shape[1] + EPS)
        y = h / norm[:, None] * s["weight"].double()
        total = h if len(parts) > 1 else None
        if case["out"] != "i8":
            return dict(y=y, total=total)
        scale = y.abs().max(1).values / 127
        return dict(y=torch.round(y / scale[:, None]) * scale[:, None], scale=scale, total=total)
    if case["op"] == "lora":
        x, index = s["x"].double(), s["index"]
        y = torch.zeros(x.shape[0], case["N"], dtype=torch.float64, device=DEV)
        if s["base"] is not None:
            y += s["base"].double()
        for a, r in enumerate(_ranks(case)):
            rows = torch.nonzero(index == a).flatten()
            low = torch.mm(x[rows], s["A"][a, :r].double().t().contiguous())
            y[rows] += s["scale"][a].double() * torch.mm(low, s["B"][a, :, :r].double().t().contiguous())
        return y
    if 2 * s["M"] * s["N"] * s["K"] > 400e9:
        return None
    E, N, K, bits = s["E"], s["N"], s["K"], s["bits"]
    offsets = s["offsets"].tolist()
    y = torch.zeros(s["M"], N, dtype=torch.float64, device=DEV)
    raw = s["packed"].view(E, N, -1).to(torch.int64)
    place = torch.arange(K, device=DEV) * bits  # the bit at which a code starts
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        if lo == hi:
            continue
        two = raw[e][:, place // 8] | (raw[e][:, (place // 8 + 1).clamp(max=raw.shape[2] - 1)] << 8)
        codes = (two >> (place % 8)) & (2 ** bits - 1)
        W = s["lut"].view(E, N, -1)[e].double().gather(1, codes)
        rows = torch.arange(lo, hi, device=DEV) if s["src"] is None else s["src"][lo:hi].long()
        x = s["X"][rows].double()
        if s["x_scale"] is not None:
            x = x * s["x_scale"][rows].double()[:, None]
        v = torch.mm(x, W.t().contiguous())
        if s["row_scale"] is not None:
            v = v * s["row_scale"][lo:hi].double()[:, None]
        y[torch.arange(lo, hi, device=DEV) if s["dst"] is None else s["dst"][lo:hi].long()] = v
    return y
