"""Cases of the operators that complete a decoder layer around the quantized products, their plain forms and
their 64-bit values.

``linear``  fqm.linear: the product with 6- or 4-bit table weights and, in its epilogue, bias, activation (or
            the gated activation of two stacked matrices) and the residual's addition.
``route``   fqm.route: a token's experts from its router logits, their weights, and the plan that the products
            grouped by expert take (rows sorted by expert, where each came from and goes back to).
``block``   fqm.block_norm: the norm behind a block, its gate and scales, the residual's addition and the norm
            in front of the next block, out in bf16, fp32 or 8 bits.

``run`` computes them with elementary torch operations in 32 bits (the router's choice in 64, so that scores
next to each other keep their order), or, where ``own`` is true, through the package.  Widths are those of the
package's configurations (5120, 17408, 4096, 1088, 1000) or generic.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-6
LARGEST = 3.4028234663852886e38  # of fp32


# ---------------------------------------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------------------------------------
def listed():
    return [
        # one token's down projection, added to its residual stream: only the weights' stream counts
        dict(name="linear_token", op="linear", bits=6, M=1, K=17408, N=5120, gated=False, act="none", bias="no",
             res="bf16", out="bf16", padx=0, pad=0),
        # a decode batch's gate and up projections in one product
        dict(name="linear_gated_decode", op="linear", bits=6, M=16, K=5120, N=17408, gated=True, act="silu", bias="no",
             res="no", out="bf16", padx=0, pad=0),
        # short prompts on an odd layer with a bias, its residual stream in fp32, all rows inside wider ones
        dict(name="linear_ragged", op="linear", bits=4, M=77, K=4160, N=1000, gated=False, act="gelu", bias="f32",
             res="f32", out="f32", padx=8, pad=3),
        # a prompt's gate and up projections
        dict(name="linear_prompt", op="linear", bits=6, M=2048, K=5120, N=8704, gated=True, act="silu", bias="bf16",
             res="no", out="bf16", padx=0, pad=0),
        # one token's experts: only latency counts
        dict(name="route_token", op="route", T=1, E=64, k=8, x="bf16", score="softmax", bias=False, groups=1,
             top_groups=1, group_score="max", renormalise=True, scale=1.0, closed=0.0, padding=0, pad=0),
        # a decode batch: sigmoid scores, a bias that balances the experts, four of eight groups by their two best
        dict(name="route_decode", op="route", T=48, E=256, k=8, x="f32", score="sigmoid", bias=True, groups=8,
             top_groups=4, group_score="top2", renormalise=True, scale=2.5, closed=0.0, padding=0, pad=0),
        # a ragged padded batch, an odd number of experts, some of them closed to some tokens, rows inside wider ones
        dict(name="route_ragged", op="route", T=777, E=60, k=6, x="f32", score="softmax", bias=True, groups=1,
             top_groups=1, group_score="max", renormalise=False, scale=1.0, closed=0.1, padding=31, pad=5),
        # a long prompt's tokens, routed as the decode batch
        dict(name="route_prompt", op="route", T=16384, E=256, k=8, x="f32", score="sigmoid", bias=True, groups=8,
             top_groups=4, group_score="top2", renormalise=True, scale=2.5, closed=0.0, padding=0, pad=0),
        # one token between two blocks of a decode step
        dict(name="block_token", op="block", rows=1, cols=5120, terms=1, x="bf16", res="bf16", gate="no", act="none",
             out="bf16", pad=0),
        # a decode batch after six experts each, a learned scale per column, out in 8 bits for the next products
        dict(name="block_decode_i8", op="block", rows=48, cols=5120, terms=6, x="bf16", res="bf16", gate="cols", act="none",
             out="i8", pad=0),
        # a ragged prompt on a narrow odd layer, a gate of its own for every value, rows inside wider ones
        dict(name="block_ragged_f32", op="block", rows=1031, cols=1087, terms=1, x="f32", res="f32", gate="full",
             act="tanh", out="bf16", pad=9),
        # a long prompt, a gate per token
        dict(name="block_prompt", op="block", rows=8192, cols=5120, terms=1, x="bf16", res="bf16", gate="rows",
             act="sigmoid", out="bf16", pad=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "route", "block"])
    if op == "linear":
        K = 1024 * _log(rng, 1, 17) if rng.random() < 0.5 else 64 * _log(rng, 4, 272)
        gated = rng.random() < 0.5
        N = _log(rng, 64, min(17408, 170_000_000 // (K * (1 + gated))))
        M = _log(rng, 1, min(4096, max(2, 180_000_000_000 // (K * N * (1 + gated)))))
        return dict(op=op, bits=rng.choice([6, 6, 4]), M=M, K=K, N=N, gated=gated,
                    act=rng.choice(["silu", "gelu", "gelu_tanh"]) if gated else rng.choice(["none", "none", "silu", "gelu", "relu"]),
                    bias=rng.choice(["no", "bf16", "f32"]), res=rng.choice(["no", "bf16", "f32"]),
                    out=rng.choice(["bf16", "bf16", "f32"]), padx=rng.choice([0, 0, 8, 64]), pad=rng.choice([0, 0, 8, 3]))
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _log(rng, max(2, 8 // groups), 512 // groups)
        top_groups = rng.randint((groups + 1) // 2, groups)
        T = _log(rng, 1, min(16384, 4_000_000 // E))
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(E // groups * top_groups, 12)), x=rng.choice(["f32", "f32", "bf16"]),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups, top_groups=top_groups,
                    group_score=rng.choice(["max", "top2"]), renormalise=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]),
                    closed=rng.choice([0.0, 0.0, 0.1, 0.6]), padding=rng.randrange(0, T // 4 + 1), pad=rng.choice([0, 0, 5]))
    cols, terms = _log(rng, 64, 17408), rng.choice([1, 1, 2, 4, 8])
    rows = _log(rng, 1, min(16384, max(2, 40_000_000 // (cols * terms))))
    x = rng.choice(["bf16", "bf16", "f32"])
    gate = rng.choice(["no", "cols", "rows", "full"])
    return dict(op=op, rows=rows, cols=cols, terms=terms, x=x, res=rng.choice([x, x, "f32"]), gate=gate,
                act="none" if gate == "no" else rng.choice(["none", "sigmoid", "tanh"]),
                out=rng.choice(["bf16", "bf16", "f32", "i8"]), pad=rng.choice([0, 0, 8, 3]))


_SIZE = {"bf16": 2, "f32": 4, "i8": 1, "no": 0}


def work(c):
    if c["op"] == "linear":
        M, K, N = c["M"], c["K"], c["N"]
        rows = N * (1 + c["gated"])
        b = rows * (K * c["bits"] / 8 + 2 * 2 ** c["bits"] + _SIZE[c["bias"]])
        b += M * (2 * K + N * (_SIZE[c["res"]] + _SIZE[c["out"]]))
        return {"bytes": int(b), "flops": 2 * M * rows * K}
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        return {"bytes": T * E * _SIZE[c["x"]] + 4 * E * (1 + c["bias"]) + T * k * 4 * 5, "flops": 8 * T * E}
    rows, cols = c["rows"], c["cols"]
    n = rows * cols
    b = n * (c["terms"] * _SIZE[c["x"]] + 2 * _SIZE[c["res"]] + _SIZE[c["out"]]) + 4 * cols
    b += {"no": 0, "cols": cols, "rows": rows, "full": n}[c["gate"]] * _SIZE[c["x"]]
    b += 4 * rows if c["out"] == "i8" else 0
    return {"bytes": b, "flops": n * (c["terms"] + 10)}


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


def _prepare_linear(c, g):
    M, K, N, bits = c["M"], c["K"], c["N"], c["bits"]
    rows, tiers = N * (1 + c["gated"]), 2 ** (bits - 1)
    # rows of different size, such that a product of normed activations is of the order of one
    sigma = torch.exp(0.5 * _randn(g, rows, 1)) * K ** -0.5
    level = torch.arange(2 * tiers, device=DEV) - tiers + 0.5
    level = level + 0.3 * (2 * torch.rand(rows, 2 * tiers, generator=g, device=DEV) - 1)
    lut = (level * (sigma * 4.5 / tiers)).to(torch.bfloat16)
    s = dict(packed=_pack(_codes(g, rows, K, bits), bits), lut=lut, K=K, N=N, bits=bits, gated=c["gated"], act=c["act"],
             x=_rows_in(_randn(g, M, K).to(torch.bfloat16), c["padx"]), bias=None, res=None, out=_DT[c["out"]])
    if c["bias"] != "no":
        s["bias"] = (0.5 * _randn(g, rows)).to(_DT[c["bias"]])
    if c["res"] != "no":
        s["res"] = _rows_in((2 * _randn(g, M, N)).to(_DT[c["res"]]), c["pad"])
    if own:
        import dequant_matmul_amd as fqm
        s["weights"] = (fqm.Lut6Weights if bits == 6 else fqm.Lut4Weights)(s["packed"], lut, rows, K)
    return s


def _prepare_route(c, g):
    T, E = c["T"], c["E"]
    liked = 0.5 * _randn(g, E)
    logits = _randn(g, T, E) + liked
    if c["closed"]:  # experts that some tokens may not take
        logits[torch.rand(T, E, generator=g, device=DEV) < c["closed"]] = -math.inf
    if c["padding"]:  # rows behind the batch's tokens
        logits[T - c["padding"]:] = -math.inf
    # the bias works against what is liked too much
    bias = -0.1 * liked + 0.02 * _randn(g, E) if c["bias"] else None
    return dict(logits=_rows_in(logits.to(_DT[c["x"]]), c["pad"]), bias=bias,
                **{n: c[n] for n in ("k", "score", "groups", "top_groups", "group_score", "renormalise", "scale")})


def _prepare_block(c, g):
    rows, cols, terms = c["rows"], c["cols"], c["terms"]
    # a residual stream: rows of different size, a few columns far above the rest
    size = torch.exp(0.5 * _randn(g, rows, 1))
    column = torch.where(torch.rand(cols, generator=g, device=DEV) < 0.002, 20.0, 1.0)
    x = _randn(g, rows, terms, cols) * (size * column)[:, None] if terms > 1 else _randn(g, rows, cols) * size * column
    dt = _DT[c["x"]]
    s = dict(x=_rows_in(x.to(dt), c["pad"]), post_weight=(0.3 * _randn(g, cols)).to(torch.bfloat16),
             weight=(0.2 * _randn(g, cols)).to(torch.bfloat16), gate=None, act=c["act"], out=c["out"],
             res=_rows_in((3 * _randn(g, rows, cols) * size * column).to(_DT[c["res"]]), c["pad"]))
    if c["gate"] != "no":
        shape = {"cols": (cols,), "rows": (rows, 1), "full": (rows, cols)}[c["gate"]]
        s["gate"] = (0.3 + 0.5 * _randn(g, *shape)).to(dt)
        if c["gate"] == "full":
            s["gate"] = _rows_in(s["gate"], c["pad"])
    return s


def prepare(case, seed):
    g = _gen(seed)
    s = {"linear": _prepare_linear, "route": _prepare_route, "block": _prepare_block}[case["op"]](case, g)
    s["op"] = case["op"]
    return s


# ---------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------
def _unpack(packed, cols, bits):
    b = packed[..., :cols * bits // 8]
    if bits == 4:
        return torch.stack([b & 15, b >> 4], -1).view(*b.shape[:-1], cols)
    b = b.reshape(*b.shape[:-1], cols // 4, 3).to(torch.int32)
    v = b[..., 0] | (b[..., 1] << 8) | (b[..., 2] << 16)
    return torch.stack([v & 63, (v >> 6) & 63, (v >> 12) & 63, v >> 18], -1).view(*v.shape[:-1], cols)


def _act(v, name):
    if name == "relu":
        return torch.where(v > 0, v, 0.0)
    if name == "silu":
        return v / (1 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * torch.erfc(v * -math.sqrt(0.5))
    if name == "gelu_tanh":
        return v / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _run_linear(s):
    if own:
        import dequant_matmul_amd as fqm
        return fqm.linear(s["weights"], s["x"], bias=s["bias"], act=None if s["act"] == "none" else s["act"],
                          gated=s["gated"], residual=s["res"], out_dtype=s["out"])
    W = torch.gather(s["lut"].float(), 1, _unpack(s["packed"], s["K"], s["bits"]).long())
    v = s["x"].float() @ W.t()
    if s["bias"] is not None:
        v = v + s["bias"].float()
    y = _act(v[:, :s["N"]], s["act"])
    if s["gated"]:
        y = y * v[:, s["N"]:]
    if s["res"] is not None:
        y = y + s["res"].float()
    return y.to(s["out"])


def _run_route(s):
    if own:
        import dequant_matmul_amd as fqm
        r = fqm.route(s["logits"], s["k"], score=s["score"], bias=s["bias"], groups=s["groups"], top_groups=s["top_groups"],
                      group_score=s["group_score"], renormalise=s["renormalise"], scale=s["scale"])
        return dict(expert=r.expert, weight=r.weight, offsets=r.offsets, src=r.src, dst=r.dst, row_scale=r.row_scale)
    k, groups, bias = s["k"], s["groups"], s["bias"]
    logits = s["logits"].double().clamp(max=LARGEST)
    T, E = logits.shape
    shut = torch.isnan(logits) | (logits == -math.inf)
    if s["score"] == "softmax":
        top = torch.where(shut, -math.inf, logits).amax(1, keepdim=True)
        score = torch.where(shut, 0.0, torch.exp(logits - top))
        score = score / score.sum(1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-logits))
    # without a bias the order is that of the logits
    key = torch.where(shut, -math.inf, logits if bias is None else score + bias.double())
    if groups > 1:
        if s["group_score"] == "top2":
            sums = torch.where(shut, -math.inf, score if bias is None else score + bias.double())
            two = torch.sort(sums.view(T, groups, -1), dim=2, descending=True)[0][:, :, :2]
            best = two[:, :, 0]
            if two.shape[2] > 1:
                best = best + torch.where(two[:, :, 1] == -math.inf, 0.0, two[:, :, 1])
        else:
            best = key.view(T, groups, -1).amax(2)
        order = torch.sort(best, dim=1, descending=True, stable=True)[1]
        kept = torch.zeros(T, groups, dtype=torch.bool, device=key.device)
        kept.scatter_(1, order[:, :s["top_groups"]], True)
        key = torch.where(kept[:, :, None], key.view(T, groups, -1), -math.inf).view(T, E)
    value, expert = (v[:, :k] for v in torch.sort(key, dim=1, descending=True, stable=True))
    live = value > -math.inf
    l = torch.gather(logits, 1, expert)
    if not s["renormalise"]:
        weight = torch.gather(score, 1, expert)
    elif s["score"] == "softmax":
        weight = torch.exp(l - torch.where(live, l, -math.inf).amax(1, keepdim=True))
    else:  # times a factor that keeps small scores away from zero
        low = l.clamp(max=0)
        weight = torch.exp(low - torch.where(live, low, -math.inf).amax(1, keepdim=True)) / (1 + torch.exp(-l.abs()))
    weight = torch.where(live, weight, 0.0)
    if s["renormalise"]:
        weight = weight / weight.sum(1, keepdim=True).clamp(min=1e-300)
    weight = (weight * s["scale"]).float()
    group = torch.where(live, expert, E).flatten()  # slots without an expert come last
    order = torch.argsort(group, stable=True)
    offsets = (group[None, :] < torch.arange(E + 1, device=group.device)[:, None]).sum(1)
    offsets[E] = T * k
    src = torch.where(live.flatten()[order], torch.div(order, k, rounding_mode="floor"), -1)
    i32 = torch.int32
    return dict(expert=torch.where(live, expert, -1).to(i32), weight=weight, offsets=offsets.to(i32), src=src.to(i32),
                dst=order.to(i32), row_scale=weight.flatten()[order])


def _run_block(s):
    x, res, gate = s["x"], s["res"], s["gate"]
    if own:
        import dequant_matmul_amd as fqm
        dt = torch.int8 if s["out"] == "i8" else _DT[s["out"]]
        y, scale, total = fqm.block_norm(x, res, post_weight=s["post_weight"], weight=s["weight"], gate=gate,
                                         gate_act=None if s["act"] == "none" else s["act"], scale=0.5, residual_scale=1.25,
                                         eps=EPS, weight_offset=1.0, out_dtype=dt)
        if s["out"] != "i8":
            return dict(y=y, total=total)
    else:
        u = x.float()
        if x.dim() == 3:
            u = u.sum(1)
        h = u * torch.rsqrt(u.square().mean(1, keepdim=True) + EPS) * (1 + s["post_weight"].float())
        if gate is not None:
            f = gate.float()
            h = h * (1 / (1 + torch.exp(-f)) if s["act"] == "sigmoid" else torch.tanh(f) if s["act"] == "tanh" else f)
        h = 1.25 * res.float() + 0.5 * h
        total = h.to(res.dtype)
        y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * (1 + s["weight"].float())
        if s["out"] != "i8":
            return dict(y=y.to(_DT[s["out"]]), total=total)
        scale = y.abs().amax(1) / 127
        y = torch.round(y / torch.where(scale > 0, scale, 1.0)[:, None])
    # what the 8 bits stand for, to be compared as such
    value = torch.empty(y.shape, dtype=torch.bfloat16, device=y.device)
    torch.mul(y, scale[:, None], out=value)
    return dict(y=value, scale=scale, total=total)


def run(state):
    return {"linear": _run_linear, "route": _run_route, "block": _run_block}[state["op"]](state)


# ---------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------
def _exact_linear(s):
    K, N, bits = s["K"], s["N"], s["bits"]
    rows, M = s["packed"].shape[0], s["x"].shape[0]
    place = torch.arange(K, device=DEV) * bits  # the bit at which a code starts
    v = torch.empty(M, rows, dtype=torch.float64, device=DEV)
    x = s["x"].double()
    for r in range(0, rows, 4096):
        raw = s["packed"][r:r + 4096].to(torch.int64)
        two = raw[:, place // 8] | (raw[:, (place // 8 + 1).clamp(max=raw.shape[1] - 1)] << 8)
        W = s["lut"][r:r + 4096].double().gather(1, (two >> (place % 8)) & (2 ** bits - 1))
        v[:, r:r + 4096] = torch.mm(x, W.t().contiguous())
    if s["bias"] is not None:
        v += s["bias"].double()
    g = v[:, :N]
    if s["act"] == "relu":
        g = g.clamp(min=0)
    elif s["act"] == "silu":
        g = g * torch.sigmoid(g)
    elif s["act"] == "gelu":
        g = g * torch.special.ndtr(g)
    elif s["act"] == "gelu_tanh":
        g = 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))
    y = g * v[:, N:] if s["gated"] else g
    return y + s["res"].double() if s["res"] is not None else y


def _exact_route(s):
    """On the host; the order of a row by (score, then index) as one lexicographic sort."""
    x = np.minimum(s["logits"].double().cpu().numpy(), LARGEST)
    T, E = x.shape
    k, G = s["k"], s["groups"]
    bias = None if s["bias"] is None else s["bias"].double().cpu().numpy()
    ok = x > -np.inf  # false for NaN as well
    z = np.where(ok, x, 0.0)
    if s["score"] == "softmax":
        top = np.where(ok, x, -np.inf).max(1, initial=-LARGEST, keepdims=True)
        p = np.exp(np.where(ok, x - top, -np.inf))
        total = p.sum(1, keepdims=True)
        p = p / np.where(total > 0, total, 1)
    else:
        with np.errstate(over="ignore"):
            p = 1 / (1 + np.exp(-z))
    choice = z if bias is None else p + bias
    if G > 1:
        part = np.where(ok, choice if s["group_score"] == "max" else p if bias is None else p + bias, -np.inf).reshape(T, G, E // G)
        ranked = -np.sort(-part, axis=2)
        best = ranked[:, :, 0].copy()
        if s["group_score"] == "top2" and E // G > 1:
            best += np.where(np.isinf(ranked[:, :, 1]), 0.0, ranked[:, :, 1])
        first = np.lexsort((np.broadcast_to(np.arange(G), (T, G)), -best), axis=1)
        rank = np.argsort(first, axis=1)
        ok = ok & np.repeat(rank < s["top_groups"], E // G, axis=1)
    seq = np.lexsort((np.broadcast_to(np.arange(E), (T, E)), np.where(ok, -choice, np.inf)), axis=1)[:, :k]
    live = np.take_along_axis(ok, seq, 1)
    if s["renormalise"]:
        c = np.take_along_axis(z, seq, 1)
        log = c if s["score"] == "softmax" else -np.logaddexp(0.0, -c)  # of the score, up to a constant
        log = np.where(live, log, -np.inf)
        top = log.max(1, keepdims=True)
        w = np.exp(log - np.where(np.isinf(top), 0.0, top))
        total = w.sum(1, keepdims=True)
        w = w / np.where(total > 0, total, 1)
    else:
        w = np.where(live, np.take_along_axis(p, seq, 1), 0.0)
    w = w * s["scale"]
    to = np.where(live, seq, E).ravel()
    dst = np.lexsort((np.arange(T * k), to))
    counts = np.bincount(to, minlength=E + 1)
    counts[E - 1] += counts[E]
    return dict(expert=np.where(live, seq, -1).astype(np.int32), weight=w,
                offsets=np.concatenate([[0], np.cumsum(counts[:E])]).astype(np.int32),
                src=np.where(live.ravel()[dst], dst // k, -1).astype(np.int32), dst=dst.astype(np.int32), row_scale=w.ravel()[dst])


def _exact_block(s):
    u = s["x"].double() if s["x"].dim() == 2 else s["x"].double().sum(1)
    cols = u.shape[1]

    def normed(v, weight):
        return v / torch.sqrt((v * v).sum(1, keepdim=True) / cols + EPS) * (weight.double() + 1)

    h = 0.5 * normed(u, s["post_weight"])
    if s["gate"] is not None:
        f = s["gate"].double()
        h = h * {"none": lambda t: t, "sigmoid": torch.sigmoid, "tanh": torch.tanh}[s["act"]](f)
    h = h + 1.25 * s["res"].double()
    y = normed(h, s["weight"])
    if s["out"] != "i8":
        return dict(y=y, total=h)
    scale = y.abs().max(1).values / 127
    return dict(y=torch.round(y / scale[:, None]) * scale[:, None], scale=scale, total=h)


def exact(case, seed):
    s = prepare(case, seed)
    return {"linear": _exact_linear, "route": _exact_route, "block": _exact_block}[case["op"]](s)
