"""fp64 definitions of what completes a block around the products (the product
with its epilogue, the routing to experts, the norms on both sides of a block),
with error bounds.

Test infrastructure only: numpy, no code shared with the GPU path.  Values come
with a bound, element by element, on what an evaluation in fp32 (unit roundoff U)
may be off, from the number and size of its roundings; `layer.rounded` adds the
rounding to the output's type.
"""
import math

import numpy as np

from .layer import U

_erfc = np.vectorize(math.erfc, otypes=[np.float64])
C = math.sqrt(2 / math.pi)


def act(v, name):
    """(value, bound on an fp32 evaluation at exactly v, the largest slope).

    A library exp or tanh is off by at most 2 ulp (4 U), a division or product by U;
    the argument z of the exponential carries a few roundings of its own, each of
    which the exponential turns into a relative error of U |z|."""
    v = np.asarray(v, dtype=np.float64)
    with np.errstate(over="ignore"):
        if name in (None, "none"):
            return v, 0 * v, 1.0
        if name == "relu":
            return np.maximum(v, 0), 0 * v, 1.0
        if name == "silu":
            y = v / (1 + np.exp(-v))
            return y, 10 * U * np.abs(y), 1.1
        if name == "gelu":  # erfc(z) falls as exp(-z^2), z = v / sqrt(2): two roundings of z weigh 2 z^2 = v^2 each
            y = 0.5 * v * _erfc(-v / math.sqrt(2))
            return y, (16 + 3 * v * v) * U * np.abs(y), 1.13
        if name == "gelu_tanh":
            z = 2 * C * (v + 0.044715 * v ** 3)
            y = v / (1 + np.exp(-z))
            return y, (10 + 6 * np.minimum(np.abs(z), 104)) * U * np.abs(y), 1.13
        if name == "sigmoid":
            y = 1 / (1 + np.exp(-v))
            return y, 10 * U * np.abs(y), 0.25
        if name == "tanh":
            return np.tanh(v), 4 * U * np.abs(np.tanh(v)), 1.0
    raise ValueError(name)


def _apply(name, v, b):
    """act of a value known to within b."""
    y, e, slope = act(v, name)
    return y, e + slope * b


def linear(W, x, bias, name, gated, residual):
    """W [rows][cols], x [M][cols], bias [rows] or None, residual [M][n] or None (fp64) -> (y, bound).

    Sums of cols exact products of centred independent terms: n fp32 roundings of
    partial sums that stay within a few root-sum-squares S of the terms add up to
    about sqrt(n) U S; the bound takes 16 of that."""
    K = W.shape[1]
    v = x @ W.T
    vb = 16 * math.sqrt(max(K, 1)) * U * np.sqrt((x * x) @ (W * W).T)
    if bias is not None:
        v = v + bias
        vb = vb + U * np.abs(v)
    n = W.shape[0] // 2 if gated else W.shape[0]
    y, b = _apply(name, v[:, :n], vb[:, :n])
    if gated:
        up, ub = v[:, n:], vb[:, n:]
        y, b = y * up, np.abs(up) * b + np.abs(y) * ub + b * ub + U * np.abs(y * up)
    if residual is not None:
        y = y + residual
        b = b + U * np.abs(y)
    return y, b


def route(logits, k, score, bias, groups, top_groups, group_score, renormalise, scale):
    """logits [T][E], bias [E] or None (fp64; sorting by pairs, token by token) -> dict(expert, weight, bound,
    offsets, src, dst)."""
    T, E = logits.shape
    largest = float(np.finfo(np.float32).max)
    expert = np.full((T, k), -1)
    weight, bound = np.zeros((T, k)), np.zeros((T, k))
    per = E // groups
    for t in range(T):
        l = [min(float(v), largest) if v > -math.inf else None for v in logits[t]]  # NaN: not greater
        if bias is not None:
            l = [v if b > -math.inf else None for v, b in zip(l, bias)]
        live = [e for e in range(E) if l[e] is not None]
        if not live:
            continue
        if score == "softmax":
            top = max(l[e] for e in live)
            s = {e: math.exp(l[e] - top) for e in live}
            z = math.fsum(s.values())
            s = {e: v / z for e, v in s.items()}
        else:
            s = {e: 1 / (1 + math.exp(-l[e])) if l[e] > -700 else 0.0 for e in live}
        c = {e: s[e] + float(bias[e]) if bias is not None else l[e] for e in live}
        if groups > 1:
            part = c if group_score == "max" or bias is not None else s
            best = []
            for g in range(groups):
                two = sorted((part[e] for e in range(g * per, (g + 1) * per) if e in part), reverse=True)[:2]
                best.append(-math.inf if not two else two[0] if group_score == "max" else sum(two))
            kept = sorted(range(groups), key=lambda g: (-best[g], g))[:top_groups]
            c = {e: v for e, v in c.items() if e // per in kept}
        chosen = sorted(c, key=lambda e: (-c[e], e))[:k]
        if not chosen:
            continue
        if renormalise:
            log = [l[e] if score == "softmax" else min(l[e], 0) - math.log1p(math.exp(-abs(l[e]))) for e in chosen]
            m = max(log)
            w = [math.exp(v - m) for v in log]
            d = [abs(v - m) for v in log]
            total = math.fsum(w)
            w = [v / total for v in w]
        else:
            w, d = [s[e] for e in chosen], [0.0] * len(chosen)
        for j, e in enumerate(chosen):
            expert[t, j], weight[t, j] = e, w[j] * scale
            # the exponent's argument is a rounded difference; then an exponential, sums over k, divisions
            bound[t, j] = abs(weight[t, j]) * (2 * min(d[j], 104) + 16 + k) * U + 2.0 ** -126 * abs(scale)
    slots = sorted(range(T * k), key=lambda i: (expert.flat[i] if expert.flat[i] >= 0 else E, i))
    counts = [int((expert == e).sum()) for e in range(E)]
    offsets = np.concatenate([[0], np.cumsum(counts)])
    offsets[E] = T * k  # slots without an expert are rows of the last one
    src = [i // k if expert.flat[i] >= 0 else -1 for i in slots]
    return dict(expert=expert, weight=weight, bound=bound, offsets=offsets, src=np.array(src, dtype=int),
                dst=np.array(slots, dtype=int))


def block_norm(x, residual, post_weight, weight, gate, gate_act, scale, residual_scale, eps, offset, post):
    """x [rows][terms][cols], residual [rows][cols] or None, weights [cols] or None, gate broadcast to [rows][cols]
    or None (fp64) -> dict(total, total_bound, y, y_bound, scale, scale_bound).

    Roundings as in layer.add_rms_norm: a sum of squares of positive terms, at most 90 of them halved by the root,
    a division, a root, a reciprocal."""
    u = x.sum(axis=1)
    ub = (x.shape[1] - 1) * U * np.abs(x).sum(axis=1)
    v, vb = u, ub
    if post:
        w = 1.0 if post_weight is None else post_weight + offset
        ms = (u * u).mean(axis=1, keepdims=True) + eps
        rel = (ub * np.abs(u)).mean(axis=1, keepdims=True) / ms + 50 * U
        v = u * w / np.sqrt(ms)
        vb = np.abs(w) / np.sqrt(ms) * ub + (rel + 6 * U) * np.abs(v)
    if gate is not None:
        f, fb, _ = act(gate, gate_act)
        v, vb = v * f, np.abs(f) * vb + np.abs(v) * fb + fb * vb + U * np.abs(v * f)
    h = scale * v
    hb = abs(scale) * vb + 3 * U * np.abs(h)
    if residual is not None:
        hb = hb + 2 * U * np.abs(residual_scale * residual) + U * np.abs(h)
        h = h + residual_scale * residual
    w = 1.0 if weight is None else weight + offset
    ms = (h * h).mean(axis=1, keepdims=True) + eps
    rel = (hb * np.abs(h)).mean(axis=1, keepdims=True) / ms + 50 * U
    y = h * w / np.sqrt(ms)
    yb = np.abs(w) / np.sqrt(ms) * hb + (rel + 6 * U) * np.abs(y)
    s = np.abs(y).max(axis=1) / 127
    return dict(total=h, total_bound=hb, y=y, y_bound=yb, scale=s, scale_bound=yb.max(axis=1) / 127 + 4 * U * s)
