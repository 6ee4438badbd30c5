"""fp64 definitions of the operators around the products, with error bounds.

Test infrastructure only: numpy, no code shared with the GPU path.  Each
function returns the values and, element by element, a bound on what an
evaluation in fp32 (unit roundoff U) may be off, from the number and size of
its roundings; bf16 outputs (8 significant bits) add half an ulp, at most 2^-8 of
the value.
"""
import numpy as np

U = 2.0 ** -24
BF16_HALF_ULP = 2.0 ** -8


def rounded(bound, value, out_dtype):
    """The bound after one rounding to the output's type."""
    b = bound * (1 + 2.0 ** -7)
    if out_dtype == "bf16":
        return b + BF16_HALF_ULP * np.abs(value) + 2.0 ** -134
    return b + 2 * U * np.abs(value) + 2.0 ** -149


def add_rms_norm(x, residual, weight, eps):
    """x [rows][terms][cols], residual [rows][cols] or None, weight [cols] or
    None (fp64) -> dict(total, total_bound, y, y_bound, scale, scale_bound).

    Roundings: one per addition, each at most U * sum|parts|; the sum of
    squares is a sum of positive terms, chains of at most 64 per thread and a
    tree above them (at most 90 roundings, halved by the root), then a
    division, a root, a reciprocal and two products."""
    parts = x if residual is None else np.concatenate([x, residual[:, None, :]], axis=1)
    h = parts.sum(axis=1)
    size = np.abs(parts).sum(axis=1)
    hb = (parts.shape[1] - 1) * U * size
    w = np.ones(h.shape[1]) if weight is None else weight
    ms = (h * h).mean(axis=1, keepdims=True) + eps
    r = 1.0 / np.sqrt(ms)
    # relative error of r: that of the root mean square, from h's own errors and the roundings
    rel = (hb * np.abs(h)).mean(axis=1, keepdims=True) / ms + 50 * U
    y = h * w * r
    yb = np.abs(w) * r * hb + (rel + 4 * U) * np.abs(y)
    scale = np.abs(y).max(axis=1) / 127
    sb = yb.max(axis=1) / 127 + 4 * U * scale
    return dict(total=h, total_bound=hb, y=y, y_bound=yb, scale=scale, scale_bound=sb)


def lora(A, B, scale, ranks, x, index, base):
    """A [count][rank][cols], B [count][rows][rank], x [M][cols], base [M][rows]
    or None (fp64) -> (y, bound).

    The products A x: cols terms in fp32; worst case one rounding a term, in
    chains no longer than cols / 8 + 64.  scale * A x is kept whole (three bf16
    parts, 24 bits, each product exact in fp32), then rank * 3 terms, scale and
    base are added."""
    M, rows = x.shape[0], B.shape[1]
    y = np.zeros((M, rows)) if base is None else base.astype(np.float64).copy()
    bound = 2 * U * np.abs(y)
    K = x.shape[1]
    for m in range(M):
        i = int(index[m])
        if not 0 <= i < A.shape[0]:
            continue
        r = min(max(int(ranks[i]), 0), A.shape[1]) if ranks is not None else A.shape[1]
        s = 1.0 if scale is None else float(scale[i])
        t = A[i, :r] @ x[m]
        tb = (K / 8 + 64) * U * (np.abs(A[i, :r]) @ np.abs(x[m]))
        Bi = B[i, :, :r]
        y[m] += s * (Bi @ t)
        bound[m] += abs(s) * (np.abs(Bi) @ (tb + (3 * r + 8) * U * np.abs(t)))
    return y, bound + 2 * U * np.abs(y)


def grouped(W, offsets, x, src, dst, row_scale, y_rows, fill):
    """W [experts][rows][cols], x [x_rows][cols] (already with its scales; fp64),
    -> (Y [y_rows][rows], bound); rows that nothing is stored to hold `fill`.

    Sums of cols products, exact ones, of centred independent terms: n fp32
    roundings of partial sums that stay within a few root-sum-squares S of
    the terms add up to about sqrt(n) U S; the bound takes 16 of that."""
    Y = np.full((y_rows, W.shape[1]), float(fill))
    bound = np.zeros_like(Y)
    K = W.shape[2]
    for e in range(W.shape[0]):
        for i in range(int(offsets[e]), int(offsets[e + 1])):
            xr = i if src is None else int(src[i])
            yr = i if dst is None else int(dst[i])
            if not 0 <= yr < y_rows:
                continue
            s = 1.0 if row_scale is None else float(row_scale[i])
            v = x[xr] if 0 <= xr < x.shape[0] else np.zeros(K)
            Y[yr] = s * (W[e] @ v)
            rms = np.sqrt((W[e] ** 2) @ (v ** 2))
            bound[yr] = abs(s) * 16 * np.sqrt(max(K, 1)) * U * rms + 4 * U * np.abs(Y[yr])
    return Y, bound
