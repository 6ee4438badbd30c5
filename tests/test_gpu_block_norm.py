"""The norms on both sides of a block against their fp64 definition: types, terms, gates, strides, odd widths, the
8-bit codes, rows of zeros, NaN and infinities."""
import numpy as np
import pytest
import torch

import dequant_matmul_amd as fqm
import oracle
from gpu_common import DEV, canaries_intact, guarded, to_f64

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f32": torch.float32, "i8": torch.int8}


def rows_at(rng, shape, dtype, pad=0, start=0, size=1.0):
    """Random rows inside wider ones, their first value `start` values in."""
    v = rng.standard_normal(shape) * size
    wide = torch.zeros(*shape[:-1], shape[-1] + pad + start, dtype=T[dtype], device=DEV)
    view = wide[..., start:start + shape[-1]]
    view.copy_(torch.from_numpy(v))
    return view


def case(rows, cols, terms, x, res, gate, pad=0, start=0, seed=0):
    rng = np.random.default_rng([rows, cols, terms, seed])
    size = np.exp(rng.standard_normal((rows,) + (1,) * (2 if terms > 1 else 1)))
    c = dict(x=rows_at(rng, (rows, terms, cols) if terms > 1 else (rows, cols), x, pad, start, size),
             residual=rows_at(rng, (rows, cols), res, pad, start, 3 * size.reshape(rows, 1)) if res else None,
             post_weight=torch.from_numpy(0.3 * rng.standard_normal(cols)).to(DEV, T["f32" if rows % 2 else "bf16"]),
             weight=torch.from_numpy(0.2 * rng.standard_normal(cols)).to(DEV, T["bf16" if rows % 2 else "f32"]))
    if gate:
        kind, dt = gate.split("-")
        shape = {"cols": (cols,), "rows": (rows, 1), "full": (rows, cols)}[kind]
        c["gate"] = (rows_at(rng, shape, dt, pad, start) if kind == "full" else torch.from_numpy(rng.standard_normal(shape)).to(DEV, T[dt]))
    return c


def check(c, out, got, total_dtype, gate_act=None, scale=1.0, residual_scale=1.0, eps=1e-6, weight_offset=0.0, post=True, pick=None):
    f = {n: None if t is None else to_f64(t) for n, t in c.items()}
    x = f["x"] if f["x"].ndim == 3 else f["x"][:, None]
    g = f.get("gate")
    g = None if g is None else np.broadcast_to(g, (x.shape[0], x.shape[2]))
    r, y, sc, total = f["residual"], got.y, got.scale, got.total
    if pick is not None:
        x, g, r = x[pick], None if g is None else g[pick], None if r is None else r[pick]
        y, sc, total = (None if t is None else t[pick] for t in (y, sc, total))
    f32 = lambda v: float(np.float32(v))  # noqa: E731
    o = oracle.block.block_norm(x, r, f["post_weight"], f["weight"], g, gate_act, f32(scale), f32(residual_scale), f32(eps),
                                f32(weight_offset), post)
    if total is not None:
        lim = oracle.layer.rounded(o["total_bound"], o["total"], total_dtype)
        assert (np.abs(to_f64(total) - o["total"]) <= lim).all()
    if y is None:
        return
    if out != "i8":
        lim = oracle.layer.rounded(o["y_bound"], o["y"], out)
        assert (np.abs(to_f64(y) - o["y"]) <= lim).all()
        return
    s, q = to_f64(sc), to_f64(y)
    assert (np.abs(s - o["scale"]) <= o["scale_bound"] + 2.0 ** -149).all()
    assert np.abs(q).max(initial=0) <= 127
    live = o["scale"] > 0
    s = np.where(live, o["scale"], 1)[:, None]
    off = np.abs(q - o["y"] / s) - 0.5
    lim = o["y_bound"] / s + 127 * (o["scale_bound"][:, None] / s + 8 * oracle.layer.U)
    assert (off <= lim)[live].all()
    assert (q[~live] == 0).all()


@pytest.mark.parametrize("out", ["bf16", "f32", "i8"])
@pytest.mark.parametrize("rows,cols,terms,x,res,gate,act,pad,start", [
    (1, 5120, 1, "bf16", "bf16", None, None, 0, 0),
    (3, 17408, 1, "bf16", "f32", "cols-bf16", "tanh", 0, 0),
    (2, 32768, 3, "f32", "f32", "full-f32", "sigmoid", 0, 0),
    (5, 24573, 2, "f32", "bf16", "rows-f32", None, 1, 1),
    (9, 1087, 1, "f32", "f32", "full-f32", "tanh", 9, 0),
    (7, 1000, 5, "bf16", "bf16", "full-bf16", "silu", 3, 3),
    (130, 64, 8, "bf16", None, "rows-bf16", "sigmoid", 0, 0),
    (11, 1, 1, "bf16", "bf16", "cols-f32", None, 0, 0),
    (6, 7, 2, "f32", None, "full-bf16", "gelu", 2, 1),
    (4, 513, 64, "bf16", "f32", "cols-f32", "gelu_tanh", 0, 0),
    (5, 8192, 1, "bf16", None, None, None, 8, 0),
    (1, 9, 1, "f32", "bf16", "rows-bf16", "relu", 0, 0),
    (4, 10000, 1, "bf16", "bf16", "full-bf16", None, 0, 0),
])
def test_against_definition(rows, cols, terms, x, res, gate, act, pad, start, out):
    print(f"block_norm {rows}x{terms}x{cols} {x} {res} {gate} {act} {out} pad {pad} start {start}", flush=True)
    c = case(rows, cols, terms, x, res, gate, pad, start)
    kw = dict(gate_act=act, scale=0.75, residual_scale=1.25, eps=1e-5, weight_offset=1.0)
    buf, y = guarded((rows, cols), T[out], fill=-123.0)
    got = fqm.block_norm(**c, y=y, **kw)
    torch.cuda.synchronize()
    assert canaries_intact(buf, fill=-123.0) and (got.scale is None) == (out != "i8")
    check(c, out, got, res or x, **kw)


@pytest.mark.parametrize("post", [True, False])
def test_parts_left_out(post):
    c = case(6, 640, 2, "f32", "f32", None)
    c["post_weight"] = c["weight"] = None
    got = fqm.block_norm(**c, post=post, out_dtype=torch.float32)
    check(c, "f32", got, "f32", post=post)
    only = fqm.block_norm(**c, post=post, out_dtype=None)  # no second norm
    assert only.y is None and only.scale is None and torch.equal(only.total, got.total)
    none = fqm.block_norm(**c, post=post, out_dtype=torch.float32, keep_total=False)
    assert none.total is None and torch.equal(none.y, got.y)
    if not post:  # then it is the residual norm
        want = fqm.add_rms_norm(c["x"], residual=c["residual"], out_dtype=torch.float32)
        assert torch.equal(got.total, want.total)
        assert ((got.y - want.y).abs() <= 4 * 2.0 ** -24 * want.y.abs()).all()


def test_total_in_place_of_the_residual_and_strided_outputs():
    c = case(37, 1000, 2, "bf16", "bf16", "full-bf16", pad=5)
    want = fqm.block_norm(**c)
    wide = torch.full((37, 1013), 7.0, dtype=torch.bfloat16, device=DEV)
    got = fqm.block_norm(**c, total=c["residual"], y=wide[:, 4:1004])
    assert got.total.data_ptr() == c["residual"].data_ptr()
    assert torch.equal(got.total, want.total) and torch.equal(got.y, want.y)
    assert (wide[:, :4] == 7).all() and (wide[:, 1004:] == 7).all()


def test_gates_of_every_stride():
    c = case(10, 264, 3, "bf16", "bf16", None)
    g = torch.randn(10, 300, device=DEV)
    full = g[:, 7:271]
    want = fqm.block_norm(**c, gate=full.contiguous())
    assert torch.equal(fqm.block_norm(**c, gate=full).y, want.y)
    one = fqm.block_norm(**c, gate=g[2, 7:271].contiguous())
    assert torch.equal(fqm.block_norm(**c, gate=g[2, 7:271][None].expand(10, 264)).y, one.y)
    rows = fqm.block_norm(**c, gate=g[:, 5:6].contiguous())
    assert torch.equal(fqm.block_norm(**c, gate=g[:, 5:6]).y, rows.y)
    assert torch.equal(fqm.block_norm(**c, gate=g[:, 5:6].expand(10, 264).contiguous()).y, rows.y)
    x = c["x"].transpose(0, 1).contiguous().transpose(0, 1)  # terms outermost
    assert torch.equal(fqm.block_norm(**dict(c, x=x)).y, fqm.block_norm(**c).y)


def test_results_do_not_depend_on_the_other_rows():
    c = case(300, 1160, 1, "bf16", "bf16", "full-f32")
    a = fqm.block_norm(**c, out_dtype=torch.float32)
    b = fqm.block_norm(**{n: t[77:78] if t.dim() == 2 else t for n, t in c.items()}, out_dtype=torch.float32)
    assert torch.equal(a.y[77:78], b.y) and torch.equal(a.total[77:78], b.total)


@pytest.mark.parametrize("cols", [2048, 2051, 5120, 8192])
@pytest.mark.parametrize("x,res", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("gate", [None, "rows-bf16", "cols-bf16", "full-bf16"])
def test_many_rows_have_the_bits_of_few(cols, x, res, gate):
    c = case(1026, cols, 1, x, res, gate, pad=5)
    c["weight"] = c["weight"].to(torch.bfloat16)
    pick = [0, 5, 1025]
    for out in (torch.float32, torch.int8):
        a = fqm.block_norm(**c, out_dtype=out, gate_act="sigmoid" if gate else None)
        few = {n: t[pick] if t is not None and t.dim() == 2 and t.shape[0] == 1026 else t for n, t in c.items()}
        b = fqm.block_norm(**few, out_dtype=out, gate_act="sigmoid" if gate else None)
        assert torch.equal(a.y[pick], b.y) and torch.equal(a.total[pick], b.total)
        if out == torch.int8:
            assert torch.equal(a.scale[pick], b.scale)
    f = fqm.block_norm(**few, out_dtype=torch.float32, gate_act="sigmoid" if gate else None)
    check(few, "f32", f, res, gate_act="sigmoid" if gate else None)


@pytest.mark.parametrize("cols", [8192, 8193, 8200, 16384, 16391, 32768])
@pytest.mark.parametrize("terms,gate", [(1, None), (3, "full-f32"), (9, "cols-bf16")])
@pytest.mark.parametrize("out", ["f32", "i8"])
def test_wide_rows(cols, terms, gate, out):
    c = case(3, cols, terms, "bf16", "f32", gate)
    check(c, out, fqm.block_norm(**c, out_dtype=T[out]), "f32")


def test_total_in_place_of_the_residual_at_odd_widths():
    """A row's last chunk starts in its neighbour's columns: their total may be stored by then."""
    for cols in (9, 263, 1087, 2051, 8197):
        c = case(1030, cols, 1, "bf16", "bf16", None)
        c["post_weight"] = None
        want = fqm.block_norm(**c, post=False)
        r = c["residual"].clone()
        got = fqm.block_norm(**dict(c, residual=r), post=False, total=r)
        assert torch.equal(got.y, want.y) and torch.equal(r, want.total)


def test_rows_of_zeros_and_what_is_not_finite():
    x = torch.randn(8, 200, device=DEV)
    r = torch.randn(8, 200, device=DEV)
    x[0] = r[0] = 0
    x[1] = 0               # a block that gives nothing
    x[2, 3] = float("nan")
    x[3, 3] = float("inf")
    r[4, 5] = float("inf")
    x[5] = 1e-40
    x[6], r[6] = 1e30, 0   # its square is infinite: the norm is zeros
    got = fqm.block_norm(x, r, out_dtype=torch.float32)
    assert (got.y[0] == 0).all() and torch.equal(got.total[1], r[1])
    assert torch.isnan(got.y[2]).all() and torch.isnan(got.y[3, 3]) and torch.isnan(got.y[4, 5])
    assert torch.isfinite(got.y[[0, 1, 5, 6, 7]]).all() and (got.total[6] == 0).all()
    q = fqm.block_norm(x, r, out_dtype=torch.int8)
    assert q.scale[0] == 0 and (q.y[0] == 0).all() and q.scale[6] == 0 and (q.y[6] == 0).all()
    for row in (2, 3, 4):
        assert not torch.isfinite(q.scale[row]) and (q.y[row] == 0).all()
    zero = fqm.block_norm(torch.zeros(3, 50, device=DEV), eps=0.0, post=False, out_dtype=torch.int8)
    assert (zero.scale == 0).all() and (zero.y == 0).all()


def test_empty():
    for rows, cols in ((0, 128), (3, 0)):
        x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
        got = fqm.block_norm(x, out_dtype=torch.int8, y_scale=torch.full((rows,), 9.0, device=DEV))
        assert got.y.shape == (rows, cols) and (got.scale == 0).all()


def test_another_stream_and_graph_replays():
    c = case(16, 5120, 6, "bf16", "bf16", "rows-bf16")
    kw = dict(gate_act="sigmoid", out_dtype=torch.int8)
    want = fqm.block_norm(**c, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fqm.block_norm(**c, stream=side, **kw)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    y, total, sc = torch.empty_like(want.y), torch.empty_like(want.total), torch.empty_like(want.scale)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fqm.block_norm(**c, y=y, total=total, y_scale=sc, **kw)
    for _ in range(3):
        c["x"].copy_(torch.roll(c["x"], 1, 0))
        want = fqm.block_norm(**c, **kw)
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want.y) and torch.equal(total, want.total) and torch.equal(sc, want.scale)


@pytest.mark.parametrize("rows,cols,x,out", [(2048, 5120, "bf16", "bf16"), (2500, 1000, "f32", "i8"), (2049, 17416, "bf16", "f32"),
                                             (4097, 128, "bf16", "bf16"), (3001, 100, "f32", "i8"), (70, 129, "bf16", "f32"),
                                             (33, 256, "bf16", "i8"), (5, 257, "f32", "bf16"), (2100, 8, "bf16", "f32"),
                                             (8200, 1024, "bf16", "bf16"), (2111, 9000, "f32", "f32"), (2050, 26000, "bf16", "bf16")])
def test_many_rows_and_rows_of_part_of_a_wave(rows, cols, x, out):
    """A sample of the rows checked."""
    print(f"block_norm {rows}x{cols} {x} {out}", flush=True)
    c = case(rows, cols, 1, x, "f32" if rows % 2 else "bf16", "rows-f32")
    buf, y = guarded((rows, cols), T[out], fill=-123.0)
    got = fqm.block_norm(**c, y=y, eps=1e-5)
    torch.cuda.synchronize()
    assert canaries_intact(buf, fill=-123.0)
    pick = sorted({r for r in (0, 1, 2, 3, 15, rows // 2, rows // 3, rows - 17, rows - 2, rows - 1) if 0 <= r < rows})
    check(c, out, got, "f32" if rows % 2 else "bf16", eps=1e-5, pick=pick)


def test_refusals_of_the_binding():
    x = torch.zeros(4, 24, device=DEV)
    for kw, match in ((dict(residual=torch.zeros(4, 23, device=DEV)), "residual"), (dict(weight=torch.zeros(23, device=DEV)), "weight"),
                      (dict(post_weight=torch.zeros(24, device=DEV), post=False), "post_weight"), (dict(gate_act="tanh"), "without a gate"),
                      (dict(gate=torch.zeros(4, device=DEV)), "gate has shape"), (dict(gate=torch.zeros(1, 24, device=DEV)), "gate has shape"),
                      (dict(gate=torch.zeros(24, 4, device=DEV).t()), "dense"), (dict(gate=torch.zeros(24, device=DEV), gate_act="max"), "gate_act must be"),
                      (dict(out_dtype=torch.float16), "out_dtype"), (dict(out_dtype=None, keep_total=False), "nothing to compute"),
                      (dict(total=torch.zeros(4, 24, dtype=torch.bfloat16, device=DEV)), "total"), (dict(gate=torch.zeros(24)), "GPU tensors")):
        with pytest.raises(ValueError, match=match):
            fqm.block_norm(x, **kw)
    with pytest.raises(ValueError, match="overlapping"):
        fqm.block_norm(torch.zeros(1, 24, device=DEV).expand(4, 24))
    with pytest.raises(ValueError, match="terms"):
        fqm.block_norm(torch.zeros(4, 65, 8, device=DEV))
