"""The residual norm against its fp64 definition: types, terms, strides, odd
widths, the 8-bit codes, rows of zeros, NaN and infinities."""
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


def case(rows, cols, terms, x, res, pad=0, start=0, seed=0):
    rng = np.random.default_rng([rows, cols, terms, seed])
    size = np.exp(rng.standard_normal((rows,) + (1,) * (2 if terms > 1 else 1)))
    xs = rows_at(rng, (rows, terms, cols) if terms > 1 else (rows, cols), x, pad, start, size)
    rs = rows_at(rng, (rows, cols), res, pad, start, 3 * size.reshape(rows, 1)) if res else None
    w = torch.from_numpy(1 + 0.2 * rng.standard_normal(cols)).float().to(DEV)
    return xs, rs, w


def check(xs, rs, w, eps, out, got, total_dtype):
    o = oracle.layer.add_rms_norm(to_f64(xs) if xs.dim() == 3 else to_f64(xs)[:, None], None if rs is None else to_f64(rs),
                                  None if w is None else to_f64(w), eps)
    if got.total is not None:
        lim = oracle.layer.rounded(o["total_bound"], o["total"], total_dtype)
        assert (np.abs(to_f64(got.total) - o["total"]) <= lim).all()
    if out != "i8":
        lim = oracle.layer.rounded(o["y_bound"], o["y"], out)
        assert (np.abs(to_f64(got.y) - o["y"]) <= lim).all()
        return
    sc, q = to_f64(got.scale), to_f64(got.y)
    assert (np.abs(sc - o["scale"]) <= o["scale_bound"] + 2.0 ** -149).all()
    assert np.abs(q).max(initial=0) <= 127
    live = o["scale"] > 0
    s = np.where(live, o["scale"], 1)[:, None]
    off = np.abs(q - o["y"] / s) - 0.5
    lim = o["y_bound"] / s + 127 * (o["scale_bound"][:, None] / s + 8 * oracle.layer.U)
    assert (off <= lim)[live].all()
    assert (q[~live] == 0).all()


@pytest.mark.parametrize("out", ["bf16", "f32", "i8"])
@pytest.mark.parametrize("rows,cols,terms,x,res,pad,start", [
    (1, 5120, 1, "bf16", "bf16", 0, 0),
    (3, 17408, 1, "bf16", "f32", 0, 0),
    (2, 32768, 3, "f32", "f32", 0, 0),
    (5, 24573, 2, "f32", "bf16", 1, 1),
    (9, 1087, 1, "f32", "f32", 9, 0),
    (7, 1000, 5, "bf16", "bf16", 3, 3),
    (130, 64, 8, "bf16", None, 0, 0),
    (11, 1, 1, "bf16", "bf16", 0, 0),
    (6, 7, 2, "f32", None, 2, 1),
    (4, 513, 64, "bf16", "f32", 0, 0),
    (5, 8192, 1, "bf16", None, 8, 0),
    (1, 9, 1, "f32", "bf16", 0, 0),
])
def test_against_definition(rows, cols, terms, x, res, pad, start, out):
    print(f"add_rms_norm {rows}x{terms}x{cols} {x} {res} {out} pad {pad} start {start}", flush=True)
    xs, rs, w = case(rows, cols, terms, x, res, pad, start)
    w = w.to(torch.bfloat16 if rows % 2 else torch.float32)
    buf, y = guarded((rows, cols), T[out], fill=-123.0)
    got = fqm.add_rms_norm(xs, w, eps=1e-5, residual=rs, y=y)
    torch.cuda.synchronize()
    assert canaries_intact(buf, fill=-123.0)
    assert (got.total is None) == (res is None and terms == 1)
    assert (got.scale is None) == (out != "i8")
    check(xs, rs, w, float(np.float32(1e-5)), out, got, res or x)


def test_no_weight_no_total_and_eps():
    xs, rs, _ = case(4, 640, 1, "f32", "f32")
    got = fqm.add_rms_norm(xs * 1e-4, None, eps=0.5, residual=rs * 1e-4, out_dtype=torch.float32, keep_total=False)
    assert got.total is None
    check(xs * 1e-4, rs * 1e-4, None, 0.5, "f32", got, "f32")
    got = fqm.add_rms_norm(xs, None, keep_total=True)
    assert torch.equal(got.total, xs)


def test_total_in_place_of_the_residual_and_strided_outputs():
    xs, rs, w = case(37, 1000, 2, "bf16", "bf16", pad=5)
    want = fqm.add_rms_norm(xs, w, residual=rs)
    wide = torch.full((37, 1013), 7.0, dtype=torch.bfloat16, device=DEV)
    got = fqm.add_rms_norm(xs, w, residual=rs, total=rs, y=wide[:, 4:1004])
    assert got.total.data_ptr() == rs.data_ptr()
    assert torch.equal(got.total, want.total) and torch.equal(got.y, want.y)
    assert (wide[:, :4] == 7).all() and (wide[:, 1004:] == 7).all()


def test_term_and_row_strides_may_lie_either_way():
    """Terms outermost, as Y of one product per expert: [terms][rows][cols]."""
    rng = np.random.default_rng(3)
    x = rows_at(rng, (3, 10, 264), "bf16").transpose(0, 1)
    assert torch.equal(fqm.add_rms_norm(x).y, fqm.add_rms_norm(x.contiguous()).y)


def test_results_do_not_depend_on_the_other_rows():
    xs, rs, w = case(300, 1160, 1, "bf16", "bf16")
    a = fqm.add_rms_norm(xs, w, residual=rs, out_dtype=torch.float32)
    b = fqm.add_rms_norm(xs[77:78], w, residual=rs[77:78], out_dtype=torch.float32)
    assert torch.equal(a.y[77:78], b.y)


def test_rows_of_zeros_tiny_rows_and_what_is_not_finite():
    x = torch.zeros(8, 200, device=DEV)
    x[1] = 1e-40
    x[2, 3] = float("nan")
    x[3, 3] = float("inf")
    x[4] = 1e-35
    x[4, 1:] = 0
    x[5] = 1.0
    x[6, 5] = -2e-42  # a row of one denormal
    x[7] = -3.0
    got = fqm.add_rms_norm(x, out_dtype=torch.float32)
    want = x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6)
    assert torch.equal(torch.isnan(got.y), torch.isnan(want))
    assert (got.y[0] == 0).all()
    q = fqm.add_rms_norm(x, out_dtype=torch.int8)
    assert q.scale[0] == 0 and (q.y[0] == 0).all()
    assert not torch.isfinite(q.scale[2]) and (q.y[2] == 0).all()
    assert not torch.isfinite(q.scale[3]) and (q.y[3] == 0).all()
    assert q.y[4, 0] == 127 and (q.y[4, 1:] == 0).all()
    assert q.y[6, 5] == -127 and (q.y[1] == 127).all()
    assert (q.y[5] == 127).all() and (q.y[7] == -127).all()
    # a weight's NaN reaches the scale as well
    w = torch.ones(200, device=DEV)
    w[9] = float("nan")
    q = fqm.add_rms_norm(x[5:6], w, out_dtype=torch.int8)
    assert torch.isnan(q.scale).all() and (q.y == 0).all()


def test_empty():
    for rows, cols in ((0, 128), (3, 0)):
        x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
        got = fqm.add_rms_norm(x, out_dtype=torch.int8, scale=torch.full((rows,), 9.0, device=DEV))
        assert got.y.shape == (rows, cols) and (got.scale == 0).all()


def test_another_stream_and_graph_replays():
    xs, rs, w = case(16, 5120, 1, "bf16", "bf16")
    want = fqm.add_rms_norm(xs, w, residual=rs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, total = torch.empty_like(want.y), torch.empty_like(want.total)
    fqm.add_rms_norm(xs, w, residual=rs, y=y, total=total, stream=side)
    side.synchronize()
    assert torch.equal(y, want.y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fqm.add_rms_norm(xs, w, residual=rs, y=y, total=total)
    for k in range(3):
        xs.copy_(torch.roll(xs, 1, 0))
        want = fqm.add_rms_norm(xs, w, residual=rs)
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want.y) and torch.equal(total, want.total)


@pytest.mark.parametrize("rows,cols,out", [(2048, 5120, "bf16"), (2500, 1000, "i8"), (2049, 17416, "f32"), (4097, 128, "bf16"),
                                           (3001, 100, "i8"), (70, 129, "f32"), (33, 256, "i8"), (5, 257, "bf16"), (2100, 8, "f32")])
def test_many_rows_and_rows_of_part_of_a_wave(rows, cols, out):
    """The forms with several chunks a thread and several rows a wave, a sample of the rows checked."""
    print(f"add_rms_norm {rows}x{cols} {out}", flush=True)
    xs, rs, w = case(rows, cols, 1, "bf16", "f32")
    buf, y = guarded((rows, cols), T[out], fill=-123.0)
    got = fqm.add_rms_norm(xs, w, eps=1e-5, residual=rs, y=y)
    torch.cuda.synchronize()
    assert canaries_intact(buf, fill=-123.0)
    pick = sorted({r for r in (0, 1, 2, 3, 15, rows // 2, rows // 3, rows - 17, rows - 2, rows - 1) if 0 <= r < rows})
    part = fqm.NormOut(got.y[pick], None if got.scale is None else got.scale[pick], got.total[pick])
    check(xs[pick], rs[pick], w, float(np.float32(1e-5)), out, part, "f32")
