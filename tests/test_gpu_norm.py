"""ar_reduce_norm and ar_norm_bwd on the GPU against the plain 64-bit forms.

Tolerances, from the arithmetic alone (u = 2^-24, binary32's unit roundoff):
the rank sum is compared bit for bit (same order).  The sum of squares of a
row adds at most 64 terms in a lane, 6 wave steps and 16 waves, then a
division, a square root, a reciprocal and two products: each result is
within 100 u of the exact one, relatively, besides the error of h itself,
(P + 1) u sum|x|.  bf16 results add 2^-8 relatively.
"""
import numpy as np
import pytest
import torch

import block_ref as ref
import tensor_all_reduce_amd as tar
from gpu_util import DEV, note, up16, down16

pytestmark = pytest.mark.gpu

U = ref.U32


def rows16(a) -> torch.Tensor:
    """binary32 matrix of bf16 values -> device bf16 matrix."""
    return up16(ref.bf16_bits(a)).view(torch.bfloat16).reshape(a.shape)


def vals(t) -> np.ndarray:
    return ref.bf16_val(down16(t).reshape(-1)).reshape(t.shape)


def out16(rows, cols):
    """A bf16 matrix with a sentinel row past its end: (whole, matrix)."""
    buf = torch.full(((rows + 1) * cols + 8,), 0x5A5A, dtype=torch.int16, device=DEV)
    return buf, buf[:rows * cols].view(torch.bfloat16).reshape(rows, cols)


def untouched(buf, n):
    return bool((buf[n:] == 0x5A5A).all())


def make(rows, cols, P, seed, spread=1.0):
    g = np.random.default_rng([seed, rows, cols, P])
    xs = [ref.as_bf16(g.standard_normal((rows, cols)) * spread) for _ in range(P)]
    res = ref.as_bf16(g.standard_normal((rows, cols)) * np.exp(g.standard_normal(cols)))
    w = ref.as_bf16(1 + 0.3 * g.standard_normal(cols))
    return xs, res, w


def y_bound(xs, res, h, w, eps):
    """|y - exact| of a binary32 y: the norm's own steps plus h's rounding."""
    mag = sum(np.abs(x.astype(np.float64)) for x in xs) + (0 if res is None else np.abs(res.astype(np.float64)))
    y = np.abs(ref.norm(h, w, eps))
    r = 1 / np.sqrt((h.astype(np.float64) ** 2).mean(1, keepdims=True) + eps)
    aw = 1.0 if w is None else np.abs(w.astype(np.float64))
    n = len(xs) + 1
    # h enters twice: its own element, and through the row's mean square
    row = n * U * np.sqrt((mag ** 2).mean(1, keepdims=True)) * r
    return 100 * U * y + n * U * mag * r * aw + row * y


def check_codes(codes, scales, y, tol, what):
    """Codes and scales of a result known within tol: each scale is that of
    the block's largest magnitude, and no element is further from its code's
    value than half a step."""
    s = ref.scale_val(scales)
    amax = ref.block_amax(y, 1)
    slack = ref.block_amax(tol, 1)
    if scales.dtype == np.uint8:
        assert np.all(amax - slack <= 448 * s * (1 + 4 * U)), what
        assert np.all((amax + slack > 224 * s * (1 - 4 * U)) | (scales == 0)), what
    else:
        assert np.all(np.abs(s - np.maximum(amax / 448, 2.0 ** -126)) <= slack / 448 + 2 * U * s), what
    full = ref.spread(s, y.shape, 1)
    q = y / full
    step = 2.0 ** (np.clip(np.floor(np.log2(np.maximum(np.abs(q), 2.0 ** -20))), -6, 8) - 3)
    got = ref.E4M3[codes] * full
    assert np.all(np.isfinite(got)), what
    # x * (1 / s) is within 1.5 u of x / s, and a value beside a power of two
    # may round by the larger step
    assert np.all(np.abs(got - y) <= 0.5 * full * step * (1 + 2.0 ** -15) * np.where(np.abs(q) * (1 + 1e-5) >= 2 * 2.0 ** np.floor(np.log2(np.maximum(np.abs(q), 2.0 ** -20))), 2, 1)
                  + 4 * U * np.abs(y) + tol), what


@pytest.mark.parametrize("e8m0", [False, True])
@pytest.mark.parametrize("rows,cols,P", [
    (1, 1, 1), (3, 7, 2), (2, 8, 8), (5, 127, 3), (4, 128, 4), (3, 129, 5), (1, 8192, 8), (9, 1000, 6), (2, 5003, 7),
    (3, 8193, 8), (2, 16384, 8), (2, 20000, 2), (1, 65536, 8), (2, 65535, 1), (300, 512, 8),
])
def test_norm_matches_plain(rows, cols, P, e8m0):
    xs, res, w = make(rows, cols, P, 1)
    note(f"norm rows={rows} cols={cols} P={P} e8m0={e8m0}")
    rbuf, r_out = out16(rows, cols)
    ybuf, y = out16(rows, cols)
    ld = -(-cols // 16) * 16
    cbuf = torch.full((rows + 1, ld), 0xA5, dtype=torch.uint8, device=DEV)
    codes = cbuf[:rows, :cols]
    nb = -(-cols // 128)
    sbuf = torch.full((nb, rows + 3), 77, dtype=torch.uint8 if e8m0 else torch.float32, device=DEV)
    scales = sbuf[:, :rows].t()
    tar.ar_reduce_norm([rows16(x) for x in xs], rows16(w[None])[0], residual=rows16(res), res_out=r_out, y=y, codes=codes,
                       scales=scales, eps=1e-5)
    torch.cuda.synchronize()
    h = ref.rank_sum(xs, res)
    assert np.array_equal(down16(r_out).reshape(rows, cols), ref.bf16_bits(h).reshape(rows, cols)), "res_out"
    want, tol = ref.norm(h, w, 1e-5), y_bound(xs, res, h, w, 1e-5)
    assert np.all(np.abs(vals(y) - want) <= tol + ref.U16 * np.abs(want) * (1 + 2.0 ** -7) + 2.0 ** -133), "y"
    check_codes(codes.cpu().numpy(), scales.cpu().numpy(), want, tol, "codes")
    assert untouched(rbuf, rows * cols) and untouched(ybuf, rows * cols)
    assert bool((cbuf[rows:] == 0xA5).all()) and bool((cbuf[:, cols:] == 0xA5).all()), "wrote past the codes"
    assert bool((sbuf[:, rows:] == 77).all()), "wrote past the scales"


def test_each_output_alone_and_optional_inputs():
    rows, cols, P = 7, 640, 3
    xs, res, w = make(rows, cols, P, 2)
    ins = [rows16(x) for x in xs]
    note("norm: each output alone, no residual, no gain, binary32 gain")
    h = ref.rank_sum(xs)
    r_out = torch.empty_like(ins[0])
    tar.ar_reduce_norm(ins, res_out=r_out)                               # the plain rank sum
    y1, y2 = torch.empty_like(r_out), torch.empty_like(r_out)
    tar.ar_reduce_norm(ins, y=y1)
    w32 = torch.from_numpy((w * 1.0001).astype(np.float32)).to(DEV)
    tar.ar_reduce_norm(ins, w32, y=y2)
    codes, scales = tar.fp8_codes_empty(rows, cols, DEV), tar.fp8_scales_empty(rows, cols, DEV)
    tar.ar_reduce_norm(ins, w32, codes=codes, scales=scales)
    torch.cuda.synchronize()
    assert np.array_equal(down16(r_out).ravel(), ref.bf16_bits(h).ravel())
    for got, gain in ((y1, None), (y2, w32.cpu().numpy())):
        want = ref.norm(h, gain, 1e-6)
        assert np.all(np.abs(vals(got) - want) <= y_bound(xs, None, h, gain, 1e-6) + 1.01 * ref.U16 * np.abs(want))
    want = ref.norm(h, w32.cpu().numpy(), 1e-6)
    check_codes(codes.cpu().numpy(), scales.cpu().numpy(), want, y_bound(xs, None, h, w32.cpu().numpy(), 1e-6), "codes")


def test_in_place_and_side_stream():
    rows, cols, P = 33, 1001, 4
    xs, res, w = make(rows, cols, P, 3)
    ins, r, wd = [rows16(x) for x in xs], rows16(res), rows16(w[None])[0]
    note("norm in place: res_out is the residual, y is a contribution; on a stream of its own")
    want_r, want_y = torch.empty_like(r), torch.empty_like(r)
    tar.ar_reduce_norm(ins, wd, residual=r, res_out=want_r, y=want_y)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    tar.ar_reduce_norm(ins, wd, residual=r, res_out=r, y=ins[2], stream=s)
    s.synchronize()
    assert torch.equal(r.view(torch.int16), want_r.view(torch.int16))
    assert torch.equal(ins[2].view(torch.int16), want_y.view(torch.int16))


def test_rows_of_zeros_infinities_and_nan():
    cols = 384
    x = np.zeros((5, cols), dtype=np.float32)
    g = np.random.default_rng(5)
    x[1:] = ref.as_bf16(g.standard_normal((4, cols)))
    x[1, 130] = np.inf
    x[2, 5] = np.nan
    x[3, 300] = -np.inf
    note("norm: a row of zeros, infinities and NaN stay in their rows")
    y = torch.empty(5, cols, dtype=torch.bfloat16, device=DEV)
    outs = []
    for e8m0 in (False, True):
        codes, scales = tar.fp8_codes_empty(5, cols, DEV), tar.fp8_scales_empty(5, cols, DEV, e8m0=e8m0)
        tar.ar_reduce_norm([rows16(x)], y=y, codes=codes, scales=scales, eps=1e-6)
        torch.cuda.synchronize()
        outs.append((codes.cpu().numpy(), scales.cpu().numpy()))
    got = vals(y)
    assert np.all(got[0] == 0)
    with np.errstate(invalid="ignore"):
        want = ref.norm(x, None, 1e-6)                # an infinity: itself NaN, the rest of its row 0
    for i in (1, 2, 3):
        assert np.array_equal(np.isnan(got[i]), np.isnan(want[i])) and np.all(got[i][~np.isnan(want[i])] == 0)
    assert np.all(np.abs(got[4] - want[4]) <= 0.01 * np.abs(want[4]))
    for (codes, scales), zero in zip(outs, (np.float32(2.0 ** -126), 0)):
        assert np.all(codes[0] == 0) and np.all(scales[0] == zero)
        assert np.array_equal(codes[1:4] == 0x7F, np.isnan(want[1:4]))
        assert np.all(scales[1:4] == zero)
    x = np.zeros((1, 128), dtype=np.float32)
    tar.ar_reduce_norm([rows16(x)], y=y[:1, :128].contiguous(), eps=0.0)   # 0 * inf: NaN, as documented


def test_extreme_magnitudes():
    """Rows near binary32's ends: squares that under- or overflow give the
    formula's own binary32 result, no fault of the code path."""
    cols = 256
    x = np.full((3, cols), 1.0, dtype=np.float32)
    x[0] = 2.0 ** -100
    x[1] = 2.0 ** 60
    x[2] = 2.0 ** 100                                     # squares overflow: 1 / inf = 0
    y = torch.empty(3, cols, dtype=torch.bfloat16, device=DEV)
    tar.ar_reduce_norm([rows16(x)], y=y, eps=1e-6)
    torch.cuda.synchronize()
    got = vals(y)
    assert np.all(np.abs(got[0] / (2.0 ** -100 * 1e3) - 1) <= 2 * ref.U16)
    assert np.all(got[1] == 1) and np.all(got[2] == 0)


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 8192), (5, 7), (3, 128), (130, 129), (600, 640), (1025, 1000), (2, 5003),
                                       (3, 16384), (2, 65536)])
@pytest.mark.parametrize("dres", [False, True])
def test_gradient_matches_formula(rows, cols, dres):
    g = np.random.default_rng([11, rows, cols])
    h = ref.as_bf16(g.standard_normal((rows, cols)) * np.exp(0.5 * g.standard_normal(cols)))
    dy = ref.as_bf16(0.01 * g.standard_normal((rows, cols)))
    w = ref.as_bf16(1 + 0.3 * g.standard_normal(cols))
    dr = ref.as_bf16(0.01 * g.standard_normal((rows, cols))) if dres else None
    note(f"norm gradient rows={rows} cols={cols} dres={dres}")
    xbuf, dx = out16(rows, cols)
    dwbuf = torch.full((cols + 4,), 7.0, dtype=torch.float32, device=DEV)
    ws = torch.full((tar.norm_bwd_workspace(rows, cols),), 0xFF, dtype=torch.uint8, device=DEV)
    args = (rows16(dy), rows16(h), rows16(w[None])[0])
    for _ in range(2):                                    # a second call overwrites, it does not add
        tar.ar_norm_bwd(*args, dx=dx, dres=None if dr is None else rows16(dr), dweight=dwbuf[:cols], workspace=ws, eps=1e-5)
    torch.cuda.synchronize()
    want, wdw = ref.norm_bwd(dy, h, w, dr, 1e-5)
    h64, dy64, w64 = h.astype(np.float64), dy.astype(np.float64), w.astype(np.float64)
    r = 1 / np.sqrt((h64 ** 2).mean(1, keepdims=True) + 1e-5)
    x, gg = h64 * r, np.abs(dy64 * w64)
    # the row's two sums, of magnitudes mean h^2 and mean |g x|, each within 100 u
    size = r * (gg + np.abs(x) * (gg * np.abs(x)).mean(1, keepdims=True)) + (0 if dr is None else np.abs(dr))
    assert np.all(np.abs(vals(dx) - want) <= 220 * U * size + 1.01 * ref.U16 * np.abs(want) + 2.0 ** -133), "dx"
    # a workgroup adds its rows, then at most 64 partial sums of every 64th workgroup and those of 64 (fewer
    # than the terms counted here for these sizes); each term within 110 u
    terms = -(-rows // 512) + 130 + 110
    assert np.all(np.abs(dwbuf[:cols].cpu().numpy() - wdw) <= terms * U * np.abs(dy64 * x).sum(0)), "dweight"
    assert untouched(xbuf, rows * cols) and bool((dwbuf[cols:] == 7).all())


def test_gradient_against_differences():
    """Directional derivatives of L(h) = sum(dy * y(h)) + sum(dres * h), by
    central differences in 64 bits, against the kernel's dx and dweight."""
    rows, cols, eps = 6, 200, 1e-5
    g = np.random.default_rng(21)
    h = ref.as_bf16(g.standard_normal((rows, cols)))
    dy, dr = (ref.as_bf16(g.standard_normal((rows, cols))) for _ in range(2))
    w = ref.as_bf16(1 + 0.3 * g.standard_normal(cols))
    dx = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    dw = torch.empty(cols, dtype=torch.float32, device=DEV)
    ws = torch.empty(tar.norm_bwd_workspace(rows, cols), dtype=torch.uint8, device=DEV)
    tar.ar_norm_bwd(rows16(dy), rows16(h), rows16(w[None])[0], dx=dx, dres=rows16(dr), dweight=dw, workspace=ws, eps=eps)
    torch.cuda.synchronize()
    got, gdw = vals(dx).astype(np.float64), dw.cpu().numpy().astype(np.float64)

    def loss(hh, ww):
        y = hh / np.sqrt((hh * hh).mean(1, keepdims=True) + eps) * ww
        return (dy * y).sum() + (dr * hh).sum()

    t = 1e-5
    for k in range(4):
        v = g.standard_normal((rows, cols))
        num = (loss(h + t * v, w.astype(np.float64)) - loss(h - t * v, w.astype(np.float64))) / (2 * t)
        # bf16 rounding of each dx, and the difference's own t^2 error (~1e-8 here)
        assert abs(num - (got * v).sum()) <= 1.05 * ref.U16 * np.abs(got * v).sum() + 1e-5
        v = g.standard_normal(cols)
        num = (loss(h.astype(np.float64), w + t * v) - loss(h.astype(np.float64), w - t * v)) / (2 * t)
        assert abs(num - (gdw * v).sum()) <= 1e-5 * np.abs(gdw * v).sum() + 1e-6


def test_gradient_parts_alone_in_place_and_no_rows():
    rows, cols = 40, 1003
    g = np.random.default_rng(31)
    h, dy, dr = (ref.as_bf16(g.standard_normal((rows, cols))) for _ in range(3))
    hd, yd, rd = rows16(h), rows16(dy), rows16(dr)
    ws = torch.empty(tar.norm_bwd_workspace(rows, cols), dtype=torch.uint8, device=DEV)
    dx, dw, dw2 = torch.empty_like(hd), torch.empty(cols, device=DEV), torch.full((cols,), 3.0, device=DEV)
    note("norm gradient: parts alone, in place, no rows")
    tar.ar_norm_bwd(yd, hd, dx=dx, dres=rd, dweight=dw, workspace=ws)
    dx2 = torch.empty_like(dx)
    tar.ar_norm_bwd(yd, hd, dx=dx2, dres=rd)
    tar.ar_norm_bwd(yd, hd, dweight=dw2, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(dx.view(torch.int16), dx2.view(torch.int16)) and torch.equal(dw, dw2)
    tar.ar_norm_bwd(yd, hd, dx=rd, dres=rd)
    torch.cuda.synchronize()
    assert torch.equal(dx.view(torch.int16), rd.view(torch.int16))
    empty = torch.empty(0, cols, dtype=torch.bfloat16, device=DEV)
    tar.ar_norm_bwd(empty, empty, dx=empty, dweight=dw)
    torch.cuda.synchronize()
    assert bool((dw == 0).all())


def test_repeats_bit_for_bit_and_in_a_graph():
    rows, cols, P = 700, 2050, 5
    xs, res, w = make(rows, cols, P, 6)
    ins, r, wd = [rows16(x) for x in xs], rows16(res), rows16(w[None])[0]
    y = torch.empty_like(r)
    codes, scales = tar.fp8_codes_empty(rows, cols, DEV), tar.fp8_scales_empty(rows, cols, DEV)
    dx, dw = torch.empty_like(r), torch.empty(cols, device=DEV)
    ws = torch.empty(tar.norm_bwd_workspace(rows, cols), dtype=torch.uint8, device=DEV)
    r_out = torch.empty_like(r)

    def step(stream=None):
        tar.ar_reduce_norm(ins, wd, residual=r, res_out=r_out, y=y, codes=codes, scales=scales, stream=stream)
        tar.ar_norm_bwd(y, r_out, wd, dx=dx, dres=r, dweight=dw, workspace=ws, stream=stream)

    def shot():
        torch.cuda.synchronize()
        return [t.clone() for t in (r_out.view(torch.int16), y.view(torch.int16), codes, scales, dx.view(torch.int16), dw)]

    note("norm and gradient: eager and replayed")
    step()
    want = shot()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(torch.cuda.current_stream())
    for k in range(3):
        for t in (r_out, y, dx, dw):
            t.zero_()
        graph.replay()
        for a, b in zip(shot(), want):
            assert torch.equal(a, b), f"replay {k}"
        step()
        for a, b in zip(shot(), want):
            assert torch.equal(a, b), f"eager {k}"
