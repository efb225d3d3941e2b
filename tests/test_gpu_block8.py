"""ar_quantize_block and ar_gemm_fp8 on the GPU against the plain forms.

The quantiser is compared bit for bit (every step is one binary32 operation).
Products: with u = 2^-23 for one matrix-core addition (which may truncate),
a sum over K products and ceil(K / 128) scaled blocks is within
(K + 3 ceil(K / 128)) u of the sum of the products' magnitudes; bf16 adds
2^-8 relatively.  Small integers with power-of-two scales are exact whatever
the order, and are compared exactly.
"""
import numpy as np
import pytest
import torch

import block_ref as ref
import tensor_all_reduce_amd as tar
from gpu_util import DEV, note, up16, down16

pytestmark = pytest.mark.gpu

FMT = [False, True]


def rows16(a, ld=None):
    t = up16(ref.bf16_bits(a)).view(torch.bfloat16).reshape(a.shape)
    if ld is None:
        return t
    buf = torch.full((a.shape[0], ld), float("nan"), dtype=torch.bfloat16, device=DEV)
    buf[:, :a.shape[1]] = t
    return buf[:, :a.shape[1]]


def code_buf(rows, cols, pad=0):
    buf = torch.full((rows + 1, -(-cols // 16) * 16 + pad), 0xA5, dtype=torch.uint8, device=DEV)
    return buf, buf[:rows, :cols]


def scale_buf(rows, cols, brows, e8m0, by_col):
    R, C = -(-rows // brows), -(-cols // 128)
    dt = torch.uint8 if e8m0 else torch.float32
    if by_col:
        buf = torch.full((C + 1, R + 2), 77, dtype=dt, device=DEV)
        return buf, buf[:C, :R].t()
    buf = torch.full((R + 1, C + 2), 77, dtype=dt, device=DEV)
    return buf, buf[:R, :C]


@pytest.mark.parametrize("e8m0", FMT)
@pytest.mark.parametrize("turn", [False, True])
@pytest.mark.parametrize("brows", [1, 128])
@pytest.mark.parametrize("rows,cols,ld", [(1, 1, None), (1, 1000, None), (130, 1, 5), (127, 129, 131), (128, 128, None),
                                          (257, 384, 400), (16, 8192, None), (301, 517, 523)])
def test_quantise_bit_for_bit(rows, cols, ld, brows, turn, e8m0):
    g = np.random.default_rng([rows, cols, brows])
    x = ref.as_bf16(g.standard_normal((rows, cols)) * np.exp(2 * g.standard_normal(cols)))
    x[:, : cols // 3] = 0                                        # blocks of zeros
    if rows > 2 and cols > 2:
        x[1, cols - 1], x[2, 0], x[0, cols // 2] = np.nan, np.inf, -np.inf
        x[rows - 1, cols - 2] = 3.38953139e38                    # the largest finite bf16
    x[0, cols - 1] = 1e-39                                       # a subnormal
    note(f"quantise rows={rows} cols={cols} brows={brows} turn={turn} e8m0={e8m0}")
    shape = (cols, rows) if turn else (rows, cols)
    cbuf, codes = code_buf(*shape, pad=16)
    sbuf, scales = scale_buf(*shape, brows, e8m0, by_col=turn)
    tar.ar_quantize_block(rows16(x, ld), codes, scales, block_rows=brows, transpose=turn)
    torch.cuda.synchronize()
    wc, ws = ref.quantise(x.T if turn else x, brows, e8m0)
    gc, gs = codes.cpu().numpy(), scales.cpu().numpy()
    assert np.array_equal(gs.view(np.uint8 if e8m0 else np.uint32), np.ascontiguousarray(ws).view(np.uint8 if e8m0 else np.uint32)), "scales"
    bad = np.argwhere(gc != wc)
    assert bad.size == 0, f"{len(bad)} codes differ, first at {bad[0]}: {gc[tuple(bad[0])]:#x} for {wc[tuple(bad[0])]:#x}"
    assert bool((cbuf[shape[0]:] == 0xA5).all()) and bool((cbuf[:, shape[1]:] == 0xA5).all()), "wrote past the codes"
    assert int((sbuf != 77).sum()) <= ws.size, "wrote past the scales"


def test_quantise_every_bf16_value():
    """Each finite pattern once, in blocks led by 448 (scale 1): all codes, both signs, every tie."""
    p = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    v = ref.bf16_val(p)
    v = v[np.isfinite(v) & (np.abs(v) <= 448)]
    x = np.zeros((-(-v.size // 127), 128), dtype=np.float32)
    x[:, 0] = 448
    x[:, 1:].flat[:v.size] = v
    codes, scales = tar.fp8_codes_empty(*x.shape, DEV), tar.fp8_scales_empty(*x.shape, DEV)
    tar.ar_quantize_block(rows16(x), codes, scales)
    torch.cuda.synchronize()
    assert bool((scales == 1).all())
    assert np.array_equal(codes.cpu().numpy(), ref.e4m3_codes(x))


# ------------------------------------------------------------------ products

def int_codes(g, rows, cols):
    """Codes of small whole numbers."""
    return ref.e4m3_codes(g.integers(-3, 4, size=(rows, cols)).astype(np.float64))


def put(codes, scales, by_col=True, pad=16):
    """Host codes and scales on the device; padding holds NaN codes."""
    rows, cols = codes.shape
    buf = torch.full((rows + 1, -(-cols // 16) * 16 + pad), 0x7F, dtype=torch.uint8, device=DEV)
    buf[:rows, :cols] = torch.from_numpy(codes).to(DEV)
    s = torch.from_numpy(np.ascontiguousarray(scales.T if by_col else scales)).to(DEV)
    return buf[:rows, :cols], s.t() if by_col else s


def out_buf(M, N, f32, pad):
    buf = torch.full((M + 1, N + pad), 9.0, dtype=torch.float32 if f32 else torch.bfloat16, device=DEV)
    return buf, buf[:M, :N]


def run(A, B, brows, M, N, K, f32, pad, split, by_col=True):
    G = len(A)
    a, b = [put(*v, by_col=by_col) for v in A], [put(*v, by_col=by_col) for v in B]
    outs = [out_buf(M, N, f32, pad) for _ in range(G)]
    ws = torch.zeros(tar.gemm_fp8_workspace(M, N, K, G), dtype=torch.uint8, device=DEV) if split else None
    for _ in range(2):                                   # the second call finds the workspace as the first left it
        tar.ar_gemm_fp8([v[0] for v in a], [v[1] for v in a], [v[0] for v in b], [v[1] for v in b], [v[1] for v in outs],
                        b_block_rows=brows, workspace=ws)
    torch.cuda.synchronize()
    for whole, _ in outs:
        assert bool((whole[M:] == 9).all()) and bool((whole[:, N:] == 9).all()), "wrote past the result"
    return [o.float().cpu().numpy() for _, o in outs]


SIZES = [(1, 1, 1), (1, 16, 128), (1, 128, 1024), (2, 100, 130), (5, 513, 1000), (15, 130, 256), (16, 256, 384),
         (17, 129, 129), (31, 64, 2048), (32, 1000, 511), (33, 200, 640), (48, 384, 1025), (64, 257, 300), (65, 128, 4096),
         (100, 1000, 100), (129, 127, 513), (200, 520, 1040), (257, 260, 272), (300, 130, 2176), (513, 770, 385)]


@pytest.mark.parametrize("e8m0", FMT)
@pytest.mark.parametrize("brows", [1, 128])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product_of_whole_numbers_is_exact(M, N, K, brows, e8m0):
    g = np.random.default_rng([M, N, K])
    note(f"product M={M} N={N} K={K} brows={brows} e8m0={e8m0}")

    def scales(rows, br):
        k = g.integers(-1, 2, size=(-(-rows // br), -(-K // 128)))
        return (k + 127).astype(np.uint8) if e8m0 else (2.0 ** k).astype(np.float32)

    A, B = (int_codes(g, M, K), scales(M, 1)), (int_codes(g, N, K), scales(N, brows))
    want = ref.dequantise(*A, 1) @ ref.dequantise(*B, brows).T     # multiples of 1/4 below 2^24: exact in binary32
    for split in (False, True):
        got, = run([A], [B], brows, M, N, K, True, 3, split, by_col=split)
        assert np.array_equal(got, want.astype(np.float32)), f"split={split}: {int((got != want).sum())} differ"
    got, = run([A], [B], brows, M, N, K, False, 0, True)
    assert np.array_equal(got, ref.as_bf16(want)), "bf16"


@pytest.mark.parametrize("e8m0", FMT)
@pytest.mark.parametrize("M,N,K,brows,G", [(1, 1024, 1024, 128, 8), (7, 300, 900, 128, 3), (64, 256, 4096, 1, 1),
                                           (300, 400, 1500, 128, 2), (512, 512, 2049, 1, 1)])
def test_product_matches_plain(M, N, K, brows, G, e8m0):
    g = np.random.default_rng([7, M, N, K])
    note(f"product of quantised values M={M} N={N} K={K} brows={brows} G={G} e8m0={e8m0}")
    A = [ref.quantise(ref.as_bf16(g.standard_normal((M, K)) * np.exp(g.standard_normal(K))), 1, e8m0) for _ in range(G)]
    B = [ref.quantise(ref.as_bf16(0.02 * g.standard_normal((N, K))), brows, e8m0) for _ in range(G)]
    for f32 in (False, True):
        got = run(A, B, brows, M, N, K, f32, 0, True)
        for i in range(G):
            a, b = ref.dequantise(*A[i], 1), ref.dequantise(*B[i], brows)
            want = a @ b.T
            tol = (K + 3 * -(-K // 128)) * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T)
            if not f32:
                tol = tol + 1.01 * ref.U16 * np.abs(want)
            assert np.all(np.abs(got[i] - want) <= tol), f"problem {i} f32={f32}: {np.abs(got[i] - want).max()}"


@pytest.mark.parametrize("M,N", [(3, 50), (200, 300)])
def test_nan_reaches_its_row_and_column_only(M, N):
    K = 300
    g = np.random.default_rng(3)
    A, B = int_codes(g, M, K), int_codes(g, N, K)
    A[M // 2, 299], B[N // 3, 5] = 0x7F, 0xFF
    one = lambda r: np.ones((r, 3), dtype=np.float32)    # noqa: E731
    got, = run([(A, one(M))], [(B, one(N))], 1, M, N, K, True, 1, True)
    nan = np.isnan(got)
    want = np.zeros((M, N), dtype=bool)
    want[M // 2], want[:, N // 3] = True, True
    assert np.array_equal(nan, want)
    s = np.full((M, 3), 127, dtype=np.uint8)
    s[0, 1] = 255                                        # a NaN scale byte
    A[M // 2, 299] = 0
    B[N // 3, 5] = 0
    got, = run([(A, s)], [(B, np.full((N, 3), 127, dtype=np.uint8))], 1, M, N, K, True, 0, True)
    assert np.all(np.isnan(got[0])) and np.all(np.isfinite(got[1:]))


def test_no_columns_of_k_writes_zeros_and_empty_results():
    note("product with K = 0, M = 0, N = 0")
    out = torch.full((5, 9), 3.0, device=DEV)
    z = lambda r, c: (torch.empty(r, c, dtype=torch.uint8, device=DEV), torch.empty(r, 0 if not c else 1, device=DEV))  # noqa: E731
    a, b = z(5, 0), z(9, 0)
    tar.ar_gemm_fp8([a[0]], [a[1]], [b[0]], [b[1]], [out], b_block_rows=1)
    torch.cuda.synchronize()
    assert bool((out == 0).all())
    out.fill_(3)
    a = z(0, 16)
    b = (torch.zeros(9, 16, dtype=torch.uint8, device=DEV), torch.ones(9, 1, device=DEV))
    tar.ar_gemm_fp8([a[0]], [a[1]], [b[0]], [b[1]], [out[:0]], b_block_rows=1)
    torch.cuda.synchronize()
    assert bool((out == 3).all())


def test_product_repeats_and_replays():
    """Bit for bit on every pass, eager or replayed, on two streams with a
    workspace each."""
    M, N, K, G = 24, 640, 8192, 2
    g = np.random.default_rng(13)
    A = [put(*ref.quantise(ref.as_bf16(g.standard_normal((M, K))), 1, False)) for _ in range(G)]
    B = [put(*ref.quantise(ref.as_bf16(g.standard_normal((N, K))), 128, False)) for _ in range(G)]
    outs = [torch.empty(M, N, device=DEV) for _ in range(G)]
    ws = torch.zeros(max(1, tar.gemm_fp8_workspace(M, N, K, G)), dtype=torch.uint8, device=DEV)

    def step(o=outs, w=ws, stream=None):
        tar.ar_gemm_fp8([v[0] for v in A], [v[1] for v in A], [v[0] for v in B], [v[1] for v in B], o, workspace=w, stream=stream)

    step()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(stream=torch.cuda.current_stream())
    for k in range(4):
        for o in outs:
            o.zero_()
        graph.replay() if k % 2 == 0 else step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), k
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    o2 = [torch.zeros_like(o) for o in outs]
    w2 = torch.zeros_like(ws)
    torch.cuda.synchronize()
    for _ in range(3):
        step(outs, ws, s1)
        step(o2, w2, s2)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs + o2, want + want))


@pytest.mark.parametrize("e8m0", FMT)
@pytest.mark.parametrize("K,brows", [(300, 128), (513, 1), (1152, 128)])
def test_product_of_many_tiles_is_exact(K, brows, e8m0):
    """More tiles than the device has compute units, ragged along M and N:
    every workgroup takes several, and the blocks of one follow another's."""
    M, N = 4130, 4360
    g = np.random.default_rng([17, K, brows])
    note(f"product M={M} N={N} K={K} brows={brows} e8m0={e8m0}")

    def scales(rows, br):
        k = g.integers(-1, 2, size=(-(-rows // br), -(-K // 128)))
        return (k + 127).astype(np.uint8) if e8m0 else (2.0 ** k).astype(np.float32)

    A, B = (int_codes(g, M, K), scales(M, 1)), (int_codes(g, N, K), scales(N, brows))
    want = (ref.dequantise(*A, 1).astype(np.float32) @ ref.dequantise(*B, brows).astype(np.float32).T)   # exact in binary32
    got, = run([A], [B], brows, M, N, K, True, 5, True)
    assert np.array_equal(got, want), f"{int((got != want).sum())} differ"
    got, = run([A], [B], brows, M, N, K, False, 8, True)
    assert np.array_equal(got, ref.as_bf16(want)), "bf16"


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("M,N,K", [(2, 70, 300), (200, 4100, 1280)])
def test_power_of_two_scales_far_apart(M, N, K, f32):
    """Scales near both ends of the byte's range whose products are moderate."""
    g = np.random.default_rng([23, M])
    A, B = int_codes(g, M, K), int_codes(g, N, K)
    sa = g.integers(10, 14, size=(M, -(-K // 128))).astype(np.uint8)            # 2^-117 .. 2^-114
    sb = g.integers(238, 242, size=(-(-N // 128), -(-K // 128))).astype(np.uint8)
    note(f"product with distant scales M={M} N={N} K={K}")
    want = ref.dequantise(A, sa, 1) @ ref.dequantise(B, sb, 128).T
    got, = run([(A, sa)], [(B, sb)], 128, M, N, K, f32, 0, True)
    assert np.array_equal(got, want.astype(np.float32) if f32 else ref.as_bf16(want))


@pytest.mark.parametrize("M,N,K", [(130, 8200, 8192 + 17), (200, 260, 2500), (700, 1030, 4200)])
def test_product_slices_agree(M, N, K):
    """With and without a workspace (slices of K or not), whole numbers."""
    g = np.random.default_rng([29, M])
    A = (int_codes(g, M, K), (2.0 ** g.integers(-1, 2, size=(M, -(-K // 128)))).astype(np.float32))
    B = (int_codes(g, N, K), (2.0 ** g.integers(-1, 2, size=(-(-N // 128), -(-K // 128)))).astype(np.float32))
    want = (ref.dequantise(*A, 1).astype(np.float32) @ ref.dequantise(*B, 128).astype(np.float32).T)
    note(f"product in slices M={M} N={N} K={K}: workspace {tar.gemm_fp8_workspace(M, N, K)}")
    for split in (True, False):
        got, = run([A], [B], 128, M, N, K, True, 0, split)
        assert np.array_equal(got, want), split


@pytest.mark.parametrize("f32,e8m0", [(False, False), (True, True), (True, False), (False, True)])
def test_product_of_rows_far_apart(f32, e8m0):
    """Rows 8 MiB and more apart, and scales with strides of their own."""
    M, N, K, ld = 3, 5, 300, (1 << 23) + 16
    g = np.random.default_rng(31)
    A, B = int_codes(g, M, K), int_codes(g, N, K)
    big = torch.full((M + N, ld), 0x7F, dtype=torch.uint8, device=DEV)
    a, b = big[:M, :K], big[M:, :K]
    a.copy_(torch.from_numpy(A).to(DEV))
    b.copy_(torch.from_numpy(B).to(DEV))
    k = g.integers(-1, 2, size=(M + N, 3))
    s = torch.from_numpy((k + 127).astype(np.uint8) if e8m0 else (2.0 ** k).astype(np.float32)).to(DEV)
    sc = torch.zeros(M + N, 21, dtype=s.dtype, device=DEV)[:, ::7]
    sc.copy_(s)
    out = torch.empty(M, N, dtype=torch.float32 if f32 else torch.bfloat16, device=DEV)
    note("product of rows far apart")
    tar.ar_gemm_fp8([a], [sc[:M]], [b], [sc[M:]], [out], b_block_rows=1)
    torch.cuda.synchronize()
    v = ref.spread(2.0 ** k.astype(np.float64), (M + N, K), 1)
    want = (ref.E4M3[A] * v[:M]) @ (ref.E4M3[B] * v[M:]).T
    assert np.array_equal(out.float().cpu().numpy(), want.astype(np.float32) if f32 else ref.as_bf16(want))


@pytest.mark.parametrize("M,N,K", [(4200, 1000, 200), (70, 9000, 256)])
def test_product_of_short_rows(M, N, K):
    g = np.random.default_rng([37, M])
    A = (int_codes(g, M, K), np.ones((M, 2), dtype=np.float32))
    B = (int_codes(g, N, K), np.ones((-(-N // 128), 2), dtype=np.float32))
    want = ref.dequantise(*A, 1).astype(np.float32) @ ref.dequantise(*B, 128).astype(np.float32).T
    note(f"product of short rows M={M} N={N} K={K}")
    for f32 in (True, False):
        got, = run([A], [B], 128, M, N, K, f32, 1, True)
        assert np.array_equal(got, want if f32 else ref.as_bf16(want))


def test_one_workspace_for_products_of_different_shapes():
    """Calls in stream order may share a workspace whatever their shapes: the
    counters of one do not lie where another kept its parts."""
    g = np.random.default_rng(41)
    shapes = [(1, 128, 8192), (1, 8192, 8192), (40, 1000, 4096), (128, 8192, 8320), (1, 8192, 8192), (128, 8192, 8320)]
    ws = torch.zeros(max(tar.gemm_fp8_workspace(*s) for s in shapes), dtype=torch.uint8, device=DEV)
    todo = []
    for M, N, K in shapes:
        A, B = int_codes(g, M, K), int_codes(g, N, K)
        one = lambda r: np.ones((r, K // 128), dtype=np.float32)    # noqa: E731
        a, b = put(A, one(M)), put(B, one(-(-N // 128)))
        todo.append((a, b, torch.full((M, N), 9.0, device=DEV), ref.E4M3[A].astype(np.float32) @ ref.E4M3[B].astype(np.float32).T))
    note("one workspace, several shapes")
    for _ in range(2):
        for a, b, out, _w in todo:
            tar.ar_gemm_fp8([a[0]], [a[1]], [b[0]], [b[1]], [out], workspace=ws)
    torch.cuda.synchronize()
    for i, (_a, _b, out, want) in enumerate(todo):
        assert np.array_equal(out.cpu().numpy(), want), f"product {i}: {shapes[i]}"


@pytest.mark.parametrize("e8m0", FMT)
def test_product_with_a_short_last_slice(e8m0):
    """65 blocks in slices of 9: the last has two, one of them with a tail."""
    M, N, K = 128, 8192, 8300
    g = np.random.default_rng(43)
    k = [g.integers(-1, 2, size=(r, 65)) for r in (M, N // 128)]
    s = [(v + 127).astype(np.uint8) if e8m0 else (2.0 ** v).astype(np.float32) for v in k]
    A, B = (int_codes(g, M, K), s[0]), (int_codes(g, N, K), s[1])
    want = ref.dequantise(*A, 1).astype(np.float32) @ ref.dequantise(*B, 128).astype(np.float32).T
    note("product with a short last slice")
    for f32 in (True, False):
        got, = run([A], [B], 128, M, N, K, f32, 0, True)
        assert np.array_equal(got, want if f32 else ref.as_bf16(want))


@pytest.mark.parametrize("M,N,K", [(3, 50, 300), (300, 4200, 700)])
@pytest.mark.parametrize("f32", [False, True])
def test_nan_scale_byte(M, N, K, f32):
    g = np.random.default_rng(47)
    A, B = int_codes(g, M, K), int_codes(g, N, K)
    nb = -(-K // 128)
    sa, sb = np.full((M, nb), 127, dtype=np.uint8), np.full((-(-N // 128), nb), 127, dtype=np.uint8)
    sa[1, nb - 1] = 255
    got, = run([(A, sa)], [(B, sb)], 128, M, N, K, f32, 0, True)
    assert np.all(np.isnan(got[1])) and np.all(np.isfinite(got[0])) and np.all(np.isfinite(got[2:]))


@pytest.mark.parametrize("M,f32", [(3, True), (150, False), (400, False)])
def test_results_side_by_side(M, f32):
    """Two problems write the two halves of one matrix."""
    N, K = 264, 700
    g = np.random.default_rng(53)
    A, B = [int_codes(g, M, K) for _ in range(2)], [int_codes(g, N, K) for _ in range(2)]
    one = lambda r: np.ones((r, 6), dtype=np.float32)    # noqa: E731
    a, b = [put(x, one(M)) for x in A], [put(x, one(3)) for x in B]
    whole = torch.full((M, 2 * N), 9.0, dtype=torch.float32 if f32 else torch.bfloat16, device=DEV)
    tar.ar_gemm_fp8([v[0] for v in a], [v[1] for v in a], [v[0] for v in b], [v[1] for v in b], [whole[:, :N], whole[:, N:]])
    torch.cuda.synchronize()
    want = np.concatenate([ref.E4M3[x] @ ref.E4M3[y].T for x, y in zip(A, B)], 1)
    assert np.array_equal(whole.float().cpu().numpy(), want.astype(np.float32) if f32 else ref.as_bf16(want))


@pytest.mark.parametrize("e8m0", FMT)
@pytest.mark.parametrize("brows", [1, 128])
@pytest.mark.parametrize("K", [1, 100, 128, 200, 256, 300, 384])
def test_large_tiles_of_few_blocks(K, brows, e8m0):
    """K shorter than the large tiles' run ahead."""
    M, N = 4170, 1100
    g = np.random.default_rng([59, K])
    note(f"large tiles K={K} brows={brows} e8m0={e8m0}")

    def scales(rows, br):
        k = g.integers(-1, 2, size=(-(-rows // br), -(-K // 128)))
        return (k + 127).astype(np.uint8) if e8m0 else (2.0 ** k).astype(np.float32)

    A, B = (int_codes(g, M, K), scales(M, 1)), (int_codes(g, N, K), scales(N, brows))
    want = ref.dequantise(*A, 1).astype(np.float32) @ ref.dequantise(*B, brows).astype(np.float32).T
    for f32 in (True, False):
        got, = run([A], [B], brows, M, N, K, f32, 1, True)
        assert np.array_equal(got, want if f32 else ref.as_bf16(want))


@pytest.mark.parametrize("e8m0", FMT)
@pytest.mark.parametrize("M,N,K,ld", [(8, 640, 700, None), (40, 300, 8192, None), (128, 8192, 8300, None), (4170, 1100, 700, None),
                                      (3, 5, 700, (1 << 23) + 16)])
def test_binary32_result_has_binary32_precision(M, N, K, ld, e8m0):
    """Each way a product can go.  A sum of K products takes K / 32 matrix
    instructions and as many scaled additions as blocks, each within 2^-24 of
    a partial sum of the result's size or so, at random: sqrt(K / 32 +
    K / 128) 2^-24, at most 1.1e-6 here; allowed is 2e-6 of the result's
    norm.  (Products of fp8 instructions are 1e-5 off.)"""
    g = np.random.default_rng([61, M, K])
    A = ref.quantise(ref.as_bf16(g.standard_normal((M, K)) * np.exp(g.standard_normal(K))), 1, e8m0)
    B = ref.quantise(ref.as_bf16(0.02 * g.standard_normal((N, K))), 1, e8m0)
    note(f"binary32 result M={M} N={N} K={K} ld={ld} e8m0={e8m0}")
    if ld is None:
        got, = run([A], [B], 1, M, N, K, True, 0, True)
    else:
        big = torch.zeros(M + N, ld, dtype=torch.uint8, device=DEV)
        big[:M, :K], big[M:, :K] = torch.from_numpy(A[0]).to(DEV), torch.from_numpy(B[0]).to(DEV)
        out = torch.empty(M, N, device=DEV)
        tar.ar_gemm_fp8([big[:M, :K]], [torch.from_numpy(A[1]).to(DEV)], [big[M:, :K]], [torch.from_numpy(B[1]).to(DEV)], [out],
                        b_block_rows=1)
        torch.cuda.synchronize()
        got = out.cpu().numpy()
    a, b = ref.dequantise(*A, 1), ref.dequantise(*B, 1)
    want = a @ b.T
    assert np.linalg.norm(got - want) <= 2e-6 * np.linalg.norm(want)
