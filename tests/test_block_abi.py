"""Argument checks of the norm, its gradient, the block quantiser and the fp8
product, and the plain forms the GPU tests compare with (CPU only: every
call here fails validation or has nothing to do)."""
import ctypes

import numpy as np
import pytest

import block_ref as ref
import tensor_all_reduce_amd as tar

vp = ctypes.c_void_p
A, B, C, D, E, F = (0x10000000 * k for k in range(1, 7))     # never dereferenced
INV, ALIGN, ALIAS, UNS, OK = tar.AR_ERR_INVALID, tar.AR_ERR_ALIGN, tar.AR_ERR_ALIAS, tar.AR_ERR_UNSUPPORTED, tar.AR_OK


def arr(*p):
    return (vp * len(p))(*p)


def mat(codes=E, ld=256, scales=F, rs=1, cs=64, fmt=0, br=1):
    return tar._Fp8Matrix(codes, ld, scales, rs, cs, fmt, br)


def norm(ins=(A, B), P=2, res=None, w=None, wf=0, rows=4, cols=200, eps=1e-6, r_out=C, y=None, q=None):
    return tar.lib().ar_reduce_norm(None if ins is None else arr(*ins), P, res, w, wf, rows, cols, eps, r_out, y,
                                    None if q is None else ctypes.byref(q), None)


def test_norm_refusals():
    assert norm(ins=None) == INV
    assert norm(P=0) == INV and norm(ins=(A,) * 9, P=9) == INV
    assert norm(ins=(A, None)) == INV
    assert norm(r_out=None) == INV                           # nothing to write
    assert norm(eps=-1e-6) == INV and norm(eps=float("nan")) == INV and norm(eps=float("inf")) == INV
    assert norm(cols=tar.AR_NORM_MAX_COLS + 1) == UNS
    assert norm(rows=2 ** 40, cols=2 ** 40) == INV
    assert norm(wf=2, w=D) == INV and norm(w=D + 4) == ALIGN
    for k in ("res", "r_out", "y"):
        assert norm(**{k: D + 2}) == ALIGN, k
    assert norm(r_out=A + 16) == ALIAS and norm(r_out=C, y=C) == ALIAS and norm(res=D, r_out=D + 32) == ALIAS
    assert norm(w=C) == ALIAS                                # the gain under an output
    assert norm(r_out=A, y=B, rows=0) == OK                  # exactly in place, no rows
    assert norm(rows=0) == OK and norm(cols=0) == OK
    # the fp8 result
    assert norm(q=mat(br=128)) == INV and norm(q=mat(br=2)) == INV and norm(q=mat(fmt=2)) == INV
    assert norm(q=mat(ld=192)) == INV and norm(q=mat(codes=None)) == INV and norm(q=mat(scales=None)) == INV
    assert norm(q=mat(ld=200)) == INV or norm(q=mat(ld=200)) == ALIGN
    assert norm(q=mat(ld=216)) == ALIGN and norm(q=mat(codes=E + 8)) == ALIGN and norm(q=mat(scales=F + 2)) == ALIGN
    assert norm(q=mat(rs=1, cs=3)) == ALIAS and norm(q=mat(rs=0)) == ALIAS and norm(q=mat(cs=0)) == ALIAS
    assert norm(q=mat(codes=C + 16)) == ALIAS and norm(q=mat(scales=E + 64)) == ALIAS and norm(q=mat(codes=A)) == ALIAS


def bwd(dy=A, h=B, w=None, wf=0, dres=None, rows=4, cols=200, eps=1e-6, dx=C, dw=None, ws=None, wb=0):
    return tar.lib().ar_norm_bwd(dy, h, w, wf, dres, rows, cols, eps, dx, dw, ws, wb, None)


def test_norm_bwd_refusals():
    need = tar.norm_bwd_workspace(4, 200)
    assert need >= 800
    assert bwd(dy=None) == INV and bwd(h=None) == INV and bwd(dx=None) == INV and bwd(eps=-1.0) == INV
    assert bwd(cols=tar.AR_NORM_MAX_COLS + 1) == UNS and bwd(rows=2 ** 40, cols=2 ** 24) == INV
    assert bwd(dw=D) == INV and bwd(dw=D, ws=E, wb=need - 1) == INV
    assert bwd(dw=D + 4, ws=E, wb=need) == ALIGN and bwd(dw=D, ws=E + 8, wb=need) == ALIGN
    for k in ("dy", "h", "dres", "dx"):
        assert bwd(**{k: D + 2}) == ALIGN, k
    assert bwd(dx=A + 16) == ALIAS and bwd(w=C) == ALIAS
    assert bwd(dw=C, ws=E, wb=need) == ALIAS and bwd(dw=D, ws=A, wb=need) == ALIAS and bwd(dw=D, ws=D, wb=need) == ALIAS
    assert bwd(rows=0) == OK and bwd(cols=0) == OK and bwd(dx=A, rows=0) == OK
    assert tar.norm_bwd_workspace(0, 100) == 0


def quant(x=A, ldx=200, rows=300, cols=200, q=None, turn=0):
    q = mat(cs=512) if q is None else q
    return tar.lib().ar_quantize_block(x, ldx, rows, cols, ctypes.byref(q), turn, None)


def test_quantise_refusals():
    L = tar.lib()
    assert L.ar_quantize_block(A, 200, 4, 200, None, 0, None) == INV
    assert quant(x=None) == INV and quant(ldx=199) == INV and quant(x=A + 1) == ALIGN
    assert quant(q=mat(ld=192, cs=512)) == INV and quant(q=mat(fmt=7, cs=512)) == INV and quant(q=mat(br=64, cs=512)) == INV
    assert quant(q=mat(ld=256, cs=512), turn=1) == INV                    # rows of 300 codes
    assert quant(q=mat(codes=A + 4096, cs=512)) == ALIAS and quant(q=mat(scales=E + 4, cs=512)) == ALIAS
    assert quant(q=mat(cs=299)) == ALIAS
    assert quant(rows=2 ** 62, ldx=2 ** 10) == INV
    assert quant(rows=0) == OK and quant(cols=0) == OK


def gemm(a=None, b=None, c=(C,), G=1, M=4, N=40, K=200, ldc=40, out=0, ws=None, wb=0):
    a = [mat(A, 256, B, 1, 4)] * G if a is None else a
    b = [mat(D, 256, E, 1, 1, br=128)] * G if b is None else b
    pack = lambda m: (tar._Fp8Matrix * len(m))(*m)           # noqa: E731
    return tar.lib().ar_gemm_fp8(pack(a), pack(b), arr(*c), G, M, N, K, ldc, out, ws, wb, None)


def test_product_refusals():
    L = tar.lib()
    assert L.ar_gemm_fp8(None, None, arr(C), 1, 4, 40, 200, 40, 0, None, 0, None) == INV
    assert gemm(G=0) == INV and gemm(G=9, c=(C,) * 9) == INV and gemm(c=(None,)) == INV
    assert gemm(ldc=39) == INV and gemm(out=2) == INV
    assert gemm(M=2 ** 31) == UNS and gemm(K=2 ** 31) == UNS and gemm(N=2 ** 22, ldc=2 ** 22) == UNS
    assert gemm(c=(C + 8,)) == ALIGN and gemm(ws=F + 8, wb=64) == ALIGN
    good_a, good_b = mat(A, 256, B, 1, 4), mat(D, 256, E, 1, 1, br=128)
    assert gemm(a=[mat(A, 256, B, 1, 4, br=128)]) == INV                  # activations have row scales
    assert gemm(a=[mat(A, 256, B, 1, 4, fmt=1)]) == INV                   # one scale format for both
    assert gemm(a=[mat(A, 208, B, 1, 4), good_a], b=[good_b] * 2, G=2, c=(C, F)) == INV
    assert gemm(a=[mat(A, 192, B, 1, 4)]) == INV and gemm(a=[mat(A, 200, B, 1, 4)]) == ALIGN
    assert gemm(a=[mat(A + 8, 256, B, 1, 4)]) == ALIGN and gemm(b=[mat(D, 256, E + 2, 1, 1, br=128)]) == ALIGN
    assert gemm(c=(A,)) == ALIAS and gemm(c=(E,)) == ALIAS
    assert gemm(G=2, c=(C, C + 16)) == ALIAS and gemm(G=2, c=(C, C + 16), ldc=96) == ALIAS
    assert gemm(G=2, c=(C, C + 192 - 16), ldc=96) == ALIAS               # 16 bytes short of the next row
    assert gemm(M=0) == OK and gemm(N=0) == OK
    assert tar.gemm_fp8_workspace(0, 5, 5) == 0 and tar.gemm_fp8_workspace(5, 5, 5, 9) == 0


class FakeTensor:
    is_cuda = True

    def __init__(self, ptr, shape, es, stride=None, fp=True):
        self.p, self.shape, self.es, self.fp = ptr, tuple(shape), es, fp
        self._st = stride or ((shape[1], 1) if len(shape) == 2 else (1,))

    def dim(self):
        return len(self.shape)

    def numel(self):
        return int(np.prod(self.shape))

    def element_size(self):
        return self.es

    def stride(self, i):
        return self._st[i]

    def is_contiguous(self):
        return True

    def is_floating_point(self):
        return self.fp

    def data_ptr(self):
        return self.p


def test_binding_refusals_and_prepared_calls():
    t = lambda p, s, es=2, **k: FakeTensor(p, s, es, **k)    # noqa: E731
    ins, out = [t(A, (4, 256)), t(B, (4, 256))], t(C, (4, 256))
    with pytest.raises(ValueError, match="shape"):
        tar.ar_reduce_norm(ins, res_out=t(C, (4, 128)), stream=0)
    with pytest.raises(ValueError, match="weight holds"):
        tar.ar_reduce_norm(ins, t(D, (255,)), res_out=out, stream=0)
    with pytest.raises(ValueError, match="come together"):
        tar.ar_reduce_norm(ins, codes=t(E, (4, 256), 1), stream=0)
    with pytest.raises(ValueError, match="scales must have shape"):
        tar.ar_reduce_norm(ins, codes=t(E, (4, 256), 1), scales=t(F, (4, 3), 4), stream=0)
    with pytest.raises(ValueError, match="binary32 or power-of-two"):
        tar.ar_reduce_norm(ins, codes=t(E, (4, 256), 1), scales=t(F, (4, 2), 2), stream=0)
    with pytest.raises(ValueError, match="contiguous rows"):
        tar.ar_quantize_block(t(A, (4, 256), stride=(1, 4)), t(E, (4, 256), 1), t(F, (4, 2), 4), stream=0)
    with pytest.raises(ValueError, match="one matrix"):
        tar.ar_gemm_fp8([], [], [], [], [], stream=0)
    a, b = t(A, (4, 256), 1), t(B, (8, 128), 1)
    with pytest.raises(ValueError, match="shape"):           # another K
        tar.ar_gemm_fp8([a], [t(C, (4, 2), 4)], [b], [t(D, (1, 2), 4)], [t(E, (4, 8))], stream=0)
    # each call prepares, and its handle reaches the C checks
    bad = t(C + 2, (4, 256))
    calls = [
        (tar.ar_reduce_norm, (ins,), dict(res_out=bad)),
        (tar.ar_norm_bwd, (ins[0], ins[1]), dict(dx=bad)),
        (tar.ar_quantize_block, (ins[0], t(E + 8, (4, 256), 1), t(F, (4, 2), 4)), {}),
        (tar.ar_gemm_fp8, ([a], [t(C, (4, 2), 4)], [t(B, (8, 256), 1)], [t(D, (1, 2), 4)], [t(E + 2, (4, 8))]), {}),
    ]
    assert {c[0] for c in calls} == tar._PREPARABLE_BLOCK
    for func, args, kw in calls:
        handle = tar.prepare(func, *args, stream=0, **kw)
        assert handle.name == func.__name__
        with pytest.raises(tar.ARError) as e:
            handle()
        assert e.value.code == ALIGN, func.__name__


# ------------------------------------------------ the plain forms themselves

def test_plain_codes_against_a_search():
    g = np.random.default_rng(0)
    x = np.concatenate([g.standard_normal(2000) * np.exp(3 * g.standard_normal(2000)), ref._MID, -ref._MID, ref.E4M3[:127]])
    x = x[np.abs(x) <= 448]
    for v, c in zip(x, ref.e4m3_codes(x)):
        d = np.abs(ref._POS - abs(v))
        near = np.flatnonzero(d == d.min())
        best = near[0] if len(near) == 1 else near[near % 2 == 0][0]
        assert c & 0x7F == best and (c >> 7) == int(np.signbit(v))


def test_plain_scales_are_the_smallest_that_fit():
    g = np.random.default_rng(1)
    f = (g.standard_normal((5, 700)) * np.exp(10 * g.standard_normal((5, 1)))).astype(np.float32)
    f[1, :128] = 0
    amax = ref.block_amax(f, 1).astype(np.float64)
    _, s = ref.quantise(f, 1, True)
    v = ref.scale_val(s)
    assert np.all(amax <= 448 * v) and np.all((amax > 224 * v) | (s == 0))
    c, s = ref.quantise(f, 1, False)
    assert np.all(np.abs(ref.scale_val(s) * 448 - amax) <= 2.0 ** -23 * amax + 448 * 2.0 ** -126)
    d = ref.dequantise(c, s, 1)
    assert np.all(np.abs(d - f) <= np.maximum(np.abs(f) / 16, ref.spread(ref.scale_val(s), f.shape, 1) * 2.0 ** -10) * 1.001)


def test_plain_gradient_against_differences():
    g = np.random.default_rng(2)
    h, dy, dr = (g.standard_normal((3, 50)) for _ in range(3))
    w, eps, t = 1 + 0.3 * g.standard_normal(50), 1e-3, 1e-5
    dx, dw = ref.norm_bwd(dy, h, w, dr, eps)
    loss = lambda hh, ww: (dy * ref.norm(hh, ww, eps)).sum() + (dr * hh).sum()   # noqa: E731
    for _ in range(5):
        v, u = g.standard_normal(h.shape), g.standard_normal(50)
        assert abs((loss(h + t * v, w) - loss(h - t * v, w)) / (2 * t) - (dx * v).sum()) < 1e-7
        assert abs((loss(h, w + t * u) - loss(h, w - t * u)) / (2 * t) - (dw * u).sum()) < 1e-7
