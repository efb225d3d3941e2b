"""The bindings of the norm, the block quantiser and the fp8 product refuse
element types that their bytes would be misread as: every other type of the
same size is a silent wrong answer."""
import pytest
import torch

import tensor_all_reduce_amd as tar

A, B, C, D, E, F = (0x10000000 * k for k in range(1, 7))     # never dereferenced


class FakeTensor:
    """A device tensor of a type, by address."""
    is_cuda = True

    def __init__(self, ptr, shape, dtype):
        self.ptr, self.shape, self.dtype = ptr, shape, dtype

    def dim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def element_size(self):
        return self.dtype.itemsize

    def stride(self, i):
        return (self.shape[1], 1)[i]

    def is_contiguous(self):
        return True

    def is_floating_point(self):
        return self.dtype.is_floating_point

    def data_ptr(self):
        return self.ptr


BF16, F16, F32, U8 = torch.bfloat16, torch.float16, torch.float32, torch.uint8
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def norm(x=BF16, residual=BF16, res_out=BF16, y=BF16, weight=BF16, codes=E4M3, scales=F32):
    t = lambda p, d, s=(4, 256): FakeTensor(p, s, d)         # noqa: E731
    return tar.prepare(tar.ar_reduce_norm, [t(A, x)], t(F, weight, (256,)), residual=t(B, residual), res_out=t(C, res_out), y=t(D, y),
                       codes=t(E, codes), scales=t(E + 4096, scales, (4, 2)), stream=0)


def bwd(dy=BF16, h=BF16, weight=F32, dx=BF16, dres=BF16, dweight=F32):
    t = lambda p, d, s=(4, 256): FakeTensor(p, s, d)         # noqa: E731
    return tar.prepare(tar.ar_norm_bwd, t(A, dy), t(B, h), t(F, weight, (256,)), dx=t(C, dx), dres=t(D, dres),
                       dweight=t(E, dweight, (256,)), workspace=t(E + 65536, U8, (tar.norm_bwd_workspace(4, 256),)), stream=0)


def quant(x=BF16, codes=U8, scales=F32):
    return tar.prepare(tar.ar_quantize_block, FakeTensor(A, (4, 256), x), FakeTensor(B, (4, 256), codes),
                       FakeTensor(C, (4, 2), scales), stream=0)


def gemm(a=U8, sa=F32, b=E4M3, sb=F32, out=BF16):
    t = lambda p, s, d: [FakeTensor(p, s, d)]                # noqa: E731
    return tar.prepare(tar.ar_gemm_fp8, t(A, (4, 256), a), t(B, (4, 2), sa), t(C, (8, 256), b), t(D, (1, 2), sb), t(E, (4, 8), out),
                       stream=0)


def test_types_that_the_operators_take():
    norm(), norm(x=torch.int16, weight=F32, codes=U8, scales=E8M0), norm(y=torch.uint16, scales=U8)
    bwd(), bwd(weight=BF16, dx=torch.int16)
    quant(), quant(torch.int16, E4M3, E8M0), quant(scales=U8)
    gemm(), gemm(E4M3, E8M0, U8, U8), gemm(out=F32), gemm(out=torch.int16)


@pytest.mark.parametrize("call,name,dtype", [
    (norm, "x", F16), (norm, "residual", F16), (norm, "res_out", F16), (norm, "y", F16), (norm, "weight", F16),
    (norm, "weight", torch.int32), (norm, "codes", torch.float8_e5m2), (norm, "codes", torch.float8_e4m3fnuz), (norm, "codes", E8M0),
    (norm, "codes", torch.bool), (norm, "scales", E4M3), (norm, "scales", torch.int32),
    (bwd, "dy", F16), (bwd, "h", F16), (bwd, "dx", F16), (bwd, "dres", F16), (bwd, "weight", F16), (bwd, "dweight", torch.int32),
    (quant, "x", F16), (quant, "codes", torch.float8_e5m2), (quant, "scales", E4M3), (quant, "scales", torch.int32),
    (gemm, "a", torch.float8_e5m2), (gemm, "b", torch.float8_e5m2fnuz), (gemm, "sa", E4M3), (gemm, "sb", torch.float8_e5m2),
    (gemm, "a", E8M0), (gemm, "out", F16), (gemm, "out", torch.int32)])
def test_types_that_they_refuse(call, name, dtype):
    with pytest.raises(ValueError, match="must (have|be)"):
        call(**{name: dtype})


def test_row_strides_that_the_codes_refuse():
    """A stride of at least the row's length that is no multiple of 16, apart
    from one that is shorter."""
    def call(ld):
        m = tar._Fp8Matrix(E, ld, F, 1, 64, 0, 1)
        ins = (tar._vp * 1)(A)
        return tar.lib().ar_reduce_norm(ins, 1, None, None, 0, 4, 200, 1e-6, C, None, tar.ctypes.byref(m), None)

    assert call(200) == tar.AR_ERR_ALIGN and call(216) == tar.AR_ERR_ALIGN
    assert call(192) == tar.AR_ERR_INVALID and call(0) == tar.AR_ERR_INVALID
