"""The norm, its gradient, the block quantiser and the fp8 product on buffers
of more than 2^31 elements: the first rows and the last are compared."""
import numpy as np
import pytest
import torch

import block_ref as ref
import tensor_all_reduce_amd as tar
from gpu_util import DEV, note, down16

pytestmark = pytest.mark.gpu

COLS = 8192
ROWS = (1 << 31) // COLS + 37


def vals(t):
    return ref.bf16_val(down16(t).reshape(-1)).reshape(t.shape)


@pytest.fixture(scope="module")
def x():
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    t = torch.empty(ROWS, COLS, dtype=torch.bfloat16, device=DEV)
    for a in range(0, ROWS, 32768):
        t[a:a + 32768] = torch.randn(min(32768, ROWS - a), COLS, generator=g, device=DEV).to(torch.bfloat16)
    yield t
    del t
    torch.cuda.empty_cache()


ENDS = (slice(0, 3), slice(ROWS - 40, ROWS))


def test_norm_beyond_32_bits(x):
    note(f"norm of {ROWS} x {COLS}")
    y = torch.empty_like(x)
    codes, scales = tar.fp8_codes_empty(ROWS, COLS, DEV), tar.fp8_scales_empty(ROWS, COLS, DEV)
    tar.ar_reduce_norm([x], y=y, codes=codes, scales=scales)
    torch.cuda.synchronize()
    for at in ENDS:
        want = ref.norm(vals(x[at]), None, 1e-6)
        assert np.all(np.abs(vals(y[at]) - want) <= 1.01 * ref.U16 * np.abs(want) + 1e-7)
        d = ref.dequantise(codes[at].cpu().numpy(), scales[at].cpu().numpy(), 1)
        s = ref.spread(scales[at].cpu().numpy().astype(np.float64), d.shape, 1)
        assert np.all(np.abs(d - want) <= 1.001 * np.maximum(np.abs(want) / 16, s * 2.0 ** -10))


def test_gradient_beyond_32_bits(x):
    note(f"norm gradient of {ROWS} x {COLS}")
    dx, dw = torch.empty_like(x), torch.empty(COLS, device=DEV)
    ws = torch.empty(tar.norm_bwd_workspace(ROWS, COLS), dtype=torch.uint8, device=DEV)
    tar.ar_norm_bwd(x, x, dx=dx, dres=x, dweight=dw, workspace=ws)
    torch.cuda.synchronize()
    for at in ENDS:
        v = vals(x[at])
        want, _ = ref.norm_bwd(v, v, None, v, 1e-6)
        assert np.all(np.abs(vals(dx[at]) - want) <= 1.01 * ref.U16 * np.abs(want) + 1e-5)
    # sum over rows of x^2 r, r close to 1: close to the number of rows
    assert np.all(np.abs(dw.cpu().numpy() / ROWS - 1) < 0.05)


@pytest.mark.parametrize("turn", [False, True])
def test_quantise_beyond_32_bits(x, turn):
    note(f"quantise {ROWS} x {COLS} turn={turn}")
    shape = (COLS, ROWS) if turn else (ROWS, COLS)
    codes, scales = tar.fp8_codes_empty(*shape, DEV), tar.fp8_scales_empty(*shape, DEV, e8m0=True)
    tar.ar_quantize_block(x, codes, scales, transpose=turn)
    torch.cuda.synchronize()
    if turn:
        first = (ROWS - 165) // 128 * 128                 # whole blocks and the ragged last
        v = vals(x[first:]).T
        c, s = codes[:, first:].cpu().numpy(), scales[:, first // 128:].cpu().numpy()
    else:
        v = vals(x[ENDS[1]])
        c, s = codes[ENDS[1]].cpu().numpy(), scales[ENDS[1]].cpu().numpy()
    wc, ws = ref.quantise(v, 1, True)
    assert np.array_equal(s, ws) and np.array_equal(c, wc)


def test_product_beyond_32_bits(x):
    """A [rows x 8192] result, and rows of a that start beyond 2^31 codes."""
    note(f"product of {ROWS} x {COLS}")
    M, N, K = ROWS, COLS, 256
    wide = torch.zeros(M, COLS + 16, dtype=torch.uint8, device=DEV)
    a = wide[:, 64:64 + K]
    g = np.random.default_rng(3)
    last = ref.e4m3_codes(g.integers(-3, 4, size=(40, K)).astype(np.float64))
    a[-40:] = torch.from_numpy(last).to(DEV)
    B = ref.e4m3_codes(g.integers(-3, 4, size=(N, K)).astype(np.float64))
    sa = torch.ones(M, 2, device=DEV)
    out = torch.full((M, N), 9.0, dtype=torch.bfloat16, device=DEV)
    for k in (K, 200):                                    # the two kernels' ranges of K differ below 257 only in length
        tar.ar_gemm_fp8([a[:, :k]], [sa], [torch.from_numpy(B).to(DEV)[:, :k]], [torch.ones(N // 128, 2, device=DEV)], [out])
        torch.cuda.synchronize()
        want = ref.as_bf16(ref.E4M3[last][:, :k] @ ref.E4M3[B][:, :k].T)
        assert np.array_equal(vals(out[-40:]), want) and bool((out[:3] == 0).all())
    del wide, out


def test_product_of_large_tiles_beyond_32_bits():
    M, N, K = ROWS, COLS, 384
    note(f"product of {M} x {N} x {K}")
    g = np.random.default_rng(5)
    a = torch.zeros(M, K, dtype=torch.uint8, device=DEV)
    last = ref.e4m3_codes(g.integers(-3, 4, size=(300, K)).astype(np.float64))
    a[-300:] = torch.from_numpy(last).to(DEV)
    B = ref.e4m3_codes(g.integers(-3, 4, size=(N, K)).astype(np.float64))
    out = torch.full((M, N), 9.0, dtype=torch.bfloat16, device=DEV)
    tar.ar_gemm_fp8([a], [torch.ones(M, 3, device=DEV)], [torch.from_numpy(B).to(DEV)], [torch.ones(N // 128, 3, device=DEV)], [out])
    torch.cuda.synchronize()
    assert np.array_equal(vals(out[-300:]), ref.as_bf16(ref.E4M3[last] @ ref.E4M3[B].T)) and bool((out[:3] == 0).all())
