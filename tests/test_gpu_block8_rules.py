"""ar_gemm_fp8 on both sides of the rules that choose its kernel, on whole
numbers with power-of-two scales: the results are multiples of 1/4 below 2^24,
exact in binary32 whatever the order, and the plain binary32 product gives
them on the device."""
import numpy as np
import pytest
import torch

import block_ref as ref
import tensor_all_reduce_amd as tar
from gpu_util import DEV, note

pytestmark = pytest.mark.gpu

CODES = torch.from_numpy(ref.e4m3_codes(np.arange(-3.0, 4.0)))


def matrix(gen, rows, K, brows, e8m0):
    """(codes, scales, the binary32 matrix they stand for); codes of the padding are NaN."""
    pick = torch.randint(0, 7, (rows, K), generator=gen, device=DEV)
    codes = torch.full((rows, -(-K // 16) * 16), 0x7F, dtype=torch.uint8, device=DEV)[:, :K]
    codes.copy_(CODES.to(DEV)[pick])
    scales = tar.fp8_scales_empty(rows, K, DEV, brows, e8m0)
    k = torch.randint(-1, 2, tuple(scales.shape), generator=gen, device=DEV)
    s = torch.exp2(k.float())
    scales.copy_(k + 127 if e8m0 else s)
    return codes, scales, (pick - 3).float() * s.repeat_interleave(brows, 0)[:rows].repeat_interleave(128, 1)[:, :K]


def check(G, M, N, K, brows, e8m0, f32):
    note(f"product G={G} M={M} N={N} K={K} brows={brows} e8m0={e8m0} f32={f32}")
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)
    A, B = [matrix(gen, M, K, 1, e8m0) for _ in range(G)], [matrix(gen, N, K, brows, e8m0) for _ in range(G)]
    outs = [torch.full((M, N), 9.0, dtype=torch.float32 if f32 else torch.bfloat16, device=DEV) for _ in range(G)]
    ws = torch.zeros(tar.gemm_fp8_workspace(M, N, K, G), dtype=torch.uint8, device=DEV)
    for _ in range(2):                                   # the second call finds the workspace as the first left it
        tar.ar_gemm_fp8([v[0] for v in A], [v[1] for v in A], [v[0] for v in B], [v[1] for v in B], outs, b_block_rows=brows,
                        workspace=ws)
    for i, out in enumerate(outs):
        want = (A[i][2] @ B[i][2].t()).to(out.dtype)
        assert torch.equal(out, want), f"problem {i}: {int((out != want).sum())} differ"


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("e8m0", [False, True])
@pytest.mark.parametrize("G,M,N,K,brows", [
    # 64-column tiles of all problems: up to 768 | more, up to 1024
    (6, 1, 8192, 1024, 128), (7, 1, 8192, 1024, 128), (8, 32, 8192, 1024, 128), (6, 17, 8200, 2047, 128), (1, 32, 50000, 130, 128),
    (7, 5, 9000, 1, 128),
    # with scales for each row of b: up to 512 | more, up to 768 | more
    (4, 32, 8192, 1024, 1), (4, 1, 8200, 1024, 1), (5, 32, 9000, 130, 1), (1, 17, 33000, 900, 1), (6, 7, 8192, 1, 1),
    (7, 32, 8192, 700, 1)])
def test_rings_of_one_and_two_blocks(G, M, N, K, brows, e8m0, f32):
    check(G, M, N, K, brows, e8m0, f32)


@pytest.mark.parametrize("f32,e8m0", [(False, False), (False, True), (True, False)])
@pytest.mark.parametrize("G,M,N,K,brows", [
    # a long K: up to 768 tiles of 32 rows | more
    (6, 1, 8192, 4200, 128), (7, 1, 8192, 4200, 128), (5, 32, 9000, 3300, 1),
    # up to 512 tiles of 64 rows | more
    (4, 64, 8192, 4200, 128), (4, 33, 8200, 4224, 128), (3, 40, 8192, 8300, 1),
    # large tiles of 128 rows | of 256
    (8, 128, 8192, 700, 128), (8, 129, 8192, 700, 128), (8, 100, 4300, 300, 1), (1, 65, 66000, 300, 128)])
def test_kernels_of_few_rows(G, M, N, K, brows, e8m0, f32):
    check(G, M, N, K, brows, e8m0, f32)


def test_most_rows_without_columns_of_k():
    """K = 0 writes zeros, up to the largest M there is."""
    M = 2 ** 31 - 1
    note(f"product M={M} N=1 K=0")
    out = torch.full((M, 1), 3.0, dtype=torch.bfloat16, device=DEV)
    z = lambda r: (torch.empty(r, 0, dtype=torch.uint8, device=DEV), torch.empty(r, 0, device=DEV))  # noqa: E731
    a, b = z(M), z(1)
    tar.ar_gemm_fp8([a[0]], [a[1]], [b[0]], [b[1]], [out], b_block_rows=1)
    torch.cuda.synchronize()
    assert not bool(out.view(torch.int16).any())
    del out
    torch.cuda.empty_cache()
