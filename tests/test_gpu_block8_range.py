"""ar_gemm_fp8 at the ends of the range of scales that include/ar.h states: the
product of a block's two scales from 2^-126 to 2^127.  Whole numbers times one
power of two, so every partial sum is a normal binary32 number and exact; a
sum of no codes is zero, whatever the scales."""
import pytest
import torch

import tensor_all_reduce_amd as tar
from gpu_util import DEV, note

pytestmark = pytest.mark.gpu

ONE, THREE = 0x38, 0x44                                      # E4M3 codes of 1 and 3


def spread_scales(rows, K, brows, e8m0, k):
    s = tar.fp8_scales_empty(rows, K, DEV, brows, e8m0)
    s.fill_(k + 127 if e8m0 else 2.0 ** k)
    return s


def product(a, b, M, N, K, brows, e8m0, f32, ka, kb, workspace):
    """Scales 2^ka and 2^kb; codes given as [M, K] and [N, K] byte matrices."""
    out = torch.full((M, N), 9.0, dtype=torch.float32 if f32 else torch.bfloat16, device=DEV)
    ws = torch.zeros(tar.gemm_fp8_workspace(M, N, K), dtype=torch.uint8, device=DEV) if workspace else None
    tar.ar_gemm_fp8([a], [spread_scales(M, K, 1, e8m0, ka)], [b], [spread_scales(N, K, brows, e8m0, kb)], [out],
                    b_block_rows=brows, workspace=ws)
    return out


def codes(rows, K, ld=None):
    ld = ld or -(-K // 16) * 16
    c = torch.full((rows, ld), 0x7F, dtype=torch.uint8, device=DEV)[:, :K]
    return c.zero_()


# streaming kernel | large tiles: 128 rows, 256 rows, fewer blocks than they run ahead, slices | rows far apart
SIZES = [(3, 70, 300, None, False), (40, 300, 8192, None, True), (200, 4400, 700, None, False), (4200, 1100, 700, None, False),
         (4170, 1100, 100, None, False), (200, 4100, 1280, None, True), (3, 5, 300, (1 << 23) + 16, False)]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("e8m0", [False, True])
@pytest.mark.parametrize("brows", [1, 128])
@pytest.mark.parametrize("M,N,K,ld,split", SIZES)
def test_scales_at_the_ends_of_their_range(M, N, K, ld, split, brows, e8m0, f32):
    note(f"product with scales at the ends M={M} N={N} K={K} ld={ld} split={split} brows={brows} e8m0={e8m0} f32={f32}")
    m, n = torch.arange(M, device=DEV), torch.arange(N, device=DEV)
    a, b = codes(M, K, ld), codes(N, K, ld)
    # row m of a has a 1 in columns m % K and K - 1; row n of b has a 3 wherever n + k is a multiple of 3
    a[m, m % K] = ONE
    a[:, K - 1] = ONE
    k = torch.arange(K, device=DEV)
    b.copy_(torch.where((n[:, None] + k) % 3 == 0, THREE, 0))
    three = 3.0 * ((n[:, None] + k) % 3 == 0).float()
    want = three[:, m % K].t() + three[:, K - 1] * (m % K != K - 1).float()[:, None]       # 0, 3 or 6
    for ka, kb in ((-63, -63), (-100, -26), (-10, -116)):
        got = product(a, b, M, N, K, brows, e8m0, f32, ka, kb, split)
        assert torch.equal(got.double(), want.double() * 2.0 ** -126), f"2^{ka} 2^{kb}"
    for ka, kb in ((62, 62), (100, 24), (10, 114)):
        got = product(a, b, M, N, K, brows, e8m0, f32, ka, kb, split)
        assert torch.equal(got.double(), want.double() * 2.0 ** 124), f"2^{ka} 2^{kb}"
    # one term a result at most: 0 or 2^127
    a.zero_()
    a[m, m % K] = ONE
    b.copy_(torch.where((n[:, None] + k) % 3 == 0, ONE, 0))
    for ka, kb in ((63, 64), (117, 10)):
        got = product(a, b, M, N, K, brows, e8m0, f32, ka, kb, split)
        assert torch.equal(got.double(), (three / 3)[:, m % K].t().double() * 2.0 ** 127), f"2^{ka} 2^{kb}"
