"""ar_gemm_fp8 on both sides of the rules that choose its kernel, on whole
numbers with power-of-two scales, which are exact whatever the order."""
import numpy as np
import pytest

import block_ref as ref
from gpu_util import note
from test_gpu_block8 import int_codes, run

pytestmark = pytest.mark.gpu


def check(G, M, N, K, brows, e8m0, f32):
    g = np.random.default_rng([G, M, N, K])
    note(f"product G={G} M={M} N={N} K={K} brows={brows} e8m0={e8m0} f32={f32}")

    def matrix(rows, br):
        k = g.integers(-1, 2, size=(-(-rows // br), -(-K // 128)))
        return int_codes(g, rows, K), (k + 127).astype(np.uint8) if e8m0 else (2.0 ** k).astype(np.float32)

    def values(codes, scales, br):
        return ref.E4M3.astype(np.float32)[codes] * ref.spread(ref.scale_val(scales).astype(np.float32), codes.shape, br)

    A, B = [matrix(M, 1) for _ in range(G)], [matrix(N, brows) for _ in range(G)]
    got = run(A, B, brows, M, N, K, f32, 0, True)
    for i in range(G):
        want = values(*A[i], 1) @ values(*B[i], brows).T          # multiples of 1/4 below 2^24: exact in binary32
        assert np.array_equal(got[i], want if f32 else ref.as_bf16(want)), f"problem {i}: {int((got[i] != want).sum())} differ"


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
