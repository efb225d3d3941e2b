"""A row of zeros without eps: 1 / sqrt(0) is infinite and 0 * infinity NaN, in
the bf16 result and in the codes; other rows are not touched by it."""
import numpy as np
import pytest
import torch

import block_ref as ref
import tensor_all_reduce_amd as tar
from gpu_util import DEV, note
from test_gpu_norm import rows16, vals

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("e8m0", [False, True])
@pytest.mark.parametrize("cols", [1, 128, 384, 1001])
def test_row_of_zeros_without_eps_is_nan(cols, e8m0):
    note(f"norm of a row of zeros, eps 0, cols={cols} e8m0={e8m0}")
    x = np.ones((3, cols), dtype=np.float32)
    x[1] = 0
    y = torch.zeros(3, cols, dtype=torch.bfloat16, device=DEV)
    codes, scales = tar.fp8_codes_empty(3, cols, DEV), tar.fp8_scales_empty(3, cols, DEV, e8m0=e8m0)
    tar.ar_reduce_norm([rows16(x)], y=y, codes=codes, scales=scales, eps=0.0)
    torch.cuda.synchronize()
    got, c, s = vals(y), codes.cpu().numpy(), scales.cpu().numpy()
    assert np.all(np.isnan(got[1])) and np.all(c[1] == 0x7F)
    assert np.all(s[1] == (0 if e8m0 else np.float32(2.0 ** -126)))
    assert np.all(got[[0, 2]] == 1)
    # 1 is 448 / 448: the largest code, or 2^-8 * 256
    assert np.all(ref.dequantise(c[[0, 2]], s[[0, 2]], 1).astype(np.float32) == 1)
