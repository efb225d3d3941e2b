"""ar_reduce_norm and ar_norm_bwd on rows whose squares overflow binary32 while
their mean square does not.  Tolerances as in test_gpu_norm.py: 100 u for the
norm's own steps, 220 u of the sum of magnitudes for the gradient, 2^-8 for a
bf16 result.  The shapes take every number of 16-byte groups a lane, in rows
of whole groups and in ragged ones."""
import numpy as np
import pytest
import torch

import block_ref as ref
import tensor_all_reduce_amd as tar
from gpu_util import DEV, note
from test_gpu_norm import check_codes, rows16, vals, y_bound

pytestmark = pytest.mark.gpu

U = ref.U32
SHAPES = [(8, 128), (1, 512), (4, 8192), (4, 8185), (2, 4096), (1, 16384), (1, 16381), (1, 32768), (1, 32761), (1, 65536), (1, 65531)]


def large_rows(cols, seed):
    """All elements 1.5e19 with either sign; normal values up to 3e18 a
    standard deviation; a single element whose square is beyond binary32."""
    g = np.random.default_rng([seed, cols])
    x = np.zeros((3, cols), dtype=np.float32)
    x[0] = 1.5e19 * g.choice([-1.0, 1.0], size=cols)
    x[1] = np.clip(3e18 * g.standard_normal(cols), -1.8e19, 1.8e19)
    x[2, cols // 2] = 1e20
    x = ref.as_bf16(x)
    mean = (x.astype(np.float64) ** 2).mean(1)
    assert np.all(mean < 3.4e38) and np.any(x.astype(np.float64) ** 2 > 3.5e38)
    return x


@pytest.mark.parametrize("P,cols", SHAPES)
def test_norm_of_rows_near_the_end_of_the_range(P, cols):
    note(f"norm of large rows P={P} cols={cols}")
    x = large_rows(cols, 1)
    w = ref.as_bf16(1 + 0.3 * np.random.default_rng(2).standard_normal(cols))
    xs = [x] + [np.zeros_like(x)] * (P - 1)
    y = torch.empty(3, cols, dtype=torch.bfloat16, device=DEV)
    codes, scales = tar.fp8_codes_empty(3, cols, DEV), tar.fp8_scales_empty(3, cols, DEV)
    tar.ar_reduce_norm([rows16(v) for v in xs], rows16(w[None])[0], y=y, codes=codes, scales=scales)
    torch.cuda.synchronize()
    want, tol = ref.norm(x, w, 1e-6), y_bound(xs, None, x, w, 1e-6)
    assert np.all(np.abs(vals(y) - want) <= tol + 1.01 * ref.U16 * np.abs(want) + 2.0 ** -133)
    check_codes(codes.cpu().numpy(), scales.cpu().numpy(), want, tol, "codes")


@pytest.mark.parametrize("cols", sorted({c for _, c in SHAPES}))
def test_gradient_of_rows_near_the_end_of_the_range(cols):
    note(f"norm gradient of large rows cols={cols}")
    h = large_rows(cols, 3)
    g = np.random.default_rng([4, cols])
    dy = ref.as_bf16(g.standard_normal((3, cols)))
    w = ref.as_bf16(1 + 0.3 * g.standard_normal(cols))
    dx, dw = torch.empty(3, cols, dtype=torch.bfloat16, device=DEV), torch.empty(cols, device=DEV)
    ws = torch.empty(tar.norm_bwd_workspace(3, cols), dtype=torch.uint8, device=DEV)
    tar.ar_norm_bwd(rows16(dy), rows16(h), rows16(w[None])[0], dx=dx, dweight=dw, workspace=ws)
    torch.cuda.synchronize()
    want, wdw = ref.norm_bwd(dy, h, w, None, 1e-6)
    h64, dy64 = h.astype(np.float64), dy.astype(np.float64)
    r = 1 / np.sqrt((h64 ** 2).mean(1, keepdims=True) + 1e-6)
    x, gg = h64 * r, np.abs(dy64 * w.astype(np.float64))
    size = r * (gg + np.abs(x) * (gg * np.abs(x)).mean(1, keepdims=True))
    assert np.all(np.abs(vals(dx) - want) <= 220 * U * size + 1.01 * ref.U16 * np.abs(want) + 2.0 ** -133), "dx"
    assert np.all(np.abs(dw.cpu().numpy() - wdw) <= 250 * U * np.abs(dy64 * x).sum(0)), "dweight"
