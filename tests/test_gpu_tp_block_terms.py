"""The gradients of the tensor-parallel step along the directions of their own
terms, against central differences in 64 bits of the unquantised step
    L(h, gain) = sum(d_outs . (norm(h) gain W^T)) + sum(d_hidden . h)
taken at the sum that the step wrote.  What is left between the two is the
rounding of d_outs and W to 8 bits and of bf16 results:

- an 8-bit value is off by at most e = max(|value| / 16, scale * 2^-10), half a
  step, so by e / sqrt(3) or less in the root mean square of even roundings;
- with U the derivative of the directional derivative by dy, d_outs comes into
  it with U W and W with d_outs^T U, so those roundings have the variance
  sum(e_d^2 (U W^T)^2) + sum(e_w^2 (d_outs^T U)^2), each over 3;
- bf16 results (a rank's gradient, their sum, dx) are off by 2^-8 or less each.
Allowed are six such standard deviations."""
import numpy as np
import pytest
import torch

import block_ref as ref
from tensor_all_reduce_amd import tp_block
from gpu_util import note
from test_gpu_tp_block import vals

pytestmark = pytest.mark.gpu


def half_steps(x, m, block_rows):
    s = ref.spread(ref.scale_val(m[1].cpu().numpy()), x.shape, block_rows)
    return np.maximum(np.abs(x) / 16, s * 2.0 ** -10)


@pytest.mark.parametrize("P,T,H,I,O,e8m0", [(2, 64, 512, 256, 384, False), (3, 40, 640, 128, 200, True)])
def test_gradients_along_their_terms(P, T, H, I, O, e8m0):
    note(f"block gradients along their terms P={P} tokens={T} hidden={H} e8m0={e8m0}")
    b, _, col = tp_block.random_block(P, T, H, I, O, seed=11, e8m0=e8m0)
    b.forward()
    b.backward()
    torch.cuda.synchronize()
    h, gain, d_hidden = vals(b.hidden_out), vals(b.gain[None])[0], vals(b.d_hidden)
    d, w = [vals(t) for t in b.d_outs], [vals(t) for t in col]
    ed, ew = [half_steps(x, m, 1) for x, m in zip(d, b.d_q)], [half_steps(x, m, 128) for x, m in zip(w, b.col_w)]
    ranks = sum(np.abs(vals(t)) for t in b.d_parts) + np.abs(vals(b.d_normed))
    dx, dgain = vals(b.d_residual), b.d_gain.double().cpu().numpy()

    def loss(hh, gg):
        y = ref.norm(hh, gg, b.eps)
        return sum((x * (y @ m.T)).sum() for x, m in zip(d, w)) + (d_hidden * hh).sum()

    def sigma(U):
        var = sum(((e * (U @ m.T)) ** 2).sum() + ((f * (x.T @ U)) ** 2).sum() for x, m, e, f in zip(d, w, ed, ew)) / 3
        return np.sqrt(var) + 2.0 ** -8 * np.linalg.norm(U * ranks)

    r = 1 / np.sqrt((h * h).mean(1, keepdims=True) + b.eps)
    x, dy = h * r, vals(b.d_normed)
    t, g = 1e-5, np.random.default_rng(12)
    radial = x * ((dy * gain * x).mean(1, keepdims=True))
    for name, v in (("itself", dx), ("the part through the norm", dx - d_hidden), ("the part past it", d_hidden), ("the row", h),
                    ("its mean term", r * radial), ("its first term", r * dy * gain), ("any", g.standard_normal(h.shape))):
        v = v / np.sqrt((v * v).mean())
        num = (loss(h + t * v, gain) - loss(h - t * v, gain)) / (2 * t)
        U = r * gain * (v - x * (v * x).mean(1, keepdims=True))
        tol = 6 * (sigma(U) + 2.0 ** -8 * np.linalg.norm(dx * v))
        assert abs(num - (dx * v).sum()) <= tol, f"along {name}: {(dx * v).sum()} for {num}, allowed {tol}"
    for name, v in (("itself", dgain), ("any", g.standard_normal(H))):
        v = v / np.sqrt((v * v).mean())
        num = (loss(h, gain + t * v) - loss(h, gain - t * v)) / (2 * t)
        tol = 6 * sigma(x * v)
        assert abs(num - (dgain * v).sum()) <= tol, f"gain along {name}: {(dgain * v).sum()} for {num}, allowed {tol}"
