"""The norm, the block quantiser and the fp8 product together, as a
tensor-parallel step uses them (tensor_all_reduce_amd.tp_block), against
64-bit products of the same quantised operands.

Each stage is compared on the operands that the stage before really made, so
the tolerances are the operators' own: (K + 3 ceil(K / 128)) 2^-23 of the
sums of magnitudes for a product, 2^-8 relatively for a bf16 result.
"""
import numpy as np
import pytest
import torch

import block_ref as ref
from tensor_all_reduce_amd import tp_block
from gpu_util import note, down16

pytestmark = pytest.mark.gpu


def vals(t):
    return ref.bf16_val(down16(t).reshape(-1)).reshape(t.shape).astype(np.float64)


def deq(m, block_rows):
    return ref.dequantise(m[0].cpu().numpy(), m[1].cpu().numpy(), block_rows)


def check_product(got, a, b, what, bf16=True):
    K = a.shape[1]
    want = a @ b.T
    tol = (K + 3 * -(-K // 128)) * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T)
    assert np.all(np.abs(got - want) <= tol + (1.01 * ref.U16 * np.abs(want) if bf16 else 0)), what


def check_rounding(x, m, block_rows, what):
    """Codes stand for x within half a step: 1/16 of a normal code's value, or
    half of the smallest step."""
    d = deq(m, block_rows)
    s = ref.spread(ref.scale_val(m[1].cpu().numpy()), x.shape, block_rows)
    assert np.all(np.abs(d - x) <= 1.0001 * np.maximum(np.abs(x) / 16, s * 2.0 ** -10)), what


@pytest.mark.parametrize("P,T,H,I,O,e8m0", [(2, 1, 256, 128, 128, False), (4, 33, 640, 384, 260, True), (3, 130, 1024, 200, 512, False),
                                            (8, 300, 512, 128, 256, True)])
def test_block_forward_and_backward(P, T, H, I, O, e8m0):
    note(f"block P={P} tokens={T} hidden={H} inner={I} outer={O} e8m0={e8m0}")
    b, row, col = tp_block.random_block(P, T, H, I, O, seed=P, e8m0=e8m0)
    b.forward()
    b.backward()
    torch.cuda.synchronize()
    for r in range(P):
        check_rounding(vals(row[r]), b.row_w[r], 128, "row-parallel weight")
        check_rounding(vals(col[r]).T, b.col_wt[r], 128, "column-parallel weight, transposed")
        check_rounding(vals(b.attn[r]), b.attn_q[r], 1, "activations")
        check_product(vals(b.parts[r]), deq(b.attn_q[r], 1), deq(b.row_w[r], 128), "rank buffer")
    h = ref.rank_sum([vals(p) for p in b.parts], vals(b.residual))
    assert np.array_equal(down16(b.hidden_out).ravel(), ref.bf16_bits(h).ravel()), "sum and residual"
    y = ref.norm(h, vals(b.gain[None])[0], b.eps)
    assert np.all(np.abs(vals(b.y) - y) <= 1.01 * ref.U16 * np.abs(y) + 1e-5), "norm"
    check_rounding(vals(b.d_outs[0]).T, b.d_qt[0], 1, "output gradient, transposed")
    for r in range(P):
        check_product(vals(b.outs[r]), deq(b.normed, 1), deq(b.col_w[r], 128), "column-parallel projection")
        check_product(b.d_col[r].double().cpu().numpy(), deq(b.d_qt[r], 1), deq(b.yt, 1), "gradient of a weight", bf16=False)
        check_product(vals(b.d_parts[r]), deq(b.d_q[r], 1), deq(b.col_wt[r], 128), "gradient of the norm's result")
    dy = ref.rank_sum([vals(p) for p in b.d_parts])
    assert np.array_equal(down16(b.d_normed).ravel(), ref.bf16_bits(dy).ravel()), "sum of the ranks' gradients"
    dx, dw = ref.norm_bwd(vals(b.d_normed), vals(b.hidden_out), vals(b.gain[None])[0], vals(b.d_hidden), b.eps)
    assert np.all(np.abs(vals(b.d_residual) - dx) <= 1.01 * ref.U16 * np.abs(dx) + 1e-5 * np.abs(dx).max()), "gradient of the residual"
    assert np.allclose(b.d_gain.cpu().numpy(), dw, rtol=1e-4, atol=1e-5 * np.abs(dw).max()), "gradient of the gain"


def test_block_gradient_against_differences():
    """Directional derivative of sum(d_outs . outs) + sum(d_hidden . hidden_out)
    along the residual, by differences of the unquantised step in 64 bits:
    8-bit operands leave a few percent of the gradient's size."""
    P, T, H, I, O = 2, 64, 512, 256, 384
    b, row, col = tp_block.random_block(P, T, H, I, O, seed=9)
    b.forward()
    b.backward()
    torch.cuda.synchronize()
    parts = [vals(a) @ vals(w).T for a, w in zip(b.attn, row)]
    gain, res = vals(b.gain[None])[0], vals(b.residual)

    def loss(x):
        h = sum(parts) + x
        y = ref.norm(h, gain, b.eps)
        return sum((vals(d) * (y @ vals(w).T)).sum() for d, w in zip(b.d_outs, col)) + (vals(b.d_hidden) * h).sum()

    g, got = np.random.default_rng(4), vals(b.d_residual)
    for _ in range(3):
        v = g.standard_normal(res.shape)
        num = (loss(res + 1e-4 * v) - loss(res - 1e-4 * v)) / 2e-4
        # errors of the elements are independent of v: their sum has the size of their root mean square
        assert abs(num - (got * v).sum()) <= 0.1 * 4 * np.linalg.norm(got), (num, (got * v).sum())


def test_block_in_a_graph():
    b, _, _ = tp_block.random_block(4, 24, 768, 512, 640, seed=3)
    b.forward()
    b.backward()
    results = (b.hidden_out, b.d_residual, b.d_gain, *b.outs, *b.d_col)
    torch.cuda.synchronize()
    want = [t.clone() for t in results]
    note("block captured in a graph")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.prepare(torch.cuda.current_stream())
        b.forward()
        b.backward()
    b.prepare()
    for k in range(3):
        for t in results:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, w) for x, w in zip(results, want)), k
        b.forward()
        b.backward()
        torch.cuda.synchronize()
        assert all(torch.equal(x, w) for x, w in zip(results, want)), k
