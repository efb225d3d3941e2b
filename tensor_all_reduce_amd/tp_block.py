"""One tensor-parallel step around the all-reduce, on P simulated ranks.

    python -m tensor_all_reduce_amd.tp_block [--tokens T] [--hidden H] [--inner I] [--ranks P] [--e8m0]

The forward step is what a transformer block does between two projections:
the row-parallel projection of every rank (ar_gemm_fp8, all ranks in one
call) gives the rank buffers, ar_reduce_norm sums them, adds the residual and
norms the sum into 8 bits, and the column-parallel projection of every rank
takes those codes.  The backward step returns the gradients of the residual
stream, of the norm's gain and of the column-parallel weights:
ar_quantize_block quantises the output gradients, as they stand for the
gradient of the codes and transposed for the weights', ar_gemm_fp8 makes both,
ar_reduce_oneshot sums the ranks' gradients and ar_norm_bwd takes them
through the norm.

Every buffer is allocated once and every call prepared once, so a step is
a handful of launches on one stream and can be captured in a HIP graph.
Run as a command it times both steps.
"""
from __future__ import annotations

import argparse

import tensor_all_reduce_amd as tar


class TPBlock:
    """Row-parallel weights [hidden, inner / P], column-parallel weights
    [outer / P, hidden] of P ranks, as bf16 matrices; norm gains [hidden].

    forward(): `attn` (P bf16 matrices [tokens, inner / P]) and `residual`
    [tokens, hidden] -> `hidden_out` (bf16) and `outs` (P x [tokens, outer / P]).
    backward(): `d_outs` and `d_hidden` -> `d_residual` (bf16, the gradient of
    the residual and of every rank's contribution), `d_gain` and `d_col`
    (binary32).  All of these are this object's buffers: write the inputs
    into them and read the results from them."""

    def __init__(self, row_weights, col_weights, gain, tokens: int, eps: float = 1e-6, e8m0: bool = False):
        import torch

        self.P, self.tokens = len(row_weights), int(tokens)
        self.hidden, self.inner = map(int, row_weights[0].shape)
        self.outer, dev = int(col_weights[0].shape[0]), row_weights[0].device
        T, H, bf = self.tokens, self.hidden, torch.bfloat16
        self.gain, self.ranks = gain, range(self.P)
        codes, scales = tar.fp8_codes_empty, tar.fp8_scales_empty

        def matrix(rows, cols, block_rows=1):
            return codes(rows, cols, dev), scales(rows, cols, dev, block_rows, e8m0)

        def each(rows, cols, block_rows=1):
            return [matrix(rows, cols, block_rows) for _ in self.ranks]

        def dense(rows, cols, dtype=bf):
            return [torch.empty(rows, cols, device=dev, dtype=dtype) for _ in self.ranks]

        # weights, quantised once in 128 x 128 blocks; the column-parallel
        # ones transposed as well, for the gradient of their input
        self.row_w, self.col_w, self.col_wt = each(H, self.inner, 128), each(self.outer, H, 128), each(H, self.outer, 128)
        for r in self.ranks:
            tar.ar_quantize_block(row_weights[r], *self.row_w[r], block_rows=128)
            tar.ar_quantize_block(col_weights[r], *self.col_w[r], block_rows=128)
            tar.ar_quantize_block(col_weights[r], *self.col_wt[r], block_rows=128, transpose=True)

        self.attn, self.parts, self.outs = dense(T, self.inner), dense(T, H), dense(T, self.outer)
        self.residual, self.hidden_out = (torch.empty(T, H, device=dev, dtype=bf) for _ in range(2))
        self.attn_q, self.normed = each(T, self.inner), matrix(T, H)

        self.d_outs, self.d_parts = dense(T, self.outer), dense(T, H)
        self.d_col = dense(self.outer, H, torch.float32)
        self.d_hidden, self.d_normed, self.d_residual, self.y = (torch.empty(T, H, device=dev, dtype=bf) for _ in range(4))
        self.d_gain = torch.empty(H, device=dev, dtype=torch.float32)
        self.d_q, self.d_qt, self.yt = each(T, self.outer), each(self.outer, T), matrix(H, T)

        # one workspace: the calls follow each other on one stream
        sizes = [tar.gemm_fp8_workspace(T, H, self.inner, self.P), tar.gemm_fp8_workspace(T, self.outer, H, self.P),
                 tar.gemm_fp8_workspace(T, H, self.outer, self.P), tar.gemm_fp8_workspace(self.outer, H, T, self.P)]
        self.workspace = torch.zeros(max(sizes), device=dev, dtype=torch.uint8)
        self.sums = torch.empty(tar.norm_bwd_workspace(T, H), device=dev, dtype=torch.uint8)
        self.eps = eps
        self.prepare()

    def prepare(self, stream=None):
        """Marshals every call of the two steps for `stream` (the current
        one if None), on which forward() and backward() then run."""

        def quantise(x, m, transpose=False):
            return tar.prepare(tar.ar_quantize_block, x, *m, transpose=transpose, stream=stream)

        def product(a, b, outs, block_rows=128):
            return tar.prepare(tar.ar_gemm_fp8, [m[0] for m in a], [m[1] for m in a], [m[0] for m in b], [m[1] for m in b],
                               outs, b_block_rows=block_rows, workspace=self.workspace, stream=stream)

        self._forward = [
            *(quantise(self.attn[r], self.attn_q[r]) for r in self.ranks),
            product(self.attn_q, self.row_w, self.parts),
            # the bf16 norm is kept for the weights' gradient
            tar.prepare(tar.ar_reduce_norm, self.parts, self.gain, residual=self.residual, res_out=self.hidden_out,
                        y=self.y, codes=self.normed[0], scales=self.normed[1], eps=self.eps, stream=stream),
            product([self.normed] * self.P, self.col_w, self.outs),
        ]
        self._backward = [
            *(quantise(self.d_outs[r], self.d_q[r]) for r in self.ranks),
            *(quantise(self.d_outs[r], self.d_qt[r], transpose=True) for r in self.ranks),
            quantise(self.y, self.yt, transpose=True),
            product(self.d_qt, [self.yt] * self.P, self.d_col, block_rows=1),
            product(self.d_q, self.col_wt, self.d_parts),
            tar.prepare(tar.ar_reduce_oneshot, self.d_parts, self.d_normed, stream=stream),
            tar.prepare(tar.ar_norm_bwd, self.d_normed, self.hidden_out, self.gain, dx=self.d_residual,
                        dres=self.d_hidden, dweight=self.d_gain, workspace=self.sums, eps=self.eps, stream=stream),
        ]

    def forward(self):
        for call in self._forward:
            call()

    def backward(self):
        for call in self._backward:
            call()


def random_block(P: int, tokens: int, hidden: int, inner: int, outer: int, seed: int = 0, e8m0: bool = False,
                 device: str = "cuda:0"):
    """A block of random weights with random inputs in its buffers, and the
    bf16 weights it was made from."""
    import torch
    g = torch.Generator(device=device)
    g.manual_seed(seed)

    def normal(rows, cols, std=1.0):
        return (std * torch.randn(rows, cols, generator=g, device=device)).to(torch.bfloat16)

    row = [normal(hidden, inner, inner ** -0.5) for _ in range(P)]
    col = [normal(outer, hidden, hidden ** -0.5) for _ in range(P)]
    gain = (1 + 0.1 * torch.randn(hidden, generator=g, device=device)).to(torch.bfloat16)
    block = TPBlock(row, col, gain, tokens, e8m0=e8m0)
    for t in (*block.attn, block.residual):
        t.copy_(normal(*t.shape))
    for t in (*block.d_outs, block.d_hidden):
        t.copy_(normal(*t.shape, 0.01))
    return block, row, col


def main(argv=None) -> int:
    import time

    import torch

    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=8192)
    ap.add_argument("--inner", type=int, default=1024, help="columns of a rank's row-parallel weight")
    ap.add_argument("--outer", type=int, default=1024, help="rows of a rank's column-parallel weight")
    ap.add_argument("--ranks", type=int, default=8)
    ap.add_argument("--e8m0", action="store_true", help="power-of-two scales")
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args(argv)
    block, _, _ = random_block(a.ranks, a.tokens, a.hidden, a.inner, a.outer, e8m0=a.e8m0)
    flops = 2 * a.ranks * a.tokens * a.hidden
    for name, step, work in (("forward", block.forward, flops * (a.inner + a.outer)), ("backward", block.backward, 2 * flops * a.outer)):
        for _ in range(3):
            step()
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(a.steps):
            step()
        torch.cuda.synchronize()
        t = (time.perf_counter() - t) / a.steps
        print(f"{name}: {t * 1e6:.1f} us, {work / t / 1e12:.0f} TFLOP/s over all ranks", flush=True)
    return 0


if __name__ == "__main__":
    raise SystemExit(main())
