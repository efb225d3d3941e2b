"""The attention of one tensor-parallel block, on P simulated ranks.

    python -m tensor_all_reduce_amd.tp_attention [--step decode|prompt|train] [--tokens T] [--keys N] [--ranks P] [--e4m3]

What lies before the buffers that tp_block.TPBlock starts from: the
column-parallel projection of every rank (ar_gemm_fp8, all ranks in one call)
makes its queries, keys and values, ar_rope_kv rotates them by their positions
and, when serving, puts keys and values into the rank's pages, and attention
fills the rank's `attn` buffer:

  decode  one new token a sequence, ar_attn_decode over the pages
  prompt  the next chunks of ragged prompts, ar_attn_paged over the pages
  train   ragged sequences without pages, ar_attn; backward() takes the
          gradient of `attn` through ar_attn_bwd and the rotation back to the
          projection's result.  The caller fills that gradient: TPBlock's
          backward pass ends before the row-parallel projection

Every buffer is allocated once and every call prepared once; a step is a
handful of launches on one stream and can be captured in a HIP graph.  Run as
a command it times the step.
"""
from __future__ import annotations

import argparse

import tensor_all_reduce_amd as tar


class TPAttention:
    """Column-parallel weights [(hq + 2 hkv) dim, hidden] of P ranks (a rank's
    query heads, then its keys', then its values'), as bf16 matrices.

    Inputs: `normed` (codes and scales [tokens, hidden]), `positions`, and
    `cu` (first rows of the sequences; train, prompt), `table`, `lens` and
    `slots` (decode, prompt).  forward() -> `attn` (P x [tokens, hq dim]).
    backward() (train): `d_attn` -> `d_qkv` (P x [tokens, (hq + 2 hkv) dim]).
    All of these are this object's buffers; normed and attn may be given, so
    that they are a TPBlock's."""

    def __init__(self, weights, hq: int, hkv: int, dim: int, tokens: int, seqs: int, step: str = "decode", pages: int = 0,
                 page_size: int = 16, table_pages: int = 0, max_positions: int = 32768, rot=None, theta: float = 10000.0,
                 window: int = 0, sinks: int = 0, e4m3: bool = False, normed=None, attn=None):
        import torch

        if step not in ("decode", "prompt", "train"):
            raise ValueError(f"step must be decode, prompt or train, not {step!r}")
        if step == "decode" and tokens != seqs:
            raise ValueError("a decode step has one token a sequence")
        self.P, self.hq, self.hkv, self.dim, self.step = len(weights), int(hq), int(hkv), int(dim), step
        self.tokens, self.seqs, self.hidden = int(tokens), int(seqs), int(weights[0].shape[1])
        width, dev, T, bf = (self.hq + 2 * self.hkv) * self.dim, weights[0].device, self.tokens, torch.bfloat16
        self.mask = dict(window=int(window), sinks=int(sinks))
        self.weights = []
        for w in weights:
            m = tar.fp8_codes_empty(width, self.hidden, dev), tar.fp8_scales_empty(width, self.hidden, dev, 128)
            tar.ar_quantize_block(w, *m, block_rows=128)
            self.weights.append(m)

        def ints(n, dtype=torch.int32):
            return torch.zeros(n, device=dev, dtype=dtype)

        self.normed = normed or (tar.fp8_codes_empty(T, self.hidden, dev), tar.fp8_scales_empty(T, self.hidden, dev))
        self.qkv = [torch.empty(T, width, device=dev, dtype=bf) for _ in weights]
        self.attn = attn or [torch.empty(T, self.hq * self.dim, device=dev, dtype=bf) for _ in weights]
        self.cos_sin = tar.rope_table(max_positions, self.dim if rot is None else rot, theta, dev)
        self.positions, self.cu = ints(T), ints(self.seqs + 1)
        if step == "train":
            self.d_attn, self.d_qkv = ([torch.empty_like(t) for t in x] for x in (self.attn, self.qkv))
            self.lse = [torch.empty(self.hq, T, device=dev).t() for _ in weights]
            size = tar.attn_bwd_workspace(T, T, self.seqs, self.hq, self.hkv, self.dim, **self.mask)
        else:
            self.caches = [tar.kv_cache_empty(pages, page_size, self.hkv, self.dim, dev, e4m3) for _ in weights]
            self.table = torch.zeros(self.seqs, int(table_pages), device=dev, dtype=torch.int32)
            self.lens, self.slots = ints(self.seqs), ints(T, torch.int64)
            size = tar.attn_decode_workspace(self.seqs, self.hq, self.hkv, self.dim) if step == "decode" else 0
        # one workspace each for attention and the projection: the calls follow each other on one stream
        self.workspace = torch.zeros(size, device=dev, dtype=torch.uint8)
        self.gemm_workspace = torch.zeros(tar.gemm_fp8_workspace(T, width, self.hidden, self.P), device=dev, dtype=torch.uint8)
        self.prepare()

    def heads(self, rows):
        """(queries, keys, values) of a rank's projection result, [tokens, heads, dim] each."""
        x = rows.view(self.tokens, self.hq + 2 * self.hkv, self.dim)
        return x[:, :self.hq], x[:, self.hq:self.hq + self.hkv], x[:, self.hq + self.hkv:]

    def prepare(self, stream=None):
        """Marshals every call of the step for `stream` (the current one if
        None), on which forward() and backward() then run."""
        kw = dict(stream=stream)
        self._forward = [tar.prepare(tar.ar_gemm_fp8, [self.normed[0]] * self.P, [self.normed[1]] * self.P,
                                     [m[0] for m in self.weights], [m[1] for m in self.weights], self.qkv,
                                     workspace=self.gemm_workspace, **kw)]
        self._backward = []
        for r in range(self.P):
            q, k, v = self.heads(self.qkv[r])
            out = self.attn[r].view(self.tokens, self.hq, self.dim)
            if self.step == "train":
                self._forward += [
                    tar.prepare(tar.ar_rope_kv, q, k, None, self.cos_sin, self.positions, q_out=q, k_out=k, **kw),
                    tar.prepare(tar.ar_attn, q, k, v, self.cu, self.cu, out, lse=self.lse[r], **self.mask, **kw)]
                dq, dk, dv = self.heads(self.d_qkv[r])
                self._backward += [
                    tar.prepare(tar.ar_attn_bwd, q, k, v, out, self.lse[r], self.d_attn[r].view_as(out), self.cu, self.cu,
                                dq=dq, dk=dk, dv=dv, workspace=self.workspace, **self.mask, **kw),
                    tar.prepare(tar.ar_rope_kv, dq, dk, None, self.cos_sin, self.positions, q_out=dq, k_out=dk, inverse=True, **kw)]
                continue
            self._forward.append(tar.prepare(tar.ar_rope_kv, q, k, v, self.cos_sin, self.positions, q_out=q, cache=self.caches[r],
                                             slots=self.slots, **kw))
            if self.step == "decode":
                self._forward.append(tar.prepare(tar.ar_attn_decode, q, self.caches[r], self.table, self.lens, out,
                                                 workspace=self.workspace, **self.mask, **kw))
            else:
                self._forward.append(tar.prepare(tar.ar_attn_paged, q, self.caches[r], self.table, self.lens, self.cu, out,
                                                 **self.mask, **kw))

    def forward(self):
        for call in self._forward:
            call()

    def backward(self):
        if self.step != "train":
            raise ValueError("only a training step has gradients")
        for call in self._backward:
            call()


def random_attention(P: int, tokens: int, seqs: int, hidden: int, hq: int, hkv: int, dim: int, step: str, keys: int = 0, seed: int = 0,
                     page_size: int = 16, device: str = "cuda:0", **kw):
    """Attention of random weights with random inputs: sequences of equal
    length, with `keys` earlier tokens each in random pages (decode, prompt)."""
    import torch
    g = torch.Generator(device=device)
    g.manual_seed(seed)

    def normal(*shape, std=1.0):
        return (std * torch.randn(*shape, generator=g, device=device)).to(torch.bfloat16)

    width, each = (hq + 2 * hkv) * dim, tokens // seqs
    if each * seqs != tokens:
        raise ValueError("tokens must be a multiple of seqs")
    need = -(-(keys + each) // page_size)
    a = TPAttention([normal(width, hidden, std=hidden ** -0.5) for _ in range(P)], hq, hkv, dim, tokens, seqs, step,
                    pages=seqs * need, page_size=page_size, table_pages=need, max_positions=keys + each, **kw)
    tar.ar_quantize_block(normal(tokens, hidden), *a.normed)
    at = torch.arange(tokens, device=device)
    seq, pos = at // each, keys + at % each
    a.positions.copy_(pos)
    a.cu.copy_(torch.arange(seqs + 1, device=device) * each)
    if step == "train":
        for t in a.d_attn:
            t.copy_(normal(*t.shape, std=0.01))
        return a
    a.table.copy_(torch.randperm(seqs * need, generator=g, device=device).view(seqs, need))
    a.lens.fill_(keys + each)
    a.slots.copy_(a.table[seq, pos // page_size].long() * page_size + pos % page_size)
    for cache in a.caches:
        for t in cache:
            t.copy_(normal(*t.shape).float().abs() + 0.1 if t.dim() == 3 else normal(*t.shape))
    return a


def main(argv=None) -> int:
    import time

    import torch

    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--step", choices=("decode", "prompt", "train"), default="decode")
    ap.add_argument("--tokens", type=int, default=32)
    ap.add_argument("--seqs", type=int, default=0, help="sequences (default: one a token when decoding, else one)")
    ap.add_argument("--keys", type=int, default=4096, help="earlier tokens of each sequence")
    ap.add_argument("--hidden", type=int, default=8192)
    ap.add_argument("--heads", type=int, default=8, help="query heads of a rank")
    ap.add_argument("--kv-heads", type=int, default=1, help="key heads of a rank")
    ap.add_argument("--dim", type=int, default=128)
    ap.add_argument("--ranks", type=int, default=8)
    ap.add_argument("--window", type=int, default=0)
    ap.add_argument("--sinks", type=int, default=0)
    ap.add_argument("--e4m3", action="store_true", help="keys and values in 8 bits")
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args(argv)
    seqs = a.seqs or (a.tokens if a.step == "decode" else 1)
    keys = 0 if a.step == "train" else a.keys
    t = random_attention(a.ranks, a.tokens, seqs, a.hidden, a.heads, a.kv_heads, a.dim, a.step, keys, e4m3=a.e4m3, window=a.window,
                         sinks=a.sinks)
    for name, run in (("forward", t.forward), ("backward", t.backward)):
        if name == "backward" and a.step != "train":
            break
        for _ in range(3):
            run()
        torch.cuda.synchronize()
        s = time.perf_counter()
        for _ in range(a.steps):
            run()
        torch.cuda.synchronize()
        print(f"{name}: {(time.perf_counter() - s) / a.steps * 1e6:.1f} us", flush=True)
    return 0


if __name__ == "__main__":
    raise SystemExit(main())
