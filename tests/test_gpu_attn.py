"""Attention of ragged prompts and its gradients against 64 bits, within bounds
that count the kernels' roundings (attn_ref)."""
import pytest
import torch

import attn_ref as ref
import tensor_all_reduce_amd as tar
from gpu_util import note

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def heads(g, rows, h, dim, std=1.0):
    return (std * torch.randn(rows, h, dim, generator=g, device=DEV)).to(torch.bfloat16)


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def cu(lengths):
    return torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], device=DEV, dtype=torch.int32)


MASKS = [(0, 0), (1, 0), (37, 3), (64, 64), (200, 1), (10000, 4)]
LENGTHS = [[1], [2, 0, 63], [64, 65, 1], [255, 256, 257], [700]]


@pytest.mark.parametrize("window,sinks", MASKS)
@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("hq,hkv,dim", [(4, 2, 64), (3, 3, 128), (5, 1, 80)])
def test_forward_and_gradients(hq, hkv, dim, lengths, window, sinks):
    note(f"attn {hq}/{hkv}x{dim} {lengths} window {window} sinks {sinks}")
    g = gen(hash((hq, dim, sum(lengths), window)) % 1000)
    n, spare = sum(lengths), 3                       # rows behind the last sequence
    q, k, v, go = (heads(g, n + spare, h, dim) for h in (hq, hkv, hkv, hq))
    out = torch.full_like(q, 7.0)
    lse = torch.full((n + spare, hq), 7.0, device=DEV)
    offs = cu(lengths)
    scale = dim ** -0.5
    tar.ar_attn(q, k, v, offs, offs, out, window=window, sinks=sinks, lse=lse)
    dq, dk, dv = (torch.full_like(x, 7.0) for x in (q, k, v))
    ws = torch.empty(tar.attn_bwd_workspace(n + spare, n + spare, len(lengths), hq, hkv, dim, window, sinks), device=DEV,
                     dtype=torch.uint8)
    tar.ar_attn_bwd(q, k, v, out, lse, go, offs, offs, dq=dq, dk=dk, dv=dv, workspace=ws, window=window, sinks=sinks)
    torch.cuda.synchronize()
    want = ref.ragged(q, k, v, offs.tolist(), offs.tolist(), scale, window, sinks, go)
    got = dict(out=out, lse=lse, dq=dq, dk=dk, dv=dv)
    for x, y in got.items():
        ref.close(y, want[x], want[x + "_t"], x)
        assert bool((y[n:] == 7.0).all()), f"{x}: rows of no sequence were written"
