"""Where the kernels take a rounding less than elsewhere: single tokens'
numerators, and the gradients of queries that see up to 256 keys, whatever
lies before them or beside them in a tile."""
import pytest
import torch

import attn_ref as ref
import attn_tight as tight
import tensor_all_reduce_amd as tar
from gpu_util import note
from test_attn_tight import cancelling
from test_gpu_attn import cu, gen, heads
from test_gpu_attn_cache import tables

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("nq,nk,window,sinks", [(300, 300, 0, 0), (300, 308, 0, 0), (250, 256, 0, 0), (300, 130, 0, 0), (600, 400, 0, 0),
                                                (600, 650, 100, 4), (520, 900, 256, 0)])
@pytest.mark.parametrize("dim", [64, 128])
def test_gradients_of_queries_with_few_keys(dim, nq, nk, window, sinks):
    note(f"few keys {nq} / {nk} of {dim}, window {window}")
    g, h = gen(nq + nk), 2
    q, go = heads(g, nq, h, dim), heads(g, nq, h, dim)
    k, v = heads(g, nk, h, dim), (64 + torch.randn(nk, h, dim, generator=g, device=DEV)).to(torch.bfloat16)
    out, lse = torch.empty_like(q), torch.empty(nq, h, device=DEV)
    a, b = cu([nq]), cu([nk])
    tar.ar_attn(q, k, v, a, b, out, lse=lse, window=window, sinks=sinks)
    dq, dk, dv = (torch.empty_like(x) for x in (q, k, v))
    ws = torch.empty(tar.attn_bwd_workspace(nq, nk, 1, h, h, dim, window, sinks), device=DEV, dtype=torch.uint8)
    tar.ar_attn_bwd(q, k, v, out, lse, go, a, b, dq=dq, dk=dk, dv=dv, workspace=ws, window=window, sinks=sinks)
    torch.cuda.synchronize()
    few = ref.visible(nq, nk, window, sinks, DEV).sum(1) <= 256
    assert bool(few[:50].all())
    for x in range(h):
        want = tight.grad_bounds(q[:, x], k[:, x], v[:, x], dim ** -0.5, go[:, x], window, sinks)
        ref.close(dq[:, x][few], want["dq"][few], want["dq_t"][few], f"dq, head {x}")
        if bool(few.all()):
            ref.close(dk[:, x], want["dk"], want["dk_t"], f"dk, head {x}")


@pytest.mark.parametrize("cut", [False, True])
@pytest.mark.parametrize("keys", [24, 130, 700])
@pytest.mark.parametrize("dim", [64, 128])
def test_single_tokens_numerators(dim, keys, cut):
    """Values of which the softmax leaves hardly anything."""
    note(f"numerators {keys} of {dim}, cut {cut}")
    g, h, page = gen(keys), 4, 16
    table, pages = tables(g, [keys], page)
    cache = tar.kv_cache_empty(pages, page, h, dim, DEV)
    q, k = heads(g, 1, h, dim, 0.25), heads(g, keys, h, dim)
    v = torch.stack([cancelling(g, keys, dim, q[:, x], k[:, x], dim ** -0.5) for x in range(h)], 1)
    j = torch.arange(keys, device=DEV)
    for c, x in zip(cache, (k, v)):
        c[table[0].long()[j // page], j % page] = x
    ws = torch.zeros(tar.attn_decode_workspace(1, h, h, dim), device=DEV, dtype=torch.uint8)
    out = torch.empty_like(q)
    tar.ar_attn_decode(q, cache, table, torch.tensor([keys], device=DEV, dtype=torch.int32), out, workspace=ws if cut else None)
    torch.cuda.synchronize()
    for x in range(h):
        want = ref.attend(q[:, x], k[:, x], v[:, x], dim ** -0.5)
        ref.close(out[:, x], want["out"], tight.out_bound(q[:, x], k[:, x], v[:, x], dim ** -0.5), f"head {x}")
