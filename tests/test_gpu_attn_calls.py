"""Calls that the documentation allows beside the usual ones: more sequences
than a wave has lanes, sinks without a window, results over the queries,
workspaces of any contents."""
import math

import pytest
import torch

import attn_ref as ref
import tensor_all_reduce_amd as tar
from gpu_util import note
from test_gpu_attn import cu, gen, heads
from test_gpu_attn_cache import filled, normal, tables
from test_gpu_attn_edges import check, step

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3), (100, 130)])
@pytest.mark.parametrize("dim", [64, 128])
def test_many_sequences(dim, window, sinks):
    note(f"many sequences of {dim}, window {window} sinks {sinks}")
    g = gen(window + dim)
    lengths = [(i * 29) % 90 if i % 7 else 0 for i in range(150)]
    lengths[70], lengths[140] = 2500, 4200              # with far queries of sinks
    n, offs = sum(lengths), cu(lengths)
    q, k, v, go = (heads(g, n, h, dim) for h in (2, 1, 1, 2))
    check(step(q, k, v, offs, offs, go, window, sinks), q, k, v, offs, offs, go, window, sinks)


def test_many_sequences_in_pages():
    note("many sequences in pages")
    g, page, hq, hkv, dim = gen(3), 16, 4, 2, 80
    new = [(i * 13) % 40 for i in range(130)]
    total = [n + (i * 31) % 300 for i, n in enumerate(new)]
    table, pages = tables(g, total, page)
    for e4m3 in (False, True):
        cache = filled(g, pages, page, hkv, dim, e4m3)
        q, offs = heads(g, sum(new), hq, dim), cu(new)
        out = torch.empty_like(q)
        tar.ar_attn_paged(q, cache, table, torch.tensor(total, device=DEV, dtype=torch.int32), offs, out, window=90, sinks=2)
        torch.cuda.synchronize()
        for i in range(0, 130, 3):
            a = slice(int(offs[i]), int(offs[i + 1]))
            k, v = ref.paged(cache, table[i], total[i])
            for h in (0, hq - 1):
                want = ref.attend(q[a, h], k[:, h // 2], v[:, h // 2], dim ** -0.5, 90, 2)
                ref.close(out[a, h], want["out"], want["out_t"], f"sequence {i}, head {h}, e4m3 {e4m3}")


def test_sinks_without_a_window():
    """Nothing but the causal mask."""
    note("sinks, no window")
    g, lengths = gen(4), [300, 2200, 5]
    offs = cu(lengths)
    q, k, v, go = (heads(g, sum(lengths), h, 64) for h in (4, 2, 2, 4))
    a, b = step(q, k, v, offs, offs, go), step(q, k, v, offs, offs, go, 0, 7)
    for x in a:
        assert torch.equal(a[x], b[x]), x
    table, pages = tables(g, lengths, 16)
    cache = filled(g, pages, 16, 2, 64, False)
    lens = torch.tensor(lengths, device=DEV, dtype=torch.int32)
    res = []
    for sinks in (0, 7):
        one, out = torch.empty_like(q[:3]), torch.empty_like(q)
        tar.ar_attn_decode(q[:3], cache, table, lens, one, sinks=sinks)
        tar.ar_attn_paged(q, cache, table, lens, offs, out, sinks=sinks)
        res.append((one, out))
    torch.cuda.synchronize()
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("hq,hkv,dim,e4m3", [(40, 2, 128, False), (8, 8, 64, True), (8, 1, 80, False)])
def test_results_over_the_queries(hq, hkv, dim, e4m3, odd):
    """Sequences cut among workgroups, and passes made again (odd)."""
    note(f"in place {hq}/{hkv}x{dim} e4m3 {e4m3} odd {odd}")
    g, lengths = gen(dim), [5000, 3, 0, 900, 20000]
    table, pages = tables(g, lengths, 16)
    cache = filled(g, pages, 16, hkv, dim, e4m3)
    if odd:
        v = cache[1].view(torch.uint8) if e4m3 else cache[1]
        v[table[0, 200], 5, :, 3] = 0x7F if e4m3 else math.inf
        v[table[4, 900], 5, :, 7] = 0x7F if e4m3 else math.nan
    lens = torch.tensor(lengths, device=DEV, dtype=torch.int32)
    ws = torch.zeros(tar.attn_decode_workspace(5, hq, hkv, dim), device=DEV, dtype=torch.uint8)
    q = normal(g, 5, hq, dim).to(torch.bfloat16)
    for w in (ws, None):
        out, over = torch.empty_like(q), q.clone()
        tar.ar_attn_decode(q, cache, table, lens, out, workspace=w)
        tar.ar_attn_decode(over, cache, table, lens, over, workspace=w)
        torch.cuda.synchronize()
        assert torch.equal(out.nan_to_num(9.0), over.nan_to_num(9.0)) and torch.equal(out.isnan(), over.isnan())
    new = [64, 3, 0, 300, 130]
    offs, q = cu(new), heads(g, sum(new), hq, dim)
    out, over = torch.empty_like(q), q.clone()
    tar.ar_attn_paged(q, cache, table, lens, offs, out)
    tar.ar_attn_paged(over, cache, table, lens, offs, over)
    torch.cuda.synchronize()
    assert torch.equal(out.nan_to_num(9.0), over.nan_to_num(9.0)) and torch.equal(out.isnan(), over.isnan())


def test_workspaces_of_any_contents():
    """The gradients' workspace, and all but the counters of the single tokens'."""
    note("workspaces")
    g, lengths, hq, hkv, dim = gen(6), [2500, 90, 0, 2100], 4, 2, 64
    n, offs = sum(lengths), cu(lengths)
    q, k, v, go = (heads(g, n + 7, h, dim) for h in (hq, hkv, hkv, hq))
    out, lse = torch.empty_like(q), torch.empty(n + 7, hq, device=DEV)
    tar.ar_attn(q, k, v, offs, offs, out, lse=lse, window=50, sinks=5)
    out[n:], lse[n:] = math.nan, math.nan             # rows of no sequence
    size = tar.attn_bwd_workspace(n + 7, n + 7, len(lengths), hq, hkv, dim, 50, 5)
    res = []
    for fill in (0, 255):
        ws = torch.full((size,), fill, device=DEV, dtype=torch.uint8)
        d = [torch.full_like(x, 7.0) for x in (q, k, v)]
        tar.ar_attn_bwd(q, k, v, out, lse, go, offs, offs, dq=d[0], dk=d[1], dv=d[2], workspace=ws, window=50, sinks=5)
        res.append(d)
    torch.cuda.synchronize()
    for x, y in zip(*res):
        assert torch.equal(x, y) and bool((x[n:] == 7.0).all()) and bool(torch.isfinite(x).all())
    table, pages = tables(g, lengths, 16)
    cache = filled(g, pages, 16, hkv, dim, False)
    lens = torch.tensor(lengths, device=DEV, dtype=torch.int32)
    size = tar.attn_decode_workspace(4, hq, hkv, dim)
    counters = -(-4 * hkv * 4 // 256) * 256            # at the end
    res = []
    for fill in (0, 255):
        ws = torch.full((size,), fill, device=DEV, dtype=torch.uint8)
        ws[size - counters:] = 0
        o = torch.empty_like(q[:4])
        tar.ar_attn_decode(q[:4], cache, table, lens, o, workspace=ws)
        res.append(o)
    torch.cuda.synchronize()
    assert torch.equal(*res) and bool(torch.isfinite(res[0]).all())


@pytest.mark.parametrize("power", [-64, -40, 40, 64])
def test_scales_far_from_one(power):
    """Queries and keys as large or small as the scale makes up for."""
    note(f"scale 2^{power}")
    g, lengths, hq, hkv, dim = gen(8), [200, 33], 4, 2, 64
    n, offs, by = sum(lengths), cu(lengths), 2.0 ** (-power // 2 - 1)
    q, k, v, go = (heads(g, n, h, dim) for h in (hq, hkv, hkv, hq))
    q, k, scale = q * by, k * by, 2.0 ** power            # exact; scores of 2^-2 q . k
    out, lse = torch.empty_like(q), torch.empty(n, hq, device=DEV)
    tar.ar_attn(q, k, v, offs, offs, out, scale=scale, lse=lse)
    ws = torch.empty(tar.attn_bwd_workspace(n, n, 2, hq, hkv, dim), device=DEV, dtype=torch.uint8)
    d = [torch.empty_like(x) for x in (q, k, v)]
    tar.ar_attn_bwd(q, k, v, out, lse, go, offs, offs, dq=d[0], dk=d[1], dv=d[2], workspace=ws, scale=scale)
    torch.cuda.synchronize()
    want = ref.ragged(q, k, v, offs.tolist(), offs.tolist(), scale, 0, 0, go)
    for x, y in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *d)):
        ref.close(y, want[x], want[x + "_t"], x)
    table, pages = tables(g, lengths, 16)
    cache = filled(g, pages, 16, hkv, dim, False)
    cache[0].mul_(by)
    one = torch.empty_like(q[:2])
    tar.ar_attn_decode(q[:2], cache, table, torch.tensor(lengths, device=DEV, dtype=torch.int32), one, scale=scale)
    torch.cuda.synchronize()
    for i, m in enumerate(lengths):
        kk, vv = ref.paged(cache, table[i], m)
        for h in range(hq):
            w = ref.attend(q[i:i + 1, h], kk[:, h // 2], vv[:, h // 2], scale)
            ref.close(one[i:i + 1, h], w["out"], w["out_t"], "single token")
