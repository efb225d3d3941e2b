"""Prompts over pages of which one has a number out of range: the queries that
see a key of it have no result, all others what they have without it."""
import pytest
import torch

import attn_ref as ref
import tensor_all_reduce_amd as tar
from gpu_util import note
from test_gpu_attn import cu, gen, heads
from test_gpu_attn_cache import filled, tables

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("new,hq,hkv,dim", [([200, 70], 4, 2, 128), ([130, 1], 2, 1, 80), ([2048, 3], 24, 4, 64), ([2100, 40], 64, 8, 128)])
def test_only_readers_of_a_bad_page_lose_their_result(new, hq, hkv, dim, e4m3):
    """Few workgroups, 128 queries in four waves, 256 in eight."""
    note(f"bad page {new} {hq}/{hkv}x{dim} e4m3 {e4m3}")
    g, page, past = gen(sum(new)), 16, 100
    total = [n + past for n in new]
    table, pages = tables(g, total, page)
    cache = filled(g, pages, page, hkv, dim, e4m3)
    q, offs = heads(g, sum(new), hq, dim), cu(new)
    lens = torch.tensor(total, device=DEV, dtype=torch.int32)
    keep = table.clone()
    for window, sinks, at in ((0, 0, 9), (0, 0, (total[0] - 1) // page), (64, 0, 9), (64, 40, 2), (64, 4, 2), (20, 200, 0)):
        res = []
        for bad in (None, -1, pages, 2 ** 31 - 1):
            table.copy_(keep)
            if bad is not None:
                table[0, at] = bad
            out, lse = torch.full_like(q, 7.0), torch.full((len(q), hq), 7.0, device=DEV)
            tar.ar_attn_paged(q, cache, table, lens, offs, out, window=window, sinks=sinks, lse=lse)
            torch.cuda.synchronize()
            res.append((out, lse))
        p = past + torch.arange(new[0], device=DEV)[:, None]
        j = torch.arange(at * page, min((at + 1) * page, total[0]), device=DEV)[None]
        sees = j <= p
        if window:
            sees &= (j > p - window) | (j < sinks)
        lost = torch.zeros(len(q), device=DEV, dtype=torch.bool)
        lost[:new[0]] = sees.any(1)
        # The others within the bounds of a result, not bit for bit: a wave's
        # queries follow their running maxima together, whenever one has to,
        # and a numerator's last bits depend on the maximum.
        k, v = ref.paged(cache, keep[0], total[0])
        rows = ~lost[:new[0]]
        for out, lse in res[1:]:
            what = f"page {at}, window {window}, sinks {sinks}"
            assert bool(out[lost].isnan().all()) and bool(lse[lost].isnan().all()), what
            assert torch.equal(out[new[0]:], res[0][0][new[0]:]) and torch.equal(lse[new[0]:], res[0][1][new[0]:]), what
            for h in (0, hq - 1):
                want = ref.attend(q[:new[0], h], k[:, h // (hq // hkv)], v[:, h // (hq // hkv)], dim ** -0.5, window, sinks)
                ref.close(out[:new[0], h][rows], want["out"][rows], want["out_t"][rows], "out, " + what)
                ref.close(lse[:new[0], h][rows], want["lse"][rows], want["lse_t"][rows], "lse, " + what)
