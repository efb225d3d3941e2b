"""Gradients where tiles with sinks have their far queries cut into runs, for
heads of more than 64."""
import pytest

from gpu_util import note
from test_gpu_attn import cu, gen, heads
from test_gpu_attn_edges import check, step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,dim,sinks,window", [(2, 1, 128, 3, 100), (2, 2, 80, 200, 100), (1, 1, 128, 4097, 30), (3, 1, 112, 1, 2100)])
def test_far_queries_of_sinks(hq, hkv, dim, sinks, window):
    note(f"far {hq}/{hkv}x{dim} sinks {sinks} window {window}")
    g, lengths = gen(dim + sinks), [2300, 30, 4200, 2049, 0, 2048]
    n, offs = sum(lengths), cu(lengths)
    q, k, v, go = (heads(g, n, h, dim) for h in (hq, hkv, hkv, hq))
    check(step(q, k, v, offs, offs, go, window, sinks), q, k, v, offs, offs, go, window, sinks)


def test_far_queries_with_keys_before_them():
    note("far, keys before")
    g, nq, nk, hq, hkv, dim = gen(7), [2100, 4100, 5], [2600, 4000, 3000], 2, 1, 128
    a, b = cu(nq), cu(nk)
    q, go = heads(g, sum(nq), hq, dim), heads(g, sum(nq), hq, dim)
    k, v = heads(g, sum(nk), hkv, dim), heads(g, sum(nk), hkv, dim)
    check(step(q, k, v, a, b, go, 150, 140), q, k, v, a, b, go, 150, 140)
