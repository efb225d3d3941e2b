"""Attention where it can go wrong: masked places that hold no numbers, far
queries of sinks, queries and keys of different counts, strides, offsets
beyond 32 bits, bad pages, graphs and streams."""
import math

import pytest
import torch

import attn_ref as ref
import tensor_all_reduce_amd as tar
from gpu_util import note
from test_gpu_attn import cu, gen, heads
from test_gpu_attn_cache import filled, normal, tables

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def step(q, k, v, offs_q, offs_k, go, window=0, sinks=0, outs=None, stream=None):
    """Forward and backward pass; a dict of results."""
    hq, hkv, dim = q.shape[1], k.shape[1], q.shape[2]
    out, dq, dk, dv = outs or (torch.full_like(q, 7.0), torch.full_like(q, 7.0), torch.full_like(k, 7.0), torch.full_like(v, 7.0))
    lse = torch.full((hq, q.shape[0]), 7.0, device=DEV).t()
    ws = torch.empty(tar.attn_bwd_workspace(len(q), len(k), len(offs_q) - 1, hq, hkv, dim, window, sinks), device=DEV,
                     dtype=torch.uint8)
    tar.ar_attn(q, k, v, offs_q, offs_k, out, window=window, sinks=sinks, lse=lse, stream=stream)
    tar.ar_attn_bwd(q, k, v, out, lse, go, offs_q, offs_k, dq=dq, dk=dk, dv=dv, workspace=ws, window=window, sinks=sinks,
                    stream=stream)
    torch.cuda.synchronize()
    return dict(out=out, lse=lse, dq=dq, dk=dk, dv=dv)


def check(got, q, k, v, offs_q, offs_k, go, window=0, sinks=0):
    want = ref.ragged(q, k, v, offs_q.tolist(), offs_k.tolist(), q.shape[2] ** -0.5, window, sinks, go)
    for x, y in got.items():
        ref.close(y, want[x], want[x + "_t"], x)


@pytest.mark.parametrize("hq,hkv,sinks", [(4, 2, 3), (2, 2, 200), (3, 1, 5000)])
def test_far_queries_of_sinks(hq, hkv, sinks):
    """Sequences of more queries than a run of the keys' pass takes."""
    note(f"far {hq}/{hkv} sinks {sinks}")
    g, lengths = gen(5), [2300, 30, 4200, 2049, 0, 2048]
    n = sum(lengths)
    q, k, v, go = (heads(g, n, h, 64) for h in (hq, hkv, hkv, hq))
    offs = cu(lengths)
    check(step(q, k, v, offs, offs, go, 100, sinks), q, k, v, offs, offs, go, 100, sinks)


@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 2), (300, 0)])
def test_more_or_fewer_queries_than_keys(window, sinks):
    g, nq, nk = gen(6), [5, 9, 0, 6, 300, 70], [9, 5, 7, 0, 470, 64]
    q, go = heads(g, sum(nq), 6, 128), heads(g, sum(nq), 6, 128)
    k, v = heads(g, sum(nk), 2, 128), heads(g, sum(nk), 2, 128)
    a, b = cu(nq), cu(nk)
    got = step(q, k, v, a, b, go, window, sinks)
    check(got, q, k, v, a, b, go, window, sinks)
    assert bool((got["out"][5:9] == 0).all()) and bool((got["dq"][5:9] == 0).all())   # queries before the first key
    assert bool((got["lse"][5:9] == -math.inf).all())


@pytest.mark.parametrize("hq,hkv,dim", [(2, 2, 16), (4, 1, 32), (3, 3, 48), (2, 1, 96), (8, 2, 112), (33, 1, 64)])
def test_head_sizes(hq, hkv, dim):
    note(f"heads {hq}/{hkv}x{dim}")
    g, lengths = gen(dim), [65, 7, 130]
    n = sum(lengths)
    q, k, v, go = (heads(g, n, h, dim) for h in (hq, hkv, hkv, hq))
    offs = cu(lengths)
    check(step(q, k, v, offs, offs, go, 50, 3), q, k, v, offs, offs, go, 50, 3)


@pytest.mark.parametrize("std", [1e-3, 8.0])
def test_flat_and_steep_softmaxes(std):
    """Scores that hardly differ, and such that one key takes nearly all."""
    g, lengths = gen(24), [300, 5]
    q, k = heads(g, 305, 4, 64, std), heads(g, 305, 2, 64, std)
    v, go = heads(g, 305, 2, 64), heads(g, 305, 4, 64)
    offs = cu(lengths)
    check(step(q, k, v, offs, offs, go), q, k, v, offs, offs, go)


@pytest.mark.parametrize("source", ["rows", "pages", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128, 80])
@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 70)])
def test_enough_for_wide_workgroups(dim, source, window, sinks):
    """So many queries and heads that a workgroup takes 256 of them."""
    note(f"wide {source} {dim} window {window}")
    g, new, hq, hkv, past = gen(dim), [2043, 1, 300], 64, 4, 37
    n, offs = sum(new), cu(new)
    assert n * hq >= 2 * 256 * 256                  # of 256 compute units
    q = heads(g, n, hq, dim)
    out, lse = torch.empty_like(q), torch.empty(n, hq, device=DEV)
    if source == "rows":
        total = new
        k, v = heads(g, n, hkv, dim), heads(g, n, hkv, dim)
        tar.ar_attn(q, k, v, offs, offs, out, window=window, sinks=sinks, lse=lse)
    else:
        total = [m + past for m in new]
        table, pages = tables(g, total, 48)
        cache = filled(g, pages, 48, hkv, dim, source == "e4m3")
        lens = torch.tensor(total, device=DEV, dtype=torch.int32)
        tar.ar_attn_paged(q, cache, table, lens, offs, out, window=window, sinks=sinks, lse=lse)
    torch.cuda.synchronize()
    for i in range(3):
        a = slice(int(offs[i]), int(offs[i + 1]))
        kk, vv = (k[a], v[a]) if source == "rows" else ref.paged(cache, table[i], total[i])
        for h in (0, 17, 63):
            want = ref.attend(q[a, h], kk[:, h // 16], vv[:, h // 16], dim ** -0.5, window, sinks)
            ref.close(out[a, h], want["out"], want["out_t"], f"out of sequence {i}, head {h}")
            ref.close(lse[a, h], want["lse"], want["lse_t"], f"lse of sequence {i}, head {h}")


def test_several_heads_of_one_workgroup():
    """So many keys that a workgroup of the keys' pass takes several heads."""
    note("several heads")
    g, lengths, hq, hkv = gen(31), [16500, 200], 8, 4
    n, offs = sum(lengths), cu(lengths)
    q, k, v, go = (heads(g, n, h, 64) for h in (hq, hkv, hkv, hq))
    got = step(q, k, v, offs, offs, go, 500, 2)
    # the short sequence whole, of the long one the last keys (its window's reach) and rows
    a = slice(16500, 16700)
    want = ref.ragged(q[a], k[a], v[a], [0, 200], [0, 200], 0.125, 500, 2, go[a])
    for x, y in got.items():
        ref.close(y[a], want[x], want[x + "_t"], x)
    for h in (0, 7):
        one = ref.attend(q[:16500, h], k[:16500, h // 2], v[:16500, h // 2], 0.125, 500, 2)
        ref.close(got["out"][:16500, h], one["out"], one["out_t"], "out")
    # all gradients of one key head
    dk, dv, tk, tv = (torch.zeros(16500, 64, device=DEV, dtype=torch.float64) for _ in range(4))
    for h in (2, 3):
        w = ref.attend(q[:16500, h], k[:16500, 1], v[:16500, 1], 0.125, 500, 2, go[:16500, h])
        ref.close(got["dq"][:16500, h], w["dq"], w["dq_t"], "dq")
        dk += w["dk"]
        dv += w["dv"]
        tk += w["dk_t"]
        tv += w["dv_t"]
        del w
    ref.close(got["dk"][:16500, 1], dk, tk + (ref.U + 2 * ref.E) * dk.abs(), "dk")
    ref.close(got["dv"][:16500, 1], dv, tv + (ref.U + 2 * ref.E) * dv.abs(), "dv")


def test_no_rows_at_all():
    q, k = heads(gen(1), 0, 2, 64), heads(gen(1), 3, 1, 64)
    got = step(q, k, k.clone(), cu([0]), cu([3]), q)
    assert bool((got["dk"] == 0).all()) and bool((got["dv"] == 0).all())
    q, k = heads(gen(1), 3, 2, 64), heads(gen(1), 0, 1, 64)
    got = step(q, k, k.clone(), cu([3]), cu([0]), q)
    assert bool((got["out"] == 0).all()) and bool((got["dq"] == 0).all())


@pytest.mark.parametrize("dim", [64, 128])
def test_strides(dim):
    """Heads side by side in one projection's result, gradients likewise, and
    heads before tokens."""
    g, lengths = gen(7), [100, 3, 64]
    n, hq, hkv = sum(lengths), 4, 2
    offs = cu(lengths)
    rows = heads(g, n, hq + 2 * hkv, dim)
    go = heads(g, hq, n, dim).transpose(0, 1)
    d = torch.full_like(rows, 7.0)
    cut = lambda t: (t[:, :hq], t[:, hq:hq + hkv], t[:, hq + hkv:])
    q, k, v = cut(rows)
    out = torch.empty(hq, n, dim, device=DEV, dtype=torch.bfloat16).transpose(0, 1)
    got = step(q, k, v, offs, offs, go, 40, 1, outs=(out, *cut(d)))
    check(got, q, k, v, offs, offs, go, 40, 1)
    # results over the queries
    over = q.clone()
    tar.ar_attn(over, k, v, offs, offs, over, window=40, sinks=1)
    torch.cuda.synchronize()
    assert torch.equal(over, out)


def test_one_gradient_without_the_other():
    g, lengths = gen(8), [90, 41]
    q, k, v, go = (heads(g, 131, h, 64) for h in (4, 2, 2, 4))
    offs = cu(lengths)
    both = step(q, k, v, offs, offs, go)
    ws = torch.empty(tar.attn_bwd_workspace(131, 131, 2, 4, 2, 64), device=DEV, dtype=torch.uint8)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    tar.ar_attn_bwd(q, k, v, both["out"], both["lse"], go, offs, offs, dq=dq, workspace=ws)
    tar.ar_attn_bwd(q, k, v, both["out"], both["lse"], go, offs, offs, dk=dk, dv=dv, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(dq, both["dq"]) and torch.equal(dk, both["dk"]) and torch.equal(dv, both["dv"])


def test_repeats_bit_for_bit():
    g, lengths = gen(9), [1500, 700]
    q, k, v, go = (heads(g, 2200, h, 128) for h in (8, 2, 2, 8))
    offs = cu(lengths)
    a, b = (step(q, k, v, offs, offs, go, 600, 4) for _ in range(2))
    for x in a:
        assert torch.equal(a[x], b[x]), x


def test_gradients_against_differences():
    """sum(d_out * out) along a random direction: its difference quotient in 64
    bits, and what the gradients say."""
    g, lengths, window, sinks = gen(10), [70, 33], 25, 2
    q, k, v, go = (heads(g, 103, h, 64) for h in (4, 2, 2, 4))
    offs = cu(lengths)
    got = step(q, k, v, offs, offs, go, window, sinks)
    want = ref.ragged(q, k, v, offs.tolist(), offs.tolist(), 0.125, window, sinks, go)
    for name, x, grad in (("q", q, "dq"), ("k", k, "dk"), ("v", v, "dv")):
        d = torch.randn(x.shape, generator=g, device=DEV, dtype=torch.float64)
        h = 1e-4
        at = []
        for sign in (1, -1):
            moved = {"q": q.double(), "k": k.double(), "v": v.double()}
            moved[name] = moved[name] + sign * h * d
            r = ref.ragged(moved["q"], moved["k"], moved["v"], offs.tolist(), offs.tolist(), 0.125, window, sinks)
            at.append((go.double() * r["out"]).sum())
        slope = float((at[0] - at[1]) / (2 * h))
        told = float((got[grad].double() * d).sum())
        # the quotient's own error: its third-order term, h^2 = 1e-8 of sums of size |d|^3, and
        # 64-bit roundings of the sums over 2 h
        own = 1e-6 * float((got[grad].double().abs() * d.abs()).sum()) + 1e-6
        assert abs(slope - told) <= float((want[grad + "_t"] * d.abs()).sum()) + own, name


# ------------------------------------------- masked places that are no numbers

@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_later_values_do_not_reach_earlier_queries(dim, bad):
    g, n, at = gen(11), 150, 70
    q, k, v = (heads(g, n, h, dim) for h in (4, 2, 2))
    clean = torch.empty_like(q)
    offs = cu([n])
    tar.ar_attn(q, k, v, offs, offs, clean)
    v[at, 1, 5] = bad
    out = torch.empty_like(q)
    tar.ar_attn(q, k, v, offs, offs, out)
    torch.cuda.synchronize()
    want = ref.ragged(q, k, torch.where(torch.isfinite(v), v, torch.zeros_like(v)), [0, n], [0, n], dim ** -0.5)
    hit = torch.zeros(out.shape, device=DEV, dtype=torch.bool)
    hit[at:, 2:, 5] = True                           # queries that see it, heads of its key head
    ref.close(out, want["out"], torch.where(hit, -1.0, want["out_t"]), "out")
    assert bool((out[hit] == bad).all()) if math.isinf(bad) else bool(torch.isnan(out[hit]).all())
    # a key that is no number
    v[at, 1, 5] = 0
    k[at, 0, 9] = math.nan
    tar.ar_attn(q, k, v, offs, offs, out)
    torch.cuda.synchronize()
    assert torch.equal(out[:at, :2], clean[:at, :2]) and bool(torch.isnan(out[at:, :2]).all())
    # a query that is no number
    k[at, 0, 9] = 0
    q[at, 3] = math.nan
    tar.ar_attn(q, k, v, offs, offs, out)
    torch.cuda.synchronize()
    assert bool(torch.isnan(out[at, 3]).all()) and bool(torch.isfinite(out[:at]).all()) and bool(torch.isfinite(out[at + 1:]).all())


@pytest.mark.parametrize("window,sinks", [(20, 0), (20, 3)])
def test_values_outside_the_window(window, sinks):
    g, n, at = gen(12), 200, 50
    q, k, v = (heads(g, n, h, 64) for h in (2, 1, 1))
    v[at, 0, :] = math.nan
    out, offs = torch.empty_like(q), cu([n])
    tar.ar_attn(q, k, v, offs, offs, out, window=window, sinks=sinks)
    torch.cuda.synchronize()
    bad = torch.isnan(out).all(2).all(1)
    assert bad.nonzero()[:, 0].tolist() == list(range(at, at + window))
    assert not bool(torch.isnan(out[~bad]).any())


def test_other_sequences_keep_their_gradients():
    g, lengths = gen(13), [40, 50, 60]
    q, k, v, go = (heads(g, 150, h, 64) for h in (2, 1, 1, 2))
    offs = cu(lengths)
    clean = step(q, k, v, offs, offs, go)
    for x in (q, k, v, go):
        y = x.clone()
        y[60] = math.nan                             # of the second sequence
        got = step(*[y if z is x else z for z in (q, k, v)], offs, offs, y if x is go else go)
        for name in got:
            for rows in (slice(0, 40), slice(90, 150)):
                assert torch.equal(got[name][rows], clean[name][rows]), name


@pytest.mark.parametrize("e4m3", [False, True])
def test_what_lies_behind_a_sequence_in_its_pages(e4m3):
    g, lengths, page = gen(14), [5, 33, 100], 16
    table, pages = tables(g, lengths, page)
    cache = filled(g, pages, page, 2, 64, e4m3)
    q = normal(g, 3, 4, 64).to(torch.bfloat16)
    lens, offs = torch.tensor(lengths, device=DEV, dtype=torch.int32), cu([1, 1, 1])
    ws = torch.zeros(tar.attn_decode_workspace(3, 4, 2, 64), device=DEV, dtype=torch.uint8)

    def both():
        a, b = torch.empty_like(q), torch.empty_like(q)
        tar.ar_attn_decode(q, cache, table, lens, a, workspace=ws)
        tar.ar_attn_paged(q, cache, table, lens, offs, b)
        torch.cuda.synchronize()
        return a, b
    clean = both()
    for i, n in enumerate(lengths):
        for j in range(n, -(-n // page) * page):
            at = (int(table[i, j // page]), j % page)
            for c in cache[:2]:
                c.view(torch.uint8 if e4m3 else torch.int16)[at] = 0x7F if e4m3 else 0x7FC0
            for c in cache[2:]:
                c[at] = math.nan
    dirty = both()
    for x, y in zip(clean, dirty):
        assert bool(torch.isfinite(y).all()) and torch.equal(x, y)


@pytest.mark.parametrize("e4m3", [False, True])
def test_page_numbers_out_of_range(e4m3):
    """A page that is looked at makes its readers' results NaN; one outside the
    window is not looked at; other sequences keep theirs."""
    g, lengths, page = gen(15), [100, 500, 60], 16
    table, pages = tables(g, lengths, page)
    cache = filled(g, pages, page, 1, 128, e4m3)
    q = normal(g, 3, 2, 128).to(torch.bfloat16)
    lens, offs = torch.tensor(lengths, device=DEV, dtype=torch.int32), cu([1, 1, 1])
    for window, sinks, sees in ((0, 0, True), (64, 0, False), (64, 20, True)):
        clean, out = [], []
        for res in (clean, out):
            for paged in (False, True):
                o = torch.empty_like(q)
                if paged:
                    tar.ar_attn_paged(q, cache, table, lens, offs, o, window=window, sinks=sinks)
                else:
                    tar.ar_attn_decode(q, cache, table, lens, o, window=window, sinks=sinks)
                res.append(o)
            torch.cuda.synchronize()
            if res is clean:
                keep = table.clone()
                table[1, 1] = [pages, -1, 2 ** 31 - 1][sinks % 3]
        table.copy_(keep)
        for x, y in zip(clean, out):
            assert torch.equal(x[[0, 2]], y[[0, 2]])
            assert bool(torch.isnan(y[1]).all()) if sees else torch.equal(x[1], y[1])


# ------------------------------------------------------------- large and strided

@pytest.mark.parametrize("e4m3", [False, True])
def test_cache_beyond_32_bits(e4m3):
    """Pages whose elements lie beyond 2^32 elements of the cache's start."""
    note(f"large cache e4m3 {e4m3}")
    pages, page, hkv, dim = 2 ** 18 + 100, 16, 8, 128     # 2^32 elements and more, of keys and of values
    dt = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    cache = tuple(torch.empty(pages, page, hkv, dim, device=DEV, dtype=dt) for _ in range(2))
    if e4m3:
        cache += tuple(torch.empty(pages, page, hkv, device=DEV) for _ in range(2))
    g, n = gen(16), 70
    table = torch.tensor([[pages - 1, 3, pages - 50, 2 ** 18, pages - 7]], device=DEV, dtype=torch.int32)
    k, v = (normal(g, n, hkv, dim).to(torch.bfloat16) for _ in range(2))
    q = normal(g, n, 8, dim).to(torch.bfloat16)
    j = torch.arange(n, device=DEV)
    slots = table[0].long()[j // page] * page + j % page
    cos_sin = torch.cat([torch.ones(1, 8, device=DEV), torch.zeros(1, 8, device=DEV)], 1)
    tar.ar_rope_kv(None, k, v, cos_sin, torch.zeros(n, device=DEV, dtype=torch.int32), cache=cache, slots=slots)
    lens, offs = torch.tensor([n], device=DEV, dtype=torch.int32), cu([n])
    one, out = torch.empty(1, 8, dim, device=DEV, dtype=torch.bfloat16), torch.empty_like(q)
    tar.ar_attn_decode(q[-1:], cache, table, lens, one)
    tar.ar_attn_paged(q, cache, table, lens, offs, out)
    torch.cuda.synchronize()
    kk, vv = ref.paged(cache, table[0], n)
    if not e4m3:
        assert torch.equal(kk, k.double()) and torch.equal(vv, v.double())
    for h in range(8):
        want = ref.attend(q[:, h], kk[:, h], vv[:, h], dim ** -0.5)
        ref.close(out[:, h], want["out"], want["out_t"], "prompt")
        ref.close(one[:, h], want["out"][-1:], want["out_t"][-1:], "single token")


def test_rows_far_apart():
    """Token strides of 2^24 elements: offsets within a tile of 64 rows pass 32 bits."""
    n, dim, far = 70, 64, 2 ** 24 + 8
    room = torch.empty(4, n * far, device=DEV, dtype=torch.bfloat16)
    g = gen(17)
    q, k, v, go = (heads(g, n, 1, dim) for _ in range(4))
    wide = [room[i].as_strided((n, 1, dim), (far, dim, 1)) for i in range(4)]
    for x, y in zip(wide, (q, k, v, go)):
        x.copy_(y)
    offs = cu([n])
    a, b = step(q, k, v, offs, offs, go), step(*wide[:3], offs, offs, wide[3])
    for x in a:
        assert torch.equal(a[x], b[x]), x


@pytest.mark.parametrize("layout", ["kv side by side", "heads first"])
def test_cache_layouts(layout):
    g, lengths, page, hkv, dim = gen(18), [33, 90], 16, 2, 64
    table, pages = tables(g, lengths, page)
    if layout == "kv side by side":
        both = normal(g, pages, page, 2, hkv, dim).to(torch.bfloat16)
        cache = (both[:, :, 0], both[:, :, 1])
    else:
        both = normal(g, pages, 2, hkv, page, dim).to(torch.bfloat16)
        cache = tuple(both[:, i].transpose(1, 2) for i in range(2))
    k, v = (normal(g, 5, hkv, dim).to(torch.bfloat16) for _ in range(2))
    slots = torch.tensor([int(table[1, 0]) * page + i for i in range(5)], device=DEV)
    keep = both.clone()
    cos_sin = torch.cat([torch.ones(1, 8, device=DEV), torch.zeros(1, 8, device=DEV)], 1)
    tar.ar_rope_kv(None, k, v, cos_sin, torch.zeros(5, device=DEV, dtype=torch.int32), cache=cache, slots=slots)
    q = normal(g, 2, 4, dim).to(torch.bfloat16)
    out, lens = torch.empty_like(q), torch.tensor(lengths, device=DEV, dtype=torch.int32)
    tar.ar_attn_decode(q, cache, table, lens, out)
    torch.cuda.synchronize()
    changed = (both != keep).nonzero()[:, 0].unique().tolist()
    assert changed == [int(table[1, 0])]
    for i, n in enumerate(lengths):
        kk, vv = ref.paged(cache, table[i], n)
        if i == 1:
            assert torch.equal(kk[:5], k.double()) and torch.equal(vv[:5], v.double())
        for h in range(4):
            want = ref.attend(q[i:i + 1, h], kk[:, h // 2], vv[:, h // 2], dim ** -0.5)
            ref.close(out[i:i + 1, h], want["out"], want["out_t"], "out")


# ---------------------------------------------------------- many and few sequences

@pytest.mark.parametrize("hq,hkv,e4m3", [(8, 8, False), (64, 1, False), (16, 3 * 4, True), (5, 5, True)])
def test_decode_many_sequences(hq, hkv, e4m3):
    """More sequences than a wave has lanes, a long one among short and empty
    ones, workspaces reused by other shapes, counters zero afterwards."""
    if hq % hkv:
        hq = 2 * hkv
    note(f"many {hq}/{hkv} e4m3 {e4m3}")
    g, page, dim = gen(19), 32, 64
    lengths = [(i * 37) % 150 if i % 5 else 0 for i in range(150)]
    lengths[77] = 9000
    table, pages = tables(g, lengths, page)
    cache = filled(g, pages, page, hkv, dim, e4m3)
    q = normal(g, len(lengths), hq, dim).to(torch.bfloat16)
    lens = torch.tensor(lengths, device=DEV, dtype=torch.int32)
    size = tar.attn_decode_workspace(len(lengths), hq, hkv, dim)
    ws = torch.zeros(size, device=DEV, dtype=torch.uint8)
    out = torch.empty_like(q)
    few = torch.empty_like(q[77:79])
    for _ in range(2):
        tar.ar_attn_decode(q, cache, table, lens, out, workspace=ws)
        tar.ar_attn_decode(q[77:79], cache, table[77:79], lens[77:79], few, workspace=ws)
    torch.cuda.synchronize()
    # the counters are the workspace's end
    assert not bool(ws[size - len(lengths) * hkv * -(-(hq // hkv) // 16) * 4:].any())
    for i, n in enumerate(lengths):
        k, v = ref.paged(cache, table[i], n)
        for h in (0, hq - 1, hq // 2):
            want = ref.attend(q[i:i + 1, h], k[:, h // (hq // hkv)], v[:, h // (hq // hkv)], dim ** -0.5)
            ref.close(out[i:i + 1, h], want["out"], want["out_t"], f"sequence {i} of {n} keys, head {h}")
            if i == 77:
                ref.close(few[:1, h], want["out"], want["out_t"], "the same in a smaller batch")


def test_lengths_beyond_the_table():
    """Held within it; below 0 is 0."""
    g = gen(20)
    table = torch.tensor([[0, 1], [1, 0]], device=DEV, dtype=torch.int32)
    cache = filled(g, 2, 16, 1, 64, False)
    q = normal(g, 2, 2, 64).to(torch.bfloat16)
    out, want = torch.empty_like(q), torch.empty_like(q)
    tar.ar_attn_decode(q, cache, table, torch.tensor([1000, -3], device=DEV, dtype=torch.int32), out)
    tar.ar_attn_decode(q, cache, table, torch.tensor([32, 0], device=DEV, dtype=torch.int32), want)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and bool((out[1] == 0).all())


# ---------------------------------------------------------------- graphs, streams

def test_graph_of_a_served_step():
    """Append and decode of a step captured once and replayed with new inputs
    and growing lengths, between eager work."""
    g, page, hq, hkv, dim, seqs = gen(21), 16, 8, 2, 128, 5
    start = [3, 60, 200, 15, 0]
    table, pages = tables(g, [n + 20 for n in start], page)
    cache = filled(g, pages, page, hkv, dim, False)
    rows = torch.empty(seqs, hq + 2 * hkv, dim, device=DEV, dtype=torch.bfloat16)
    q, k, v = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
    cos_sin = tar.rope_table(400, dim, device=DEV)
    lens, pos = torch.zeros(seqs, device=DEV, dtype=torch.int32), torch.zeros(seqs, device=DEV, dtype=torch.int32)
    slots = torch.zeros(seqs, device=DEV, dtype=torch.int64)
    ws = torch.zeros(tar.attn_decode_workspace(seqs, hq, hkv, dim), device=DEV, dtype=torch.uint8)
    turned, out = torch.empty(seqs, hq, dim, device=DEV, dtype=torch.bfloat16), torch.empty(seqs, hq, dim, device=DEV, dtype=torch.bfloat16)

    def work(qo, o, w):
        tar.ar_rope_kv(q, k, v, cos_sin, pos, q_out=qo, cache=cache, slots=slots)
        tar.ar_attn_decode(qo, cache, table, lens, o, workspace=w)

    def at(i):
        now = torch.tensor([n + i for n in start], device=DEV)
        rows.copy_(normal(g, *rows.shape))
        pos.copy_(now)
        lens.copy_(now + 1)
        slots.copy_(table[torch.arange(seqs, device=DEV), now // page].long() * page + now % page)

    at(0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        work(turned, out, ws)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work(turned, out, ws)
    other = torch.zeros_like(ws)
    for i in range(1, 6):
        at(i)
        graph.replay()
        torch.cuda.synchronize()
        qo, o = torch.empty_like(turned), torch.empty_like(out)
        work(qo, o, other)
        torch.cuda.synchronize()
        assert torch.equal(turned, qo) and torch.equal(out, o), i


def test_graph_of_a_training_step():
    """Captured while eager results of the same inputs live; replayed with new
    inputs."""
    g, lengths = gen(22), [300, 90]
    q, k, v, go = (heads(g, 390, h, 64) for h in (4, 2, 2, 4))
    offs = cu(lengths)
    outs = tuple(torch.empty_like(x) for x in (q, q, k, v))
    lse = torch.empty(390, 4, device=DEV)
    ws = torch.empty(tar.attn_bwd_workspace(390, 390, 2, 4, 2, 64, 100, 2), device=DEV, dtype=torch.uint8)

    def work():
        tar.ar_attn(q, k, v, offs, offs, outs[0], window=100, sinks=2, lse=lse)
        tar.ar_attn_bwd(q, k, v, outs[0], lse, go, offs, offs, dq=outs[1], dk=outs[2], dv=outs[3], workspace=ws, window=100, sinks=2)
    eager = step(q, k, v, offs, offs, go, 100, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        work()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    for _ in range(4):
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(("out", "dq", "dk", "dv"), outs):
            assert torch.equal(eager[x], y), x
        for x in (q, k, v, go):
            x.copy_(torch.randn(x.shape, generator=g, device=DEV))
        eager = step(q, k, v, offs, offs, go, 100, 2)


def test_two_streams_at_once():
    """Calls that overlap in time, each with a workspace of its own."""
    g, page = gen(23), 16
    lengths = [4000, 10, 900]
    table, pages = tables(g, lengths, page)
    cache = filled(g, pages, page, 2, 128, True)
    lens = torch.tensor(lengths, device=DEV, dtype=torch.int32)
    streams = [torch.cuda.Stream() for _ in range(2)]
    qs = [normal(g, 3, 8, 128).to(torch.bfloat16) for _ in range(2)]
    outs = [[torch.empty_like(q) for _ in range(8)] for q in qs]
    wss = [torch.zeros(tar.attn_decode_workspace(3, 8, 2, 128), device=DEV, dtype=torch.uint8) for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(8):
        for s, q, o, w in zip(streams, qs, outs, wss):
            tar.ar_attn_decode(q, cache, table, lens, o[i], workspace=w, stream=s)
    torch.cuda.synchronize()
    for q, o in zip(qs, outs):
        want = torch.empty_like(q)
        tar.ar_attn_decode(q, cache, table, lens, want, workspace=wss[0])
        torch.cuda.synchronize()
        for x in o:
            assert torch.equal(x, want)


@pytest.mark.parametrize("source", ["rows", "pages", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new", [[640, 1, 300, 0, 129, 700, 513], [2050]])
def test_workgroups_by_their_number(dim, source, new):
    """Workgroups of 128 queries: so many that two share a compute unit, and
    long prompts of which half a workgroup takes every other tile of keys; with
    a mask that leaves such a half no key, or one of its sides a single one."""
    note(f"number {source} {dim} {new}")
    hq, hkv, g, n, offs = 24, 4, gen(dim + len(new)), sum(new), cu(new)
    q = heads(g, n, hq, dim)
    for window, sinks, past in ((0, 0, 0), (64, 0, 63), (1, 1, 64), (97, 65, 5)):
        out, lse = torch.empty_like(q), torch.empty(n, hq, device=DEV)
        total = [m + past if m else 0 for m in new]
        if source == "rows":
            ko = cu(total)
            k, v = heads(g, sum(total), hkv, dim), heads(g, sum(total), hkv, dim)
            tar.ar_attn(q, k, v, offs, ko, out, window=window, sinks=sinks, lse=lse)
        else:
            table, pages = tables(g, total, 16)
            cache = filled(g, pages, 16, hkv, dim, source == "e4m3")
            lens = torch.tensor(total, device=DEV, dtype=torch.int32)
            tar.ar_attn_paged(q, cache, table, lens, offs, out, window=window, sinks=sinks, lse=lse)
        torch.cuda.synchronize()
        for i in range(len(new)):
            if not new[i]:
                continue
            a = slice(int(offs[i]), int(offs[i + 1]))
            kk, vv = (k[int(ko[i]):int(ko[i + 1])], v[int(ko[i]):int(ko[i + 1])]) if source == "rows" else ref.paged(cache, table[i], total[i])
            for h in (0, hq - 1):
                want = ref.attend(q[a, h], kk[:, h // (hq // hkv)], vv[:, h // (hq // hkv)], dim ** -0.5, window, sinks)
                ref.close(out[a, h], want["out"], want["out_t"], f"out of sequence {i}, head {h}, window {window}")
                ref.close(lse[a, h], want["lse"], want["lse_t"], f"lse of sequence {i}, head {h}, window {window}")


@pytest.mark.parametrize("source", ["rows", "pages"])
def test_halves_with_values_that_are_no_numbers(source):
    """Values that are no numbers in either half's tiles of keys: where they
    are masked they change nothing, where they are visible they are seen."""
    note(f"halves, no numbers, {source}")
    g, n, hq, hkv, dim = gen(5), 330, 4, 2, 128
    q, k, v = heads(g, n, hq, dim), heads(g, n, hkv, dim), heads(g, n, hkv, dim)
    offs = cu([n])
    for at in (70, 140, 300):                       # tiles 1, 2 and 4
        clean, lse0 = torch.empty_like(q), torch.empty(n, hq, device=DEV)
        out, lse = torch.empty_like(q), torch.empty(n, hq, device=DEV)
        odd = v.clone()
        odd[at, 0] = float("nan")
        odd[at, 1, :3] = float("inf")
        if source == "rows":
            run = lambda vv, o, s: tar.ar_attn(q, k, vv, offs, offs, o, lse=s)
        else:
            table = torch.arange((n + 15) // 16, device=DEV, dtype=torch.int32).view(1, -1)
            lens = torch.tensor([n], device=DEV, dtype=torch.int32)

            def run(vv, o, s):
                cache = tar.kv_cache_empty(table.numel(), 16, hkv, dim, device=DEV)
                pad = table.numel() * 16 - n
                for x, y in zip(cache, (k, vv)):
                    x.copy_(torch.nn.functional.pad(y, (0, 0, 0, 0, 0, pad)).view(x.shape))
                tar.ar_attn_paged(q, cache, table, lens, offs, o, lse=s)
        run(v, clean, lse0)
        run(odd, out, lse)
        torch.cuda.synchronize()
        assert torch.isfinite(clean).all() and torch.equal(lse, lse0)
        assert torch.equal(out[:at], clean[:at])
        assert out[at:, :2].isnan().all()           # heads 0, 1 read key head 0
        assert (~torch.isfinite(out[at:, 2:, :3])).all()
        assert torch.equal(out[at:, 2:, 3:], clean[at:, 2:, 3:])
