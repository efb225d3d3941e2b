"""Attention over values that are infinite, no numbers or very large: what is
visible shows in the result as the formula has it, over pages as over rows,
for single tokens as for prompts."""
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


def place(table, i, j, page):
    return int(table[i, j // page]), j % page


def same(got, want, what):
    """Infinities and NaN in the same places."""
    inf = torch.isinf(want)
    nans, infs = (got.isnan() != want.isnan()).sum(), ((got != want) & (inf | got.isinf())).sum()
    assert int(nans) == 0 and int(infs) == 0, what


class Served:
    """Sequences in pages and one new token of each."""

    def __init__(self, g, lengths, hq, hkv, dim, page, e4m3):
        self.lengths, self.page, self.dim = lengths, page, dim
        self.table, pages = tables(g, lengths, page)
        self.cache = filled(g, pages, page, hkv, dim, e4m3)
        self.q = normal(g, len(lengths), hq, dim).to(torch.bfloat16)
        self.lens = torch.tensor(lengths, device=DEV, dtype=torch.int32)
        self.ws = torch.zeros(tar.attn_decode_workspace(len(lengths), hq, hkv, dim), device=DEV, dtype=torch.uint8)

    def decode(self, cut, **mask):
        out = torch.full_like(self.q, 7.0)
        tar.ar_attn_decode(self.q, self.cache, self.table, self.lens, out, workspace=self.ws if cut else None, **mask)
        torch.cuda.synchronize()
        return out

    def prompt(self, **mask):
        out = torch.full_like(self.q, 7.0)
        tar.ar_attn_paged(self.q, self.cache, self.table, self.lens, cu([1] * len(self.lengths)), out, **mask)
        torch.cuda.synchronize()
        return out


# ------------------------------------------------- single tokens, visible values

@pytest.mark.parametrize("cut", [False, True])
@pytest.mark.parametrize("hq,hkv,dim,page,e4m3", [(8, 2, 128, 16, False), (6, 3, 64, 48, False), (40, 2, 80, 7, False),
                                                  (16, 2, 128, 16, True), (4, 4, 64, 32, True)])
def test_single_tokens_see_what_is_no_number(hq, hkv, dim, page, e4m3, cut):
    note(f"visible {hq}/{hkv}x{dim} page {page} e4m3 {e4m3} cut {cut}")
    lengths, at = [1, 20, 129, 700, 3000], [0, 19, 64, 333, 2900]
    s = Served(gen(dim + hq), lengths, hq, hkv, dim, page, e4m3)
    clean = s.decode(cut)
    kept = [ref.paged(s.cache, s.table[i], n) for i, n in enumerate(lengths)]
    h = hkv - 1                                       # only this key head has such values
    for i, j in enumerate(at):
        p = place(s.table, i, j, page)
        v = s.cache[1][p][h]
        if e4m3:
            v.view(torch.uint8)[5] = 0x7F
        else:
            v[3], v[4], v[5], v[6] = math.inf, -math.inf, math.nan, math.inf
            s.cache[1][place(s.table, i, j // 2, page)][h][6] = -math.inf if j else math.inf
    out, prompt = s.decode(cut), s.prompt()
    group, first = hq // hkv, h * (hq // hkv)
    assert torch.equal(out[:, :first], clean[:, :first])
    same(out, prompt, "single token and prompt")
    for i, n in enumerate(lengths):
        bad = out[i, first:]
        assert bool(torch.isnan(bad[:, 5]).all())
        cols = {5}
        if not e4m3:
            assert bool((bad[:, 3] == math.inf).all()) and bool((bad[:, 4] == -math.inf).all())
            assert bool((bad[:, 6] == math.inf).all()) if i == 0 else bool(torch.isnan(bad[:, 6]).all())
            cols |= {3, 4, 6}
        rest = [c for c in range(dim) if c not in cols]
        for x in range(group):
            want = ref.attend(s.q[i:i + 1, first + x], kept[i][0][:, h], kept[i][1][:, h], dim ** -0.5)
            ref.close(bad[x:x + 1, rest], want["out"][:, rest], want["out_t"][:, rest], f"out of {n} keys, head {x}")


@pytest.mark.parametrize("cut", [False, True])
@pytest.mark.parametrize("dim", [64, 128])
def test_single_tokens_and_infinite_scales(dim, cut):
    """A value is its code times its scale: infinities with the codes' signs."""
    note(f"infinite scales {dim} cut {cut}")
    s = Served(gen(dim), [40, 2000], 8, 1, dim, 16, True)
    for i, j in enumerate((7, 1234)):
        p = place(s.table, i, j, 16)
        codes = torch.ones(dim, device=DEV)
        codes[1::2] = -2.0
        codes[6] = 0.0
        s.cache[1][p][0].copy_(codes)
        s.cache[3][p][0] = math.inf
    out = s.decode(cut)
    want = torch.full((dim,), math.inf, device=DEV)
    want[1::2] = -math.inf
    want[6] = math.nan
    for x in out.flatten(0, 1):
        same(x, want.to(x.dtype), "out")


def far_scores(cache, q, table, page, lengths, low):
    """Scores of 256, and of 0 for the keys `low`: weights of e^-256 of the others'."""
    for c in cache[:1]:
        c.zero_()
        c[..., 0] = 16.0
    q.zero_()
    q[..., 0] = 16.0
    for i, n in enumerate(lengths):
        for j in low[i]:
            cache[0][place(table, i, j, page)][:, 0] = 0.0


FAR = [[0], [39], [128], range(2816, 2944), range(0, 700)]   # the first and the last key; a wave's step, a part, an earlier part


@pytest.mark.parametrize("cut", [False, True])
@pytest.mark.parametrize("hq,hkv,dim,page", [(8, 1, 128, 16), (4, 2, 64, 48)])
def test_single_tokens_and_infinities_of_little_weight(hq, hkv, dim, page, cut):
    note(f"little weight {hq}/{hkv}x{dim} cut {cut}")
    lengths = [40, 40, 129, 3000, 3000]
    s = Served(gen(dim), lengths, hq, hkv, dim, page, False)
    far_scores(s.cache, s.q, s.table, page, lengths, FAR)
    kept = [ref.paged(s.cache, s.table[i], n) for i, n in enumerate(lengths)]
    for i, low in enumerate(FAR):
        s.cache[1][place(s.table, i, low[len(low) // 2], page)][:, 3] = math.inf
        s.cache[1][place(s.table, i, low[0], page)][:, 4] = -math.inf
    out = s.decode(cut, scale=1.0)
    assert bool((out[..., 3] == math.inf).all()) and bool((out[..., 4] == -math.inf).all())
    rest = [c for c in range(dim) if c not in (3, 4)]
    for i in range(len(lengths)):
        for h in range(hq):
            kh = h // (hq // hkv)
            want = ref.attend(s.q[i:i + 1, h], kept[i][0][:, kh], kept[i][1][:, kh], 1.0)
            ref.close(out[i:i + 1, h][:, rest], want["out"][:, rest], want["out_t"][:, rest], f"sequence {i}, head {h}")


# --------------------------------------------------------------------- prompts

@pytest.mark.parametrize("n,hq,hkv,dim", [(330, 4, 2, 128), (2048, 24, 4, 64), (2100, 64, 8, 128)])
def test_prompts_and_infinities_of_little_weight(n, hq, hkv, dim):
    """Weights of e^-256 of the others', met before, among and behind those."""
    note(f"little weight, prompt {n} {hq}/{hkv}x{dim}")
    g, offs = gen(n), cu([n])
    q, k, v = heads(g, n, hq, dim), heads(g, n, hkv, dim), heads(g, n, hkv, dim)
    q.zero_()
    k.zero_()
    q[..., 0], k[..., 0] = 16.0, 16.0
    low = (0, 64, 65, 200, 321)
    for j in low:
        k[j] = 0.0
    kept = v.clone()
    for i, j in enumerate(low):
        v[j, :, 2 * i], v[j, :, 2 * i + 1] = math.inf, -math.inf
    out = torch.empty_like(q)
    tar.ar_attn(q, k, v, offs, offs, out, scale=1.0)
    torch.cuda.synchronize()
    for i, j in enumerate(low):
        assert bool((out[j:, :, 2 * i] == math.inf).all()) and bool((out[j:, :, 2 * i + 1] == -math.inf).all()), j
        assert bool(torch.isfinite(out[:j, :, 2 * i:2 * i + 2]).all()), j
    for h in (0, hq - 1):
        want = ref.attend(q[:, h], k[:, h // (hq // hkv)], kept[:, h // (hq // hkv)], 1.0)
        tol = want["out_t"].clone()
        for i, j in enumerate(low):
            tol[j:, 2 * i:2 * i + 2] = -1.0
        ref.close(out[:, h], want["out"], tol, f"head {h}")


@pytest.mark.parametrize("source", ["rows", "pages", "e4m3"])
@pytest.mark.parametrize("n,hq,hkv,dim", [(330, 4, 2, 128), (128, 2, 2, 64), (2048, 24, 4, 64), (2100, 64, 8, 128)])
def test_prompts_and_large_values(n, hq, hkv, dim, source):
    """Means of many keys below the largest value, which their numerators' sum
    is not; a key head each magnitude."""
    note(f"large values, prompt {n} {hq}/{hkv}x{dim} {source}")
    g, offs = gen(n), cu([n])
    q, k = heads(g, n, hq, dim, 0.25), heads(g, n, hkv, dim)
    v = 1.0 + 0.75 * torch.rand(n, hkv, dim, generator=g, device=DEV)
    for powers in ((126, 110), (124, 122), (121, 120), (118, 119)):
        size = torch.tensor([2.0 ** powers[h % 2] for h in range(hkv)], device=DEV)[None, :, None]
        out, lse = torch.empty_like(q), torch.empty(n, hq, device=DEV)
        if source == "rows":
            kk, vv = k, (v * size).to(torch.bfloat16)
            tar.ar_attn(q, kk, vv, offs, offs, out, lse=lse)
        else:
            table, pages = tables(g, [n], 16)
            cache = filled(g, pages, 16, hkv, dim, source == "e4m3")
            slots = torch.arange(n, device=DEV)
            at = (table[0].long()[slots // 16], slots % 16)
            if source == "e4m3":
                cache[1][at] = (v * 128).to(torch.float8_e4m3fn)
                cache[3][at] = (size / 128).expand(n, hkv, 1)[..., 0]
            else:
                cache[1][at] = (v * size).to(torch.bfloat16)
            tar.ar_attn_paged(q, cache, table, torch.tensor([n], device=DEV, dtype=torch.int32), offs, out, lse=lse)
            kk, vv = ref.paged(cache, table[0], n)
        torch.cuda.synchronize()
        for h in (0, hq - 1):
            kh = h // (hq // hkv)
            want = ref.attend(q[:, h], kk[:, kh], vv[:, kh], dim ** -0.5)
            ref.close(out[:, h], want["out"], want["out_t"], f"2^{powers}, head {h}")
            ref.close(lse[:, h], want["lse"], want["lse_t"], f"lse, 2^{powers}, head {h}")


# ---------------------------------------------------------------- large values

EXPONENTS = [100, 112, 114, 116, 118, 120, 122, 124, 126]


@pytest.mark.parametrize("cut", [False, True])
@pytest.mark.parametrize("keys", [1, 129, 20000])
@pytest.mark.parametrize("dim,e4m3", [(128, False), (64, False), (128, True)])
def test_single_tokens_and_large_values(dim, e4m3, keys, cut):
    """The mean of many equal weights: below the largest value, which the
    numerators' own sum is not."""
    note(f"large values, {keys} keys of {dim}, e4m3 {e4m3}, cut {cut}")
    g = gen(keys)
    s = Served(g, [keys] * len(EXPONENTS), 8, 1, dim, 16, e4m3)
    s.q.mul_(0.25)
    top = 1.0 + 0.5 * torch.rand(dim, generator=g, device=DEV)
    for i, e in enumerate(EXPONENTS):
        rows = s.table[i, :-(-keys // 16)].long()
        noise = 1.0 + 0.25 * torch.rand(len(rows), 16, 1, 1, generator=g, device=DEV)
        if e4m3:                                     # codes up to 1.875 * 2^7
            s.cache[1][rows] = (128.0 * top * noise).to(torch.float8_e4m3fn)
            s.cache[3][rows] = 2.0 ** (e - 7)
        else:
            s.cache[1][rows] = (2.0 ** e * top * noise).to(torch.bfloat16)
    out = s.decode(cut)
    for i, e in enumerate(EXPONENTS):
        k, v = ref.paged(s.cache, s.table[i], keys)
        for h in (0, 7):
            want = ref.attend(s.q[i:i + 1, h], k[:, 0], v[:, 0], dim ** -0.5)
            ref.close(out[i:i + 1, h], want["out"], want["out_t"], f"values of 2^{e}, head {h}")


def test_single_tokens_and_values_that_cancel():
    """Large values of both signs, of which little is left, in one column of
    many and beside ordinary ones."""
    g, n = gen(3), 3000
    s = Served(g, [n], 8, 1, 128, 16, False)
    s.cache[1][:, :, 0, 7] = 2.0 ** 126 * (1 - 2 * torch.randint(0, 2, s.cache[1].shape[:2], generator=g, device=DEV))
    k, v = ref.paged(s.cache, s.table[0], n)
    for cut in (False, True):
        out = s.decode(cut)
        for h in (0, 5):
            want = ref.attend(s.q[:, h], k[:, 0], v[:, 0], 128 ** -0.5)
            ref.close(out[:, h], want["out"], want["out_t"], f"head {h}, cut {cut}")
