"""The cache: rotation and append, attention of single tokens over it and of
prompts' next chunks, against 64 bits."""
import math

import pytest
import torch

import attn_ref as ref
import tensor_all_reduce_amd as tar
from gpu_util import note

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def filled(g, pages, page, heads, dim, e4m3, layout="pthd"):
    """A cache of random contents; layout: the order of its axes in memory."""
    def lay(x):
        order = ["pthd".index(c) for c in layout]
        return x.permute(order).contiguous().permute([order.index(i) for i in range(4)])
    if not e4m3:
        return tuple(lay(normal(g, pages, page, heads, dim).to(torch.bfloat16)) for _ in range(2))
    codes = tuple(lay((100 * normal(g, pages, page, heads, dim)).clamp(-448, 448).to(torch.float8_e4m3fn)) for _ in range(2))
    return codes + tuple(0.01 * torch.exp(0.5 * normal(g, pages, page, heads)) for _ in range(2))


def tables(g, lengths, page, spare=1):
    need = [-(-n // page) for n in lengths]
    order = torch.randperm(sum(need) + spare, generator=g, device=DEV).to(torch.int32)
    t = torch.full((len(lengths), max(max(need), 1) + 1), -1, device=DEV, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        t[i, :n] = order[at:at + n]
        at += n
    return t, sum(need) + spare


# ------------------------------------------------------------------- append

def spin(x, cos_sin, positions, rot, pairs, sign=1):
    """Rotation in 64 bits, and its elements' absolute terms."""
    half = rot // 2
    row = cos_sin.double()[positions.long()][:, None]
    c, s = row[..., :half], sign * row[..., half:]
    x = x.double()
    i, j = (slice(0, rot, 2), slice(1, rot, 2)) if pairs else (slice(0, half), slice(half, rot))
    y, mag = x.clone(), x.abs()
    y[..., i], y[..., j] = x[..., i] * c - x[..., j] * s, x[..., j] * c + x[..., i] * s
    mag = mag.clone()
    mag[..., i], mag[..., j] = (x[..., i] * c).abs() + (x[..., j] * s).abs(), (x[..., j] * c).abs() + (x[..., i] * s).abs()
    return y, mag


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("tokens,hq,hkv,dim,rot,page", [(1, 8, 1, 128, 128, 16), (5, 3, 3, 16, 16, 1), (67, 4, 2, 80, 32, 48),
                                                        (130, 6, 2, 64, 64, 7), (33, 2, 1, 112, 96, 128), (9, 2, 2, 48, 0, 4)])
def test_append(tokens, hq, hkv, dim, rot, page, pairs, e4m3):
    note(f"append {tokens}x{hq}/{hkv}x{dim} rot {rot} page {page} pairs {pairs} e4m3 {e4m3}")
    g = gen(tokens + dim)
    rows = normal(g, tokens, hq + 2 * hkv, dim).to(torch.bfloat16)
    q, k, v = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
    table = tar.rope_table(501, rot, device=DEV) if rot else torch.zeros(501, 0, device=DEV)
    pos = torch.randint(0, 501, (tokens,), generator=g, device=DEV).to(torch.int32)
    pages = -(-tokens // page) + 2
    cache = filled(g, pages, page, hkv, dim, e4m3)
    before = [c.clone() for c in cache]
    slots = torch.randperm(pages * page, generator=g, device=DEV)[:tokens]
    slots[torch.rand(tokens, generator=g, device=DEV) < 0.2] = -1
    if tokens > 4:
        slots[1] = pages * page                      # beyond the cache: nowhere
        slots[2] = 2 ** 40
    q_out, k_out = torch.empty(tokens, hq, dim, device=DEV, dtype=torch.bfloat16), torch.empty(tokens, hkv, dim, device=DEV, dtype=torch.bfloat16)
    tar.ar_rope_kv(q, k, v, table, pos, q_out=q_out, k_out=k_out, cache=cache, slots=slots, pairs=pairs)
    torch.cuda.synchronize()
    yq, mq = spin(q, table, pos, rot, pairs)
    yk, mk = spin(k, table, pos, rot, pairs)
    # two products and their sum in binary32, one rounding to bf16
    ref.close(q_out, yq, ref.U * yq.abs() + 3 * ref.E * mq, "q_out")
    ref.close(k_out, yk, ref.U * yk.abs() + 3 * ref.E * mk, "k_out")
    kept = [i for i in range(tokens) if 0 <= int(slots[i]) < pages * page]
    for i, (y, m) in enumerate(((yk, mk), (v.double(), v.double().abs()))):
        want, tol = before[i].to(torch.float32).double(), torch.zeros(before[i].shape, device=DEV, dtype=torch.float64)
        at = (slots[kept] // page, slots[kept] % page)
        if e4m3:
            amax, size = y[kept].abs().amax(2), 3 * ref.E * m[kept].amax(2)
            got = cache[2 + i][at].double()
            floor = torch.full_like(amax, 2.0 ** -126)
            ref.close(got, torch.maximum(amax / 448, floor), size / 448 + 3 * ref.E * amax / 448, "scales")
            # the codes of x / s for the scale that is kept: half a step of a
            # code, 2^-4 of it or 2^-10 below the normal codes, and what the
            # division by s and the rotation round
            x = y[kept] / got[..., None]
            want[at] = x
            tol[at] = torch.maximum(x.abs() * 2.0 ** -4, torch.full_like(x, 2.0 ** -10)) + (3 * ref.E * m[kept]) / got[..., None] + 3 * ref.E * x.abs()
            untouched = torch.ones(before[2].shape, device=DEV, dtype=torch.bool)
            untouched[at] = False
            assert torch.equal(cache[2 + i][untouched], before[2 + i][untouched])
        else:
            want[at], tol[at] = y[kept], ref.U * y[kept].abs() + 3 * ref.E * m[kept]
        ref.close(cache[i].to(torch.float32), want, tol, "cache")


@pytest.mark.parametrize("pairs", [False, True])
def test_rotation_in_place_and_back(pairs):
    g = gen(3)
    rows = normal(g, 41, 9, 64).to(torch.bfloat16)
    keep = rows.clone()
    q, k = rows[:, :6], rows[:, 6:8]                 # the ninth head is not touched
    table, pos = tar.rope_table(300, 64, device=DEV), torch.arange(41, device=DEV, dtype=torch.int32) * 7
    tar.ar_rope_kv(q, k, None, table, pos, q_out=q, k_out=k, pairs=pairs)
    torch.cuda.synchronize()
    y, m = spin(keep[:, :8], table, pos, 64, pairs)
    ref.close(rows[:, :8], y, ref.U * y.abs() + 3 * ref.E * m, "rotated")
    assert torch.equal(rows[:, 8], keep[:, 8])
    turned = rows.clone()
    tar.ar_rope_kv(None, k, None, table, pos, k_out=k, pairs=pairs, inverse=True)
    torch.cuda.synchronize()
    y, m = spin(turned[:, 6:8], table, pos, 64, pairs, -1)
    ref.close(rows[:, 6:8], y, ref.U * y.abs() + 3 * ref.E * m, "rotated back")
    assert torch.equal(rows[:, :6], turned[:, :6])


def test_append_no_numbers():
    """Infinities and NaN: as they are in bf16, the NaN code in E4M3 with a
    scale of the finite values; positions outside the table are held within."""
    g = gen(4)
    k, v = (normal(g, 3, 1, 32).to(torch.bfloat16) for _ in range(2))
    v[0, 0, 3], v[1, 0, 5], v[2] = math.inf, math.nan, 0.0
    k[2] = math.nan
    table, pos = tar.rope_table(8, 16, device=DEV), torch.tensor([-5, 7, 100], device=DEV, dtype=torch.int32)
    cache = filled(g, 2, 4, 1, 32, True)
    slots = torch.tensor([0, 5, 2], device=DEV)
    k_out = torch.empty_like(k)
    tar.ar_rope_kv(None, k, v, table, pos, k_out=k_out, cache=cache, slots=slots)
    torch.cuda.synchronize()
    y, m = spin(k[:2], table, torch.tensor([0, 7], device=DEV), 16, False)
    ref.close(k_out[:2], y, ref.U * y.abs() + 3 * ref.E * m, "k_out")
    codes, scales = cache[1].view(torch.uint8), cache[3]
    assert int(codes[0, 0, 0, 3]) == 0x7F and int(codes[1, 1, 0, 5]) == 0x7F
    x = v.float()
    x[0, 0, 3] = x[1, 0, 5] = 0
    for i, at in enumerate(((0, 0), (1, 1), (0, 2))):
        amax = float(x[i].abs().max())
        assert float(scales[at][0]) == pytest.approx(max(amax / 448, 2.0 ** -126), rel=2 ** -22)
    assert bool((codes[0, 2] == 0).all()) and bool((cache[0].view(torch.uint8)[0, 2] == 0x7F).all())


# ------------------------------------------------------------ single tokens

@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (100, 4), (130, 300), (5000, 1)])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hq,hkv,dim,page", [(8, 1, 128, 16), (6, 6, 64, 48), (40, 2, 80, 7), (10, 2, 16, 1), (2, 1, 112, 512)])
def test_decode(hq, hkv, dim, page, e4m3, window, sinks):
    note(f"decode {hq}/{hkv}x{dim} page {page} e4m3 {e4m3} window {window} sinks {sinks}")
    g = gen(hq + dim)
    lengths = [0, 1, 31, 32, 33, 127, 128, 129, 700, 1500]
    table, pages = tables(g, lengths, page)
    cache = filled(g, pages, page, hkv, dim, e4m3, "pthd" if page != 48 else "phtd")
    q = normal(g, len(lengths), hq, dim).to(torch.bfloat16)
    lens = torch.tensor(lengths, device=DEV, dtype=torch.int32)
    scale = 1.3 * dim ** -0.5
    ws = torch.zeros(tar.attn_decode_workspace(len(lengths), hq, hkv, dim), device=DEV, dtype=torch.uint8)
    res = []
    for w in (ws, None, ws):
        out, lse = torch.full_like(q, 7.0), torch.full((hq, len(lengths)), 7.0, device=DEV).t()
        tar.ar_attn_decode(q, cache, table, lens, out, scale=scale, window=window, sinks=sinks, lse=lse, workspace=w)
        res.append((out, lse))
    torch.cuda.synchronize()
    for i, n in enumerate(lengths):
        k, v = ref.paged(cache, table[i], n)
        for h in range(hq):
            want = ref.attend(q[i:i + 1, h], k[:, h // (hq // hkv)], v[:, h // (hq // hkv)], scale, window, sinks)
            for out, lse in res[:2]:
                ref.close(out[i:i + 1, h], want["out"], want["out_t"], f"out of {n} keys, head {h}")
                ref.close(lse[i:i + 1, h], want["lse"], want["lse_t"], f"lse of {n} keys, head {h}")
    assert torch.equal(res[0][0], res[2][0]) and torch.equal(res[0][1], res[2][1])


# ------------------------------------------------------------- next chunks

@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 4), (64, 130)])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hq,hkv,dim,page", [(8, 2, 128, 16), (3, 1, 64, 48), (4, 4, 80, 7)])
def test_chunks(hq, hkv, dim, page, e4m3, window, sinks):
    note(f"chunks {hq}/{hkv}x{dim} page {page} e4m3 {e4m3} window {window} sinks {sinks}")
    g = gen(hq * dim)
    new, total = [1, 5, 300, 0, 64, 20], [1, 900, 300, 77, 65, 12]   # the last: more queries than keys
    table, pages = tables(g, total, page)
    cache = filled(g, pages, page, hkv, dim, e4m3)
    n = sum(new)
    q = normal(g, n + 2, hq, dim).to(torch.bfloat16)
    offs = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], device=DEV, dtype=torch.int32)
    lens = torch.tensor(total, device=DEV, dtype=torch.int32)
    out, lse = torch.full_like(q, 7.0), torch.full((n + 2, hq), 7.0, device=DEV)
    tar.ar_attn_paged(q, cache, table, lens, offs, out, window=window, sinks=sinks, lse=lse)
    torch.cuda.synchronize()
    assert bool((out[n:] == 7.0).all()) and bool((lse[n:] == 7.0).all())
    for i, m in enumerate(new):
        k, v = ref.paged(cache, table[i], total[i])
        a = slice(int(offs[i]), int(offs[i + 1]))
        for h in range(hq):
            want = ref.attend(q[a, h], k[:, h // (hq // hkv)], v[:, h // (hq // hkv)], dim ** -0.5, window, sinks)
            ref.close(out[a, h], want["out"], want["out_t"], f"out of sequence {i}, head {h}")
            ref.close(lse[a, h], want["lse"], want["lse_t"], f"lse of sequence {i}, head {h}")
